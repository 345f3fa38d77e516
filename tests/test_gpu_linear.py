"""GPU: the matrix product over quantised weights against a 64-bit form: every weight kind with every encoding of
x it takes, from one row to several tiles, ragged sizes, rows that start anywhere, bias, activation, residual and
output types; exact results where every sum is exact; NaN and infinities; streams, graphs, refusals."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DENSE = [(x, w) for x in ("bf16", "f16") for w in ("FP8_TENSOR", "FP8_BLOCK128", "NVFP4", "MXFP8", "MXFP4")]
EIGHT = [("FP8_ROW", "FP8_TENSOR"), ("FP8_GROUP128", "FP8_BLOCK128"), ("MXFP8", "MXFP8"), ("MXFP8", "MXFP4")]
SHAPES = [(1, 1, 32), (1, 64, 128), (3, 65, 96), (16, 80, 512), (17, 129, 160), (64, 64, 640), (65, 130, 320),
          (130, 200, 1056), (5, 48, 4096), (257, 384, 256), (33, 16, 25600), (1, 40, 2080), (11, 24, 1568)]
ODD_K = [(1, 5, 1), (2, 3, 15), (7, 33, 131), (66, 70, 257), (200, 128, 1001), (1, 30, 1039), (1, 7, 5003), (16, 40, 2311), (3, 65, 513)]   # fp8 kinds: any K


def _check(x, w, got, k, **kw):
    want, s = ref.linear(x, w, **kw)
    tol = ref.linear_tolerance(want, s, k, got.dtype)
    if not torch.is_tensor(x) and got.dtype != torch.float32:
        tol = tol + ref.f8_tolerance(x, w)
    err = (got.cpu().double().reshape(want.shape) - want).abs()
    assert (err <= tol).all(), f"worst error {(err / tol).max().item():.3g} of what is allowed, at {int((err / tol).argmax())}"


def _run(x, w, **kw):
    return st.linear(ref.to(x, DEV), ref.to(w, DEV), **{k: ref.to(v, DEV) if torch.is_tensor(v) else v for k, v in kw.items()})


@pytest.mark.parametrize("xk,wk", DENSE + EIGHT)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_product(xk, wk, m, n, k):
    print(f"linear {xk} {wk} {m} {n} {k}", flush=True)
    x, w = ref.random_rows(st, xk, m, k, 1), ref.random_weight(st, wk, n, k, 2)
    _check(x, w, _run(x, w, out_dtype="f32"), k)
    _check(x, w, _run(x, w), k)


@pytest.mark.parametrize("xk,wk", [p for p in DENSE + EIGHT if p[1].startswith("FP8")])
@pytest.mark.parametrize("m,n,k", ODD_K)
def test_odd_k(xk, wk, m, n, k):
    print(f"linear odd {xk} {wk} {m} {n} {k}", flush=True)
    x, w = ref.random_rows(st, xk, m, k, 3), ref.random_weight(st, wk, n, k, 4)
    _check(x, w, _run(x, w, out_dtype="f32"), k)
    _check(x, w, _run(x, w), k)


@pytest.mark.parametrize("xk", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1, 33, 16), (4, 20, 48), (70, 65, 5136), (1, 34, 5136), (9, 33, 2608)])
def test_nvfp4_k_of_16(xk, m, n, k):
    print(f"linear nvfp4 {xk} {m} {n} {k}", flush=True)
    x, w = ref.random_rows(st, xk, m, k, 5), ref.random_weight(st, "NVFP4", n, k, 6)
    _check(x, w, _run(x, w, out_dtype="f32"), k)


@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("out,bt,rt", [("bf16", "bf16", "bf16"), ("f16", "f32", "f16"), ("f32", "f16", "bf16")])
@pytest.mark.parametrize("m,n", [(1, 70), (19, 128), (100, 67)])
def test_epilogue(act, out, bt, rt, m, n):
    k = 256
    g = torch.Generator().manual_seed(7)
    x, w = ref.random_rows(st, "bf16", m, k, 8), ref.random_weight(st, "FP8_TENSOR", n, k, 9)
    b, r = torch.randn(n, generator=g).to(ref.DT[bt]), torch.randn(m, n, generator=g).to(ref.DT[rt])
    for kw in ({"bias": b}, {"residual": r}, {"bias": b, "residual": r}):
        print(f"epilogue {act} {out} {m} {n} {list(kw)}", flush=True)
        got = _run(x, w, activation=act, out_dtype=out, **kw)
        assert got.dtype == ref.DT[out]
        _check(x, w, got, k, activation=act, **kw)


def _whole(wk, xk, m, n, k, seed):
    """Operands of small whole numbers and powers of two: every partial sum is exact in fp32."""
    g = torch.Generator().manual_seed(seed)
    w, x = ref.random_weight(st, wk, n, k, seed), ref.random_rows(st, xk, m, k, seed + 1)
    small = torch.tensor([0.0, 1.0, -1.0, 2.0, -2.0, 3.0, -4.0, 0.5])
    pick = lambda *s: small[torch.randint(0, 8, s, generator=g)]   # noqa: E731
    if wk in ("FP8_TENSOR", "FP8_BLOCK128", "MXFP8"):
        w.data = pick(n, k).to(torch.float8_e4m3fn)
    two = lambda s: 2.0 ** torch.randint(-2, 3, s, generator=g)    # noqa: E731
    if wk in ("FP8_TENSOR", "FP8_BLOCK128"):
        w.scale = two(tuple(w.scale.shape)).float()
    elif wk == "NVFP4":
        w.scale, w.scale2 = two(tuple(w.scale.shape)).float().to(torch.float8_e4m3fn), torch.tensor(0.5)
    else:
        w.scale = torch.randint(125, 130, tuple(w.scale.shape), generator=g, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    if xk in ref.DT:
        x = pick(m, k).to(ref.DT[xk])
    else:
        x.data = pick(m, k).to(torch.float8_e4m3fn)
        x.scale = (torch.randint(125, 130, tuple(x.scale.shape), generator=g, dtype=torch.uint8).view(torch.float8_e8m0fnu)
                   if xk == "MXFP8" else two(tuple(x.scale.shape)).float())
    return x, w


@pytest.mark.parametrize("xk,wk", DENSE + EIGHT)
@pytest.mark.parametrize("m,n,k", [(1, 48, 512), (2, 130, 1280), (16, 64, 640), (31, 65, 384), (140, 300, 768), (260, 520, 192)])
def test_exact_sums(xk, wk, m, n, k):
    """Sums of multiples of 2^-8 below 2^16 have no rounding in fp32, whatever the order: equal bits."""
    print(f"exact {xk} {wk} {m} {n} {k}", flush=True)
    x, w = _whole(wk, xk, m, n, k, 11)
    want, s = ref.linear(x, w)
    assert s.max() < 2.0 ** 16
    assert torch.equal(_run(x, w, out_dtype="f32").cpu().double(), want)
    # products of magnitudes within 2^-13 of each other lose nothing in any instruction either: one rounding
    assert torch.equal(_run(x, w, out_dtype="f16").cpu(), want.to(torch.float16))


@pytest.mark.parametrize("xk,wk", DENSE + EIGHT)
@pytest.mark.parametrize("m,n,k", [(20, 70, 32), (50, 65, 96), (40, 70, 2080), (130, 140, 160), (200, 300, 1056), (140, 130, 5152)])
@pytest.mark.parametrize("at", [0, 1])
def test_partial_last_step(xk, wk, m, n, k, at):
    """Rows that start and end on 16 bytes with K off the tiles' steps, the scale words on and off 4 bytes."""
    print(f"tail {xk} {wk} {m} {n} {k} {at}", flush=True)
    x, w = ref.random_rows(st, xk, m, k, 51), ref.random_weight(st, wk, n, k, 52)
    xd, wd = ref.to(x, DEV), ref.to(w, DEV)
    for t in (xd, wd):
        if at and not torch.is_tensor(t) and t.scale.dtype != torch.float32:
            raw = torch.empty(t.scale.numel() + 1, dtype=torch.uint8, device=DEV)[1:]
            raw.copy_(t.scale.view(torch.uint8).flatten())
            t.scale = raw.view(t.scale.dtype).view(t.scale.shape)
    _check(x, w, st.linear(xd, wd, out_dtype="f32"), k)
    _check(x, w, st.linear(xd, wd), k)


@pytest.mark.parametrize("xk,wk", DENSE + EIGHT)
@pytest.mark.parametrize("m,n,k", [(4100, 4097, 160), (4096, 4352, 416)])
def test_many_tiles_partial_last_step(xk, wk, m, n, k):
    """As test_many_tiles."""
    test_many_tiles(xk, wk, m, n, k)


@pytest.mark.parametrize("xk,wk", DENSE + EIGHT)
@pytest.mark.parametrize("m,n,k", [(1500, 1100, 256), (4100, 4097, 128), (4096, 4352, 384)])
def test_many_tiles(xk, wk, m, n, k):
    """Whole and ragged bands of tiles, of every tile size; the 64-bit products on the GPU."""
    print(f"tiles {xk} {wk} {m} {n} {k}", flush=True)
    x, w = ref.random_rows(st, xk, m, k, 41), ref.random_weight(st, wk, n, k, 42)
    b = ref.weight_value(w).to(DEV)
    a = (x.double() if xk in ref.DT else ref.rows_value(x.kind, x.data, x.scale)).to(DEV)
    want, s = torch.mm(a, b.t().contiguous()), torch.mm(a.abs(), b.abs().t().contiguous())
    for out in ("bf16", "f32"):
        y = _run(x, w, out_dtype=out)
        tol = ref.linear_tolerance(want, s, k, y.dtype)
        if xk not in ref.DT and out == "bf16":
            tol = tol + ref.f8_tolerance(x, w).to(DEV)
        assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("xk,wk,m", [("bf16", "FP8_TENSOR", 1), ("bf16", "FP8_TENSOR", 3), ("FP8_ROW", "FP8_TENSOR", 40), ("f16", "FP8_TENSOR", 200)])
def test_weight_past_four_gibibytes(xk, wk, m):
    """Rows of the weight whose bytes lie past 2^32."""
    n, k = 140_000, 32_768
    x = ref.random_rows(st, xk, m, k, 43)
    data = torch.zeros(n, k, dtype=torch.uint8, device=DEV)
    tail = ref.random_codes(torch.Generator().manual_seed(44), 70, k)
    data[n - 70:] = tail.view(torch.uint8).to(DEV)
    assert (n - 70) * k > 2 ** 32
    scale = torch.tensor(0.25)
    w = st.QuantizedWeight("w", wk, (n, k), data.view(torch.float8_e4m3fn), scale.to(DEV))
    y = st.linear(ref.to(x, DEV), w, out_dtype="f32")
    assert (y[:, : n - 70] == 0).all()
    _check(x, st.QuantizedWeight("w", wk, (70, k), tail, scale), y[:, n - 70:], k)


@pytest.mark.parametrize("xk,wk", [("bf16", "NVFP4"), ("f16", "MXFP8"), ("bf16", "FP8_BLOCK128"), ("MXFP8", "MXFP4")])
def test_one_hot_places_every_element(xk, wk):
    """Row i of x is one at column 37 i + 5: y is that column of the weight, rounded."""
    m, n, k = 40, 150, 1536
    w = ref.random_weight(st, wk, n, k, 12)
    x = ref.random_rows(st, xk, m, k, 13)
    hot = torch.zeros(m, k)
    cols = (torch.arange(m) * 37 + 5) % k
    hot[torch.arange(m), cols] = 1.0
    if xk in ref.DT:
        x = hot.to(ref.DT[xk])
    else:
        x.data = hot.to(torch.float8_e4m3fn)
        x.scale = torch.full_like(x.scale.view(torch.uint8), 127).view(torch.float8_e8m0fnu)
    got = _run(x, w, out_dtype="f32").cpu()
    assert torch.equal(got, ref.weight_value(w)[:, cols].t().float())


@pytest.mark.parametrize("xk,wk", [("bf16", "FP8_TENSOR"), ("f16", "NVFP4"), ("bf16", "MXFP4"), ("MXFP8", "MXFP8"),
                                   ("FP8_GROUP128", "FP8_BLOCK128")])
@pytest.mark.parametrize("m", [1, 5, 20])
def test_weights_and_rows_at_any_byte(xk, wk, m):
    """Weights and scales as views into a blob at odd offsets, dense rows at an odd pitch."""
    n, k = 70, 320
    x, w = ref.random_rows(st, xk, m, k, 14), ref.random_weight(st, wk, n, k, 15)
    dw = ref.to(w, DEV)
    for f in ("data",) + (("scale",) if w.scale.element_size() == 1 else ()):
        t = getattr(w, f)
        raw = t.contiguous().view(torch.uint8).reshape(-1)
        blob = torch.zeros(raw.numel() + 64, dtype=torch.uint8, device=DEV)
        blob[3: 3 + raw.numel()] = raw.to(DEV)
        setattr(dw, f, blob[3: 3 + raw.numel()].view(t.dtype).view(t.shape))
    dx = ref.to(x, DEV)
    if xk in ref.DT:
        wide = torch.full((m, k + 13), float("nan"), dtype=ref.DT[xk], device=DEV)
        wide[:, 5: 5 + k] = dx
        dx = wide[:, 5: 5 + k]
    print(f"offsets {xk} {wk} {m}", flush=True)
    _check(x, w, st.linear(dx, dw, out_dtype="f32"), k)


def test_strided_out_and_residual_and_rows_behind():
    m, n, k = 37, 61, 256
    x, w = ref.random_rows(st, "bf16", m, k, 16), ref.random_weight(st, "MXFP8", n, k, 17)
    g = torch.Generator().manual_seed(18)
    r = torch.randn(m, n, generator=g)
    for off, pitch in ((0, 64), (1, 67)):
        buf = torch.full((m + 2, pitch), 7.0, device=DEV)
        out = buf[1: 1 + m, off: off + n]
        out.copy_(r)
        got = st.linear(ref.to(x, DEV), ref.to(w, DEV), residual=out, out=out)     # in place
        assert got is out
        _check(x, w, out, k, residual=r)
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[1: 1 + m, off: off + n] = False
        assert (buf[keep] == 7.0).all()
    # a residual row added to every row
    row = torch.randn(n, generator=g)
    got = st.linear(ref.to(x, DEV), ref.to(w, DEV), residual=row.to(DEV).expand(m, n), out_dtype="f32")
    _check(x, w, got, k, residual=row.expand(m, n))


def test_leading_dimensions_and_empty():
    w = ref.random_weight(st, "FP8_TENSOR", 24, 64, 19)
    dw = ref.to(w, DEV)
    x = ref.random_rows(st, "bf16", 12, 64, 20)
    y = st.linear(x.to(DEV).view(3, 4, 64), dw)
    assert y.shape == (3, 4, 24) and torch.equal(y.view(12, 24), st.linear(x.to(DEV), dw))
    assert torch.equal(st.linear(x[0].to(DEV), dw), st.linear(x[:1].to(DEV), dw)[0])
    assert st.linear(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), dw).shape == (0, 24)
    none = st.QuantizedWeight("w", "FP8_TENSOR", (0, 64), torch.empty(0, 64, dtype=torch.float8_e4m3fn, device=DEV),
                              torch.ones((), device=DEV))
    assert st.linear(x.to(DEV), none).shape == (12, 0)
    # K = 0: an empty sum, then the epilogue
    b = torch.arange(24.0) - 12
    flat = st.QuantizedWeight("w", "FP8_TENSOR", (24, 0), torch.empty(24, 0, dtype=torch.float8_e4m3fn, device=DEV),
                              torch.ones((), device=DEV))
    got = st.linear(torch.empty(5, 0, dtype=torch.bfloat16, device=DEV), flat, bias=b.to(DEV), activation="relu")
    assert torch.equal(got.cpu().float(), b.clamp_min(0).expand(5, 24))
    for xk, wk in DENSE + EIGHT:
        w = ref.random_weight(st, wk, 24, 0, 1)
        for m in (1, 5, 70):
            got = _run(ref.random_rows(st, xk, m, 0, 2), w, bias=b)
            assert torch.equal(got.cpu().float(), b.expand(m, 24))


@pytest.mark.parametrize("xk,wk", DENSE + EIGHT)
@pytest.mark.parametrize("m", [2, 70])
def test_nan_and_infinity_stay_where_they_belong(xk, wk, m):
    n, k = 66, 512
    x, w = ref.random_rows(st, xk, m, k, 21), ref.random_weight(st, wk, n, k, 22)
    if wk in ("FP8_TENSOR", "FP8_BLOCK128", "MXFP8"):
        w.data.view(torch.uint8)[5, 300] = 0x7F                        # a NaN code: column 5 of y
    elif wk == "NVFP4":
        w.scale.view(torch.uint8)[5, 300 // 16] = 0x7F
    else:
        w.scale.view(torch.uint8)[5, 300 // 32] = 0xFF
    if xk in ref.DT:
        x[1, 7] = float("inf")                                          # row 1 of y: infinite or NaN
    else:
        x.data.view(torch.uint8)[1, 7] = 0xFF
    print(f"nan {xk} {wk} {m}", flush=True)
    got = _run(x, w, out_dtype="f32").cpu()
    want, _ = ref.linear(x, w)
    assert torch.equal(got.isfinite(), want.isfinite()) and torch.equal(got.isnan(), want.isnan())
    rows = [i for i in range(m) if i != 1]
    assert got[rows][:, [c for c in range(n) if c != 5]].isfinite().all() and got[0, 5].isnan()


def test_extreme_mx_scales():
    """E8M0 codes 0 and 254, whose products lie at the ends of fp32's range."""
    n, k, m = 32, 128, 3
    for wk, xk in (("MXFP8", "bf16"), ("MXFP4", "bf16"), ("MXFP8", "f16")):
        w = ref.random_weight(st, wk, n, k, 23)
        x = torch.full((m, k), 2.0 ** -14, dtype=ref.DT[xk])
        w.scale = torch.full((n, k // 32), 254 - 20, dtype=torch.uint8).view(torch.float8_e8m0fnu)
        w.scale.view(torch.uint8)[::2] = 40
        _check(x, w, _run(x, w, out_dtype="f32"), k)


def test_other_stream_and_order():
    m, n, k = 8, 512, 2048
    x, w = ref.random_rows(st, "bf16", m, k, 24), ref.to(ref.random_weight(st, "NVFP4", n, k, 25), DEV)
    s = torch.cuda.Stream(DEV)
    dx = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
    torch.cuda._sleep(20_000_000)
    dx.copy_(x.to(DEV))                    # behind the sleep on the current stream: the call has to wait for it
    y = st.linear(dx, w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, st.linear(x.to(DEV), w))


@pytest.mark.parametrize("xk,wk,m", [("bf16", "NVFP4", 1), ("MXFP8", "MXFP8", 40), ("f16", "FP8_BLOCK128", 130)])
def test_captured_calls_replay(xk, wk, m):
    """Two captured products, each with its own workspace, replayed in turn with eager work between."""
    n, k = 256, 8192
    w = ref.to(ref.random_weight(st, wk, n, k, 26), DEV)
    xs = [ref.to(ref.random_rows(st, xk, m, k, 27 + i), DEV) for i in range(2)]
    eager = [st.linear(x, w, activation="silu") for x in xs]
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for x in xs:
            st.linear(x, w, activation="silu")
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graphs = []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = st.linear(x, w, activation="silu")
        graphs.append((g, y))
    for _ in range(4):
        for (g, y), want in zip(graphs, eager):
            y.fill_(3.0)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want)


def test_two_streams_at_once():
    """Products whose K is split, on two streams at the same time: each has its own workspace."""
    w = ref.to(ref.random_weight(st, "NVFP4", 256, 16384, 50), DEV)
    xs = [ref.random_rows(st, "bf16", m, 16384, 51).to(DEV) for m in (4, 40)]
    want = [st.linear(x, w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in xs]
    got = [[], []]
    for _ in range(8):
        for i, (x, s) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(s):
                got[i].append(st.linear(x, w))
    torch.cuda.synchronize()
    for ys, y in zip(got, want):
        assert all(torch.equal(t, y) for t in ys)


def test_refusals_on_the_gpu():
    x, w = ref.random_rows(st, "bf16", 4, 64, 52).to(DEV), ref.to(ref.random_weight(st, "FP8_TENSOR", 64, 64, 53), DEV)
    with pytest.raises(ValueError, match="overlaps"):
        st.linear(x, w, out=x)
    buf = torch.zeros(5, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        st.linear(x, w, residual=buf[:4], out=buf[1:])
    with pytest.raises(ValueError, match="stride 1"):
        st.linear(torch.zeros(64, 4, dtype=torch.bfloat16, device=DEV).t(), w)
    with pytest.raises(ValueError, match="bias"):
        st.linear(x, w, bias=torch.zeros(63, device=DEV))
    with pytest.raises(ValueError, match="residual"):
        st.linear(x, w, residual=torch.zeros(64, device=DEV))
    with pytest.raises(ValueError, match="tensors on"):
        st.linear(x, w, bias=torch.zeros(64))
    with pytest.raises(ValueError, match="activation"):
        st.linear(x, w, activation="tanh")
    with pytest.raises(ValueError, match="out_dtype"):
        st.linear(x, w, out_dtype="f64")
    with pytest.raises(ValueError, match="out is"):
        st.linear(x, w, out=buf[:4], out_dtype="f32")
    with pytest.raises(RuntimeError, match="no backward"):
        st.linear(x.clone().requires_grad_(), w)
    with pytest.raises(ValueError, match="residual"):
        st.rms_norm(x, residual=x.float())
    with pytest.raises(ValueError, match="gate"):
        st.quantize_activation(x, "MXFP8", gate=x[:2])
    with pytest.raises(ValueError, match="exclude"):
        st.rms_norm(x, quantize="MXFP8", out_dtype="f32")


def test_same_bits_every_time():
    """K split over workgroups joins in a fixed order."""
    x, w = ref.random_rows(st, "bf16", 4, 16384, 30).to(DEV), ref.to(ref.random_weight(st, "FP8_TENSOR", 100, 16384, 31), DEV)
    first = st.linear(x, w, out_dtype="f32")
    for _ in range(5):
        assert torch.equal(st.linear(x, w, out_dtype="f32"), first)


def test_workspace_is_checked_by_the_library():
    import ctypes as C

    from device_checkpoint_dequantisation_amd import _lib
    x, w = ref.random_rows(st, "bf16", 4, 16384, 30).to(DEV), ref.to(ref.random_weight(st, "FP8_TENSOR", 100, 16384, 31), DEV)
    out = torch.zeros(4, 100, device=DEV)
    a = _lib.LinearArgs(x.data_ptr(), None, w.data.data_ptr(), w.scale.data_ptr(), None, None, None, out.data_ptr(), None, 0, 4, 100,
                        16384, 16384, 0, 100, 0, 3, 0, 0, 0, 2)
    need = C.c_uint64()
    assert _lib.lib().st_linear_workspace_bytes(C.byref(a), C.byref(need)) == 0
    if need.value:
        assert _lib.lib().st_linear(C.byref(a), None) == -1
        work = torch.empty(need.value, dtype=torch.uint8, device=DEV)
        a.workspace, a.workspace_bytes = work.data_ptr(), need.value - 1
        assert _lib.lib().st_linear(C.byref(a), None) == -1
    torch.cuda.synchronize()
    assert (out == 0).all()
