"""GPU: 8-bit encoding of activations and the norm ahead of it against 64-bit forms: codes and scales equal the
definition's bit for bit, over odd widths, strides, empty and zero rows, infinities and NaN; streams and graphs."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = ("FP8_ROW", "FP8_GROUP128", "MXFP8")
WIDTHS = (32, 96, 512, 544, 2048, 4096, 4128, 12288, 16416, 25600, 33024)
ODD = (1, 7, 127, 129, 333, 5121)


def _x(m, d, dt, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(m, d, generator=g) * torch.exp(spread * torch.randn(m, 1, generator=g))).to(ref.DT[dt])


def _bits(t):
    return t.cpu().contiguous().view(torch.uint8) if t.dim() else t.cpu().reshape(1).view(torch.uint8)


def _check_codes(q, v, exact=True):
    """Codes and scales of the fp64 values v.  exact: bit for bit.  Otherwise (v itself carries an error of a few
    2^-24 in the kernel) a scale may differ by 2^-22 of itself, or one power of two where v's amax lies that near to
    one, and a code by one step where v / s lies that near to a middle: rare, and never more."""
    assert torch.equal(torch.tensor(q.data.shape), torch.tensor(v.shape))
    s, spread = ref.scale_of(q.kind, v)
    got_s = q.scale.cpu()
    want = ref.e4m3_codes(v / spread)
    got = _bits(q.data) & 127
    if exact:
        if q.kind == "MXFP8":
            assert torch.equal(got_s.view(torch.uint8), s)
        else:
            assert torch.equal(got_s, s)
        bad = got != want
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} codes differ, first at {bad.nonzero()[0].tolist()}"
    else:
        if q.kind == "MXFP8":
            assert (got_s.view(torch.uint8) != s).double().mean() < 1e-3
        else:
            assert ((got_s.double() - s.double()).abs() <= s.double() * 2.0 ** -22).all()
        step = (got.int() - want.int()).abs()
        assert step.max() <= 8 and (step > 0).double().mean() < 1e-3
    neg = (_bits(q.data) >= 128) & (got > 0) & (got < 127)
    assert not (neg & (v > 0)).any() and not ((got > 0) & (got < 127) & ~(_bits(q.data) >= 128) & (v < 0)).any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,d", [(1, w) for w in WIDTHS] + [(5, 544), (70, 2048), (3, 25600)])
def test_encode(kind, dt, m, d):
    print(f"encode {kind} {dt} {m} {d}", flush=True)
    x = _x(m, d, dt, d)
    _check_codes(st.quantize_activation(x.to(DEV), kind), x.double())


@pytest.mark.parametrize("kind", ["FP8_ROW", "FP8_GROUP128"])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("m,d", [(1, w) for w in ODD] + [(9, 333), (300, 129)])
def test_encode_odd_widths(kind, dt, m, d):
    print(f"encode odd {kind} {dt} {m} {d}", flush=True)
    x = _x(m, d, dt, d + 1)
    _check_codes(st.quantize_activation(x.to(DEV), kind), x.double())


@pytest.mark.parametrize("kind", KINDS)
def test_middles_go_to_even(kind):
    """Every middle between two codes and its neighbours, under a scale of exactly one: amax is 448."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (codes[1:] + codes[:-1]) / 2
    v = torch.cat([mid, torch.nextafter(mid.float(), torch.tensor(1e9)).double(), torch.nextafter(mid.float(), torch.tensor(0.0)).double()])
    v = torch.cat([v, -v])
    width = {"FP8_ROW": v.numel() + 1, "FP8_GROUP128": 128, "MXFP8": 32}[kind]
    rows = -(-v.numel() // (width - 1))
    x = torch.zeros(rows, width, dtype=torch.float64)
    for r in range(rows):
        part = v[r * (width - 1): (r + 1) * (width - 1)]
        x[r, 1: 1 + part.numel()] = part
        x[r, 0] = 448.0
    q = st.quantize_activation(x.float().to(DEV), kind)
    _check_codes(q, x)


@pytest.mark.parametrize("kind", KINDS)
def test_scale_of_three_keeps_middles(kind):
    """Quotients that are exact middles under a scale that is no power of two (1344 / 448 = 3; MX: the power above)."""
    t = torch.tensor([17.0, 19.0, 1.0625, 1.1875, 0.015625 * 1.0625, 27.0, -34.0, 2.0 ** -10, 3 * 2.0 ** -10])
    x = torch.zeros(4, 128)
    x[:, 0] = 1344.0
    x[:, 1: 1 + t.numel()] = 3 * t
    x[1, 40: 40 + t.numel()] = 3 * t
    q = st.quantize_activation(x.to(DEV), kind)
    _check_codes(q, x.double())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_zero_rows_and_what_is_not_finite(kind, dt):
    m, d = 6, 256
    x = _x(m, d, dt, 3, 0.5)
    x[0] = 0
    x[1, 10], x[1, 200], x[2, 33] = float("inf"), float("-inf"), float("nan")
    x[3] = float("nan")
    x[4, :128] = -0.0
    x[5] = torch.finfo(ref.DT[dt]).smallest_normal * torch.finfo(ref.DT[dt]).eps     # the smallest there is
    q = st.quantize_activation(x.to(DEV), kind)
    _check_codes(q, x.double())
    assert ((_bits(q.data) & 127) == 127).sum() == 3 + d
    assert (_bits(q.data)[0] == 0).all() and (_bits(q.data)[4, :128] & 127 == 0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_largest_values(kind):
    x = torch.full((2, 128), torch.finfo(torch.float32).max)
    x[1] = -x[1] / 3
    _check_codes(st.quantize_activation(x.to(DEV), kind), x.double())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt,m,d", [("bf16", 1, 4096), ("f16", 33, 544), ("bf16", 7, 25600), ("f32", 3, 1024)])
def test_encode_gated(kind, dt, m, d):
    print(f"gated {kind} {dt} {m} {d}", flush=True)
    x, g = _x(m, d, dt, 5, 0.5), _x(m, d, dt, 6, 0.5)
    v = x.double() * ref.activate("silu", g.double())
    _check_codes(st.quantize_activation(x.to(DEV), kind, gate=g.to(DEV)), v, exact=False)


def test_encode_strides_and_leading_dimensions():
    m, d = 12, 160
    for pad, off in ((8, 0), (3, 1)):
        wide = _x(m, d + pad + off, "bf16", 8)
        x = wide[:, off: off + d]
        for kind in KINDS:
            _check_codes(st.quantize_activation(wide.to(DEV)[:, off: off + d], kind), x.double())
    x = _x(12, 160, "f16", 9)
    q = st.quantize_activation(x.to(DEV).view(3, 4, 160), "FP8_GROUP128")
    assert q.shape == (3, 4, 160) and q.data.shape == (3, 4, 160) and q.scale.shape == (3, 4, 2)
    for kind in KINDS:
        e = st.quantize_activation(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), kind)
        assert e.data.shape == (0, 64)


# ------------------------------------------------------------------------------------------------ norm

def _norm_inputs(m, d, dt, seed, res, wt):
    g = torch.Generator().manual_seed(seed)
    x = _x(m, d, dt, seed, 1.0)
    r = _x(m, d, dt, seed + 1, 1.0) if res else None
    w = (1 + 0.1 * torch.randn(d, generator=g)).to(ref.DT[wt]) if wt else None
    return x, r, w


@pytest.mark.parametrize("dt,wt,res", [("bf16", "bf16", True), ("f16", "f32", False), ("f32", None, True), ("bf16", "f16", False)])
@pytest.mark.parametrize("m,d", [(1, w) for w in WIDTHS + ODD] + [(6, 512), (130, 1000), (5, 8192)])
def test_norm(dt, wt, res, m, d):
    print(f"norm {dt} {wt} {res} {m} {d}", flush=True)
    x, r, w = _norm_inputs(m, d, dt, d + m, res, wt)
    want, h = ref.rms_norm(x, w, 1e-6, r)
    for out in ("bf16", "f16", "f32"):
        got = st.rms_norm(x.to(DEV), ref.to(w, DEV), eps=1e-6, residual=ref.to(r, DEV), out_dtype=out)
        y, gh = got if res else (got, None)
        # h (one addition), the factor (rounded), two products: four roundings in fp32 and one to the output type
        t = torch.finfo(ref.DT[out])
        hs = x.double().abs() + (r.double().abs() if res else 0)      # the addition's own rounding is relative to h
        tol = want.abs() * (4 * 2.0 ** -24 * 1.01 + t.eps / 2) + t.smallest_normal * t.eps / 2
        assert ((y.cpu().double() - want).abs() <= tol).all()
        if res:
            th = torch.finfo(ref.DT[dt])
            assert gh.dtype == ref.DT[dt]
            assert ((gh.cpu().double() - h).abs() <= h.abs() * (2.0 ** -24 + th.eps / 2) + hs * 0 + th.smallest_normal * th.eps / 2).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt,wt,res", [("bf16", "bf16", True), ("f16", "f32", False)])
@pytest.mark.parametrize("m,d", [(1, 32), (1, 4096), (9, 544), (66, 2048), (3, 5120), (2, 25600), (2, 33024)])
def test_norm_encoded(kind, dt, wt, res, m, d):
    print(f"norm {kind} {dt} {res} {m} {d}", flush=True)
    x, r, w = _norm_inputs(m, d, dt, d + m, res, wt)
    want, h = ref.rms_norm(x, w, 1e-6, r)
    got = st.rms_norm(x.to(DEV), ref.to(w, DEV), eps=1e-6, residual=ref.to(r, DEV), quantize=kind)
    _check_codes(got[0] if res else got, want, exact=False)
    if res:
        assert torch.equal(got[1], st.rms_norm(x.to(DEV), ref.to(w, DEV), eps=1e-6, residual=ref.to(r, DEV))[1])


@pytest.mark.parametrize("kind", ["FP8_ROW", "FP8_GROUP128"])
@pytest.mark.parametrize("m,d", [(1, 1), (3, 333), (5, 5121)])
def test_norm_encoded_odd_widths(kind, m, d):
    x, r, w = _norm_inputs(m, d, "bf16", d, True, "bf16")
    want, _ = ref.rms_norm(x, w, 1e-6, r)
    _check_codes(st.rms_norm(x.to(DEV), w.to(DEV), residual=r.to(DEV), quantize=kind)[0], want, exact=False)


def test_norm_of_zero_and_nan_rows():
    x = _x(4, 512, "bf16", 4, 0.5)
    x[0] = 0
    x[2, 100] = float("nan")
    y = st.rms_norm(x.to(DEV), eps=1e-6).cpu()
    assert (y[0] == 0).all() and y[2].isnan().all() and y[1].isfinite().all() and y[3].isfinite().all()
    for kind in KINDS:
        q = st.rms_norm(x.to(DEV), eps=1e-6, quantize=kind)
        assert (_bits(q.data)[0] == 0).all() and ((_bits(q.data)[2] & 127) == 127).all()
        s = ref.e8m0(q.scale.cpu()) if kind == "MXFP8" else q.scale.cpu().double()
        assert (s[0] == 1).all() and (s[2] == 1).all()
    # a row of zeros without eps: 0 / 0
    assert st.rms_norm(x[:1].to(DEV), eps=0.0).isnan().all()


def test_norm_of_the_smallest_rows():
    """Rows whose factor 1 / rms lies beyond fp32, without eps."""
    x = torch.full((2, 64), 1e-44)
    x[1, ::2] = -3e-45
    want, _ = ref.rms_norm(x, None, 0.0, None)
    y = st.rms_norm(x.to(DEV), eps=0.0)
    assert ((y.cpu().double() - want).abs() <= want.abs() * 2.0 ** -24).all()
    for kind in KINDS:
        _check_codes(st.rms_norm(x.to(DEV), eps=0.0, quantize=kind), want, exact=False)


def test_encode_one_dimensional_and_without_columns():
    x = _x(1, 256, "bf16", 10)
    for kind in KINDS:
        q, q2 = st.quantize_activation(x[0].to(DEV), kind), st.quantize_activation(x.to(DEV), kind)
        assert q.shape == (256,) and torch.equal(_bits(q.data), _bits(q2.data)[0]) and torch.equal(_bits(q.scale).reshape(-1), _bits(q2.scale).reshape(-1))
        e = st.quantize_activation(torch.empty(3, 0, dtype=torch.bfloat16, device=DEV), kind)
        assert e.data.shape == (3, 0) and (kind != "FP8_ROW" or (e.scale == 1).all())


def test_encode_many_rows():
    """More rows than one grid dimension holds."""
    x = _x(70_001, 32, "bf16", 11, 0.5)
    for kind in KINDS:
        _check_codes(st.quantize_activation(x.to(DEV), kind), x.double())


@pytest.mark.parametrize("d", [512, 5120, 33024, 333])
@pytest.mark.parametrize("kind", [0, 2, 4])
@pytest.mark.parametrize("place", ["x", "residual"])
def test_h_in_place(d, kind, place):
    """Through the C entry: h may replace x or the residual."""
    import ctypes as C

    from device_checkpoint_dequantisation_amd import _lib
    m, d = 5, d if kind != 4 else -(-d // 32) * 32
    x, r, w = _norm_inputs(m, d, "bf16", 13, True, "bf16")
    dx, dr, dw = x.to(DEV), r.to(DEV), w.to(DEV)
    name = {0: None, 2: "FP8_ROW", 4: "MXFP8"}[kind]
    want, h = st.rms_norm(dx, dw, residual=dr, quantize=name)
    out = torch.zeros(m, d, dtype=torch.bfloat16 if kind == 0 else torch.uint8, device=DEV)
    scale = torch.zeros(m * d, dtype=torch.uint8, device=DEV)
    to = dx if place == "x" else dr
    a = _lib.RmsNormArgs(dx.data_ptr(), dr.data_ptr(), dw.data_ptr(), to.data_ptr(), out.data_ptr(), scale.data_ptr(), m, d, d, d,
                         1e-6, 0, 0, 0, kind)
    _lib.check(_lib.lib().st_rms_norm(C.byref(a), torch.cuda.current_stream().cuda_stream), "st_rms_norm")
    torch.cuda.synchronize()
    assert torch.equal(to, h)
    assert torch.equal(_bits(out), _bits(want if kind == 0 else want.data))


def test_calls_on_another_stream():
    x = _x(64, 4096, "bf16", 12)
    s = torch.cuda.Stream(DEV)
    dx = torch.zeros(64, 4096, dtype=torch.bfloat16, device=DEV)
    torch.cuda._sleep(20_000_000)
    dx.copy_(x.to(DEV))
    q = st.quantize_activation(dx, "MXFP8", stream=s)
    y, h = st.rms_norm(dx, residual=dx, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    _check_codes(q, x.double())
    assert torch.equal(y, st.rms_norm(x.to(DEV), residual=x.to(DEV))[0]) and torch.equal(h.cpu(), x * 2)


def test_norm_strided_rows_and_shapes():
    wide = _x(10, 700, "bf16", 6, 0.5).to(DEV)
    x = wide[:, 20:660]
    w = torch.rand(640, device=DEV)
    assert torch.equal(st.rms_norm(x, w), st.rms_norm(x.contiguous(), w))
    assert torch.equal(st.rms_norm(wide[:, 1:641], w), st.rms_norm(wide[:, 1:641].contiguous(), w))
    y = x.contiguous().view(2, 5, 640)
    assert torch.equal(st.rms_norm(y, w), st.rms_norm(x, w).view(2, 5, 640))
    assert torch.equal(st.rms_norm(y[0, 0], w), st.rms_norm(x, w)[0])
    assert st.rms_norm(torch.empty(0, 64, device=DEV)).shape == (0, 64)
    assert st.rms_norm(torch.empty(3, 0, device=DEV)).shape == (3, 0)


def test_rows_are_independent_of_the_batch():
    x, r, w = _norm_inputs(300, 1024, "bf16", 7, True, "bf16")
    x, r, w = x.to(DEV), r.to(DEV), w.to(DEV)
    q, h = st.rms_norm(x, w, residual=r, quantize="MXFP8")
    for i in (0, 1, 150, 299):
        q1, h1 = st.rms_norm(x[i:i + 1], w, residual=r[i:i + 1], quantize="MXFP8")
        assert torch.equal(_bits(q1.data), _bits(q.data[i:i + 1])) and torch.equal(h1, h[i:i + 1])


# ------------------------------------------------------------------------------------------------ together

def _block(x, h, wn, up, gate, down, kind):
    a, h = st.rms_norm(x, wn, residual=h, quantize=kind)
    u, g = st.linear(a, up), st.linear(a, gate)
    return st.linear(st.quantize_activation(u, kind, gate=g), down, residual=h), h


@pytest.mark.parametrize("kind,wk", [("FP8_ROW", "FP8_TENSOR"), ("FP8_GROUP128", "FP8_BLOCK128"), ("MXFP8", "MXFP8"), ("MXFP8", "MXFP4")])
@pytest.mark.parametrize("m", [1, 100])
def test_gated_block(kind, wk, m):
    """Norm, two products, gate, product and residual as a served layer runs them, eager and captured."""
    d, inter = 512, 1280
    x, h, wn = _norm_inputs(m, d, "bf16", 8, True, "bf16")
    ws = [ref.random_weight(st, wk, n, k, 9 + i) for i, (n, k) in enumerate(((inter, d), (inter, d), (d, inter)))]
    dev = [t.to(DEV) for t in (x, h, wn)] + [ref.to(w, DEV) for w in ws]
    out, dh = _block(*dev, kind)
    # each step against 64 bits, on what the step before it gave
    a, _ = st.rms_norm(dev[0], dev[2], residual=dev[1], quantize=kind)
    u, g = st.linear(a, dev[3]), st.linear(a, dev[4])
    ca = ref.to(a, "cpu")
    for got, w in ((u, ws[0]), (g, ws[1])):
        want, s = ref.linear(ca, w)
        assert ((got.cpu().double() - want).abs() <= ref.linear_tolerance(want, s, d, torch.bfloat16) + ref.f8_tolerance(ca, w)).all()
    q = ref.to(st.quantize_activation(u, kind, gate=g), "cpu")
    want, s = ref.linear(q, ws[2], residual=dh.cpu())
    assert ((out.cpu().double() - want).abs() <= ref.linear_tolerance(want, s, inter, torch.bfloat16) + ref.f8_tolerance(q, ws[2])).all()
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _block(*dev, kind)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, yh = _block(*dev, kind)
    for _ in range(3):
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, out) and torch.equal(yh, dh)
