"""GPU: products where errors of the sums or of the epilogue show: sums of whole numbers through split and long K, the
sums' own error under a residual that takes the result away, activations relative to their value."""
import math

import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import ops_reference as ref
from tests.test_gpu_linear import DENSE, EIGHT, _run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("m", [1, 5, 40, 130])
def test_activations_relative_to_their_value(act, m):
    """Arguments from -10 to 10, given by the bias over a product of zeros."""
    v = torch.linspace(-10, 10, 2001)
    w = ref.random_weight(st, "FP8_TENSOR", v.numel(), 64, 1)
    got = _run(torch.zeros(m, 64, dtype=torch.bfloat16), w, bias=v, activation=act, out_dtype="f32").cpu().double()
    d = v.double()
    # in steps of 2^-24 of the value.  gelu: 0.5 v erfc(z), z = -v / sqrt 2 to 1.5 steps, which erfc, falling like exp(-z^2),
    # takes (2 z^2 + 1) times; erfc itself to 16 steps.  silu: exp to 3 steps, a sum, a division.  gelu_tanh: as silu of
    # u = v (a + b v^2), u to 4 steps, which exp takes |u| times.
    steps, want = {
        "relu": (torch.zeros_like(d), d.clamp_min(0)),
        "silu": (3 * d.abs() + 10, d * torch.sigmoid(d)),
        "gelu": ((d * d + 1) * 1.5 + 35, 0.5 * d * torch.special.erfc(-d / math.sqrt(2))),
        "gelu_tanh": (4 * 1.5957691216057308 * (d * (1 + 0.044715 * d * d)).abs() + 12,
                      d * torch.sigmoid(1.5957691216057308 * d * (1 + 0.044715 * d * d))),
    }[act]
    bad = (got - want).abs() > want.abs() * steps * 2.0 ** -24 + 2.0 ** -149
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, first at {v[bad.nonzero()[0, 1]].item()}"


def _hot(xk, m, k, p):
    """Rows that are p = 2^e at one column each."""
    hot = torch.zeros(m, k, dtype=torch.float64)
    cols = (torch.arange(m) * 37 + 5) % k
    hot[torch.arange(m), cols] = p if xk in ref.DT else 1.0
    if xk in ref.DT:
        return hot.to(ref.DT[xk]), cols
    s = torch.full((m, k // 32), 127 + int(math.log2(p)), dtype=torch.uint8).view(torch.float8_e8m0fnu)
    return st.QuantizedActivation(xk, (m, k), hot.to(torch.float8_e4m3fn), s), cols


@pytest.mark.parametrize("xk,wk", [(x, w) for x in ("bf16", "f16", "MXFP8") for w in ("MXFP8", "MXFP4")])
@pytest.mark.parametrize("m", [1, 5, 40, 130])
def test_mx_scales_at_both_ends(xk, wk, m):
    """Every E8M0 code, with weights whose values fp32 holds, times a power of two that keeps the product in range.  Values
    below 2^-126 are taken to multiples of 2^-133, bf16's smallest step."""
    k, n = 256, 64
    for code in (0, 1, 2, 3, 10, 120, 246, 247, 250, 253, 254):
        w = ref.random_weight(st, wk, n, k, code)
        w.scale = torch.full((n, k // 32), code, dtype=torch.uint8).view(torch.float8_e8m0fnu)
        if code > 240:        # magnitudes below 2 (and codes of them alone)
            keep = 0x3F if wk == "MXFP8" else None
            w.data = ((w.data.view(torch.uint8) & (keep | 0x80)).view(torch.float8_e4m3fn) if keep else w.data & 0xBB)
        v = ref.weight_value(w)
        assert (v.abs() < 2.0 ** 128).all()
        p = 2.0 ** -14 if code > 64 else 2.0 ** 15
        x, cols = _hot(xk, m, k, p)
        print(f"mx ends {xk} {wk} {m} {code}", flush=True)
        got = _run(x, w, out_dtype="f32").cpu().double()
        want = v.to(torch.bfloat16).double()[:, cols].t() * p
        assert torch.equal(got, want)
        if xk == "MXFP8" and m > 64:      # the scaled instructions take the value as it is
            got = _run(x, w, out_dtype="bf16").cpu()
            assert torch.equal(got, (v[:, cols].t() * p).to(torch.bfloat16))


@pytest.mark.parametrize("xk,wk", DENSE + EIGHT)
@pytest.mark.parametrize("m,n,k", [(1, 70, 25600), (3, 96, 25600), (16, 64, 12288), (48, 130, 25600), (130, 200, 25600), (300, 520, 5120)])
def test_exact_sums_through_long_and_split_k(xk, wk, m, n, k):
    """Whole and half numbers through K of many steps, split over workgroups where the output is small, with tensor and
    row scales of 24 bits: every sum is exact in fp32, so the result is that sum times the scales, each product rounded
    once; a weight or a partial sum held in fewer bits shows."""
    print(f"long exact {xk} {wk} {m} {n} {k}", flush=True)
    g = torch.Generator().manual_seed(k + m)
    small = torch.tensor([0.0, 1.0, -1.0, 2.0, -2.0, 0.5, -0.5, 1.5])
    pick = lambda *s: small[torch.randint(0, 8, s, generator=g)]   # noqa: E731
    two = lambda s: torch.randint(126, 129, tuple(s), generator=g, dtype=torch.uint8)   # noqa: E731
    w, x = ref.random_weight(st, wk, n, k, 1), ref.random_rows(st, xk, m, k, 2)
    if wk in ("NVFP4", "MXFP4"):
        w.data = w.data & 0xBB                          # magnitudes up to 1.5
    else:
        w.data = pick(n, k).to(torch.float8_e4m3fn)
    tail = torch.ones(())                                # what multiplies the finished sum
    if wk == "FP8_TENSOR":
        w.scale = tail = torch.tensor(1.0 + 2.0 ** -12 + 2.0 ** -23)
    elif wk == "NVFP4":
        w.scale = (2.0 ** (two(w.scale.shape).float() - 127)).to(torch.float8_e4m3fn)
        w.scale2 = tail = torch.tensor(1.0 + 2.0 ** -11 + 2.0 ** -22)
    elif wk == "FP8_BLOCK128":
        w.scale = 2.0 ** (two(w.scale.shape).float() - 127)
    else:
        w.scale = two(w.scale.shape).view(torch.float8_e8m0fnu)
    rows = torch.ones(m, 1)
    if xk in ref.DT:
        x = pick(m, k).to(ref.DT[xk])
    else:
        x.data = pick(m, k).to(torch.float8_e4m3fn)
        if xk == "MXFP8":
            x.scale = two(x.scale.shape).view(torch.float8_e8m0fnu)
        elif xk == "FP8_GROUP128":
            x.scale = 2.0 ** (two(x.scale.shape).float() - 127)
        else:
            x.scale = 1 + torch.rand(m, generator=g)
            rows = x.scale[:, None]
    bare = st.QuantizedWeight("w", wk, (n, k), w.data, w.scale if tail is not w.scale else torch.ones(()),
                              None if w.scale2 is None else torch.ones(()))
    plain = x if xk != "FP8_ROW" else st.QuantizedActivation(xk, (m, k), x.data, torch.ones(m))
    total, s = ref.linear(plain, bare)
    assert s.max() < 2.0 ** 20                           # in steps of 2^-4 at the least: below 2^24 of them
    want = total.float() * tail * rows
    assert torch.equal(_run(x, w, out_dtype="f32").cpu(), want)


def _under_residual(xk, wk, m, n, k, out):
    """A product under a residual that takes its result away, in a 16-bit type: what is left shows the sums' own error.
    Returns (error, what fp32 sums and the rounding of the rest may be off by, sum |x w|)."""
    x, w = ref.random_rows(st, xk, m, k, 3), ref.random_weight(st, wk, n, k, 4)
    a, b = (x.double() if xk in ref.DT else ref.rows_value(x.kind, x.data, x.scale)).to(DEV), ref.weight_value(w).to(DEV)
    want, s = torch.mm(a, b.t().contiguous()), torch.mm(a.abs(), b.abs().t().contiguous())
    back = -want.float()
    left = want + back.double()                          # what rounding `back` left
    err = (_run(x, w, residual=back, out_dtype=out).double() - left).abs()
    # cutting what is below 2^-13 of the largest of 16 products: for bf16 from 8-bit rows only
    cut = ref.f8_tolerance(x, w).to(DEV) * (1 + 2.0 ** -8) if xk not in ref.DT and out == "bf16" else 0.0
    return err, ref.linear_tolerance(left, s + back.abs().double(), k, ref.DT[out]) + cut, s


@pytest.mark.parametrize("xk,wk", DENSE + EIGHT)
@pytest.mark.parametrize("out", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1, 200, 1056), (40, 200, 4096), (70, 130, 4096), (100, 200, 25600), (4096, 4352, 1056)])
def test_sums_under_a_residual(xk, wk, out, m, n, k):
    """fp32 sums for every 16-bit result but bf16 from 8-bit rows, whose scaled instructions cut from the sums no more than
    2^-13 of the largest of 16 neighbouring products for each of the others."""
    print(f"sums {xk} {wk} {m} {n} {k} {out}", flush=True)
    err, tol, s = _under_residual(xk, wk, m, n, k, out)
    print(f"  off by up to {(err / s).max().item():.2g}, rms {(err / s).square().mean().sqrt().item():.2g} of sum |x w|", flush=True)
    assert (err <= tol).all()


@pytest.mark.parametrize("xk,wk", EIGHT)
@pytest.mark.parametrize("m,n,k", [(100, 512, 4096), (4096, 4352, 1056)])
def test_fp16_results_of_8_bit_rows_have_fp32_sums(xk, wk, m, n, k):
    """The error of K / 32 matrix instructions that add 32 products each in fp32 (8 roundings or cuts of 2^-23 allowed for
    each, and 32 for joining, scales and epilogue), of which the average, not the worst element, is held: 2^-24 of the sum of
    magnitudes for each of sqrt(8 K / 32 + 32) steps that err independently, and twice that."""
    err, _, s = _under_residual(xk, wk, m, n, k, "f16")
    assert (err / s).square().mean().sqrt() <= 2 * 2.0 ** -24 * math.sqrt(8 * k / 32 + 32)


@pytest.mark.parametrize("m", [1, 7, 70])
def test_out_beside_its_input_in_one_buffer(m):
    """x, residual and out as columns of one buffer: out's are written, the others and what lies between left as they were."""
    k, n = 128, 64
    x, w = ref.random_rows(st, "bf16", m, k, 5), ref.to(ref.random_weight(st, "FP8_TENSOR", n, k, 6), DEV)
    r = torch.randn(m, n, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).to(DEV)
    buf = torch.full((m, k + 2 * n + 16), 3.0, dtype=torch.bfloat16, device=DEV)
    buf[:, :k], buf[:, k + n: k + 2 * n] = x.to(DEV), r
    before = buf.clone()
    want = st.linear(x.to(DEV), w, residual=r)
    st.linear(buf[:, :k], w, residual=buf[:, k + n: k + 2 * n], out=buf[:, k: k + n])
    assert torch.equal(buf[:, k: k + n], want)
    buf[:, k: k + n] = 3.0
    assert torch.equal(buf, before)
    with pytest.raises(ValueError, match="overlaps"):
        st.linear(buf[:, :k], w, out=buf[:, k - 1: k - 1 + n])


@pytest.mark.parametrize("xk,wk", DENSE)
@pytest.mark.parametrize("m", [1, 5, 20, 130])
def test_rows_far_apart_and_one_row_for_all(xk, wk, m):
    """Rows of x, residual and out more than 4 MiB apart (past the tiles' 32-bit offsets), and one row read for every row."""
    n, k = 70, 256
    x, w = ref.random_rows(st, xk, m, k, 8), ref.to(ref.random_weight(st, wk, n, k, 9), DEV)
    r = torch.randn(m, n, generator=torch.Generator().manual_seed(10)).to(ref.DT[xk])
    pitch = 2 ** 21 + 24
    print(f"far rows {xk} {wk} {m}", flush=True)
    far = torch.full((m, pitch), 5.0, dtype=ref.DT[xk], device=DEV)
    far[:, 8: 8 + k], far[:, 1000: 1000 + n] = x.to(DEV), r.to(DEV)
    want = st.linear(x.to(DEV), w, residual=r.to(DEV))
    st.linear(far[:, 8: 8 + k], w, residual=far[:, 1000: 1000 + n], out=far[:, 2000: 2000 + n])
    assert torch.equal(far[:, 2000: 2000 + n], want) and (far[:, 2000 + n:] == 5.0).all() and (far[:, 1000 + n: 2000] == 5.0).all()
    del far
    one = st.linear(x[:1].to(DEV).expand(m, k), w, residual=r[:1].to(DEV).expand(m, n))
    assert torch.equal(one, st.linear(x[:1].repeat(m, 1).to(DEV), w, residual=r[:1].repeat(m, 1).to(DEV)))


@pytest.mark.parametrize("m", [1, 9, 100])
def test_an_input_in_two_places(m):
    """x as the residual too, and the bias a row of it."""
    d = 256
    x, w = ref.random_rows(st, "bf16", m, d, 11), ref.random_weight(st, "MXFP4", d, d, 12)
    dx = x.to(DEV)
    got = st.linear(dx, ref.to(w, DEV), bias=dx[0], residual=dx, activation="silu", out_dtype="f32").cpu().double()
    want, s = ref.linear(x, w, bias=x[0], residual=x, activation="silu")
    assert ((got - want).abs() <= ref.linear_tolerance(want, s, d, torch.float32)).all()
