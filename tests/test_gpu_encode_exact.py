"""GPU: codes, scales and norms where they are decided: gates far below zero, sums that fp32 cannot hold, and every code
of random rows equal to the 64-bit definition's."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import ops_reference as ref
from tests.test_gpu_encode import _bits, _check_codes

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = ("FP8_ROW", "FP8_GROUP128", "MXFP8")


def _silu(g):
    return ref.activate("silu", g.double())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt,far,near", [("f16", 6e4, 1e3), ("bf16", 6e4, 1e3), ("f32", 6e4, 1e3), ("bf16", 1e30, 1e3), ("f32", 1e38, 1.0)])
def test_gates_far_below_zero(kind, dt, far, near):
    """One element per row (a wavefront's worth of columns) with a gate from -80 to -110 and a large x, among elements of
    -80: its value, down to 1e-46 of x, is not lost."""
    print(f"far gates {kind} {dt} {far}", flush=True)
    gates = torch.arange(-80.0, -110.25, -0.25)
    m, d = gates.numel(), 512
    g = torch.full((m, d), -80.0)
    x = near * (1 + torch.rand(m, d, generator=torch.Generator().manual_seed(1)))
    at = (torch.arange(m) * 37 + 5) % d
    g[torch.arange(m), at], x[torch.arange(m), at] = gates, -far
    g, x = g.to(ref.DT[dt]), x.to(ref.DT[dt])
    _check_codes(st.quantize_activation(x.to(DEV), kind, gate=g.to(DEV)), x.double() * _silu(g))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("spread", [1.0, 20.0])
def test_gated_codes_equal_the_definition(kind, dt, spread):
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(96, 4096, generator=g) * 30).to(ref.DT[dt])
    gate = (torch.randn(96, 4096, generator=g) * spread).to(ref.DT[dt])
    _check_codes(st.quantize_activation(x.to(DEV), kind, gate=gate.to(DEV)), x.double() * _silu(gate))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gates_that_almost_pass_x(kind, dt):
    """x / s at every middle between two codes and gates from 20 to 40: silu(gate) lies below the gate by 2^-24 to 2^-53 of
    itself, and so does the value below the middle."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = torch.cat([(codes[1:] + codes[:-1]) / 2, torch.tensor([448.0, 0.0])])
    gates = torch.tensor([20.0, 24.0, 26.0, 28.0, 30.0, 31.0, 32.0, 34.0, 36.0, 37.0, 40.0, 64.0])
    x = torch.zeros(gates.numel(), 128 * 32)
    g = gates[:, None].expand_as(x).clone()
    x.view(-1, 128, 32)[:, :, 7] = mid.float()           # a group of 32 or 128 around each, its largest value at the end
    x.view(-1, 128, 32)[:, :, 31] = 448.0
    # an fp32 scale is the gate itself (448 silu(gate) / 448, rounded), a power of two at or above it
    x, g = x.to(ref.DT[dt]), g.to(ref.DT[dt])
    assert (x.double().view(-1, 128, 32)[:, :, 7] == mid).all()
    _check_codes(st.quantize_activation(x.to(DEV), kind, gate=g.to(DEV)), x.double() * _silu(g))


# ------------------------------------------------------------------------------------------------ norm

def _norm_rows(m, d, dt, seed):
    """Rows and a residual whose sums mostly do not fit fp32's 24 bits."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(m, d, generator=g)
    r = torch.randn(m, d, generator=g) * 2.0 ** (-torch.randint(6, 20, (m, d), generator=g).float())
    return x.to(ref.DT[dt]), r.to(ref.DT[dt]), 1 + 0.1 * torch.randn(d, generator=g)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,d", [(40, 512), (20, 1000), (9, 5120), (3, 33024), (5, 333)])
def test_norm_of_the_unrounded_sum(dt, m, d):
    """An fp32 result is the 64-bit one rounded once: half a step, and 2^-40 for the 64-bit sum in another order."""
    x, r, w = _norm_rows(m, d, dt, d)
    want, h = ref.rms_norm(x, w, 1e-6, r)
    y, gh = st.rms_norm(x.to(DEV), w.to(DEV), eps=1e-6, residual=r.to(DEV), out_dtype="f32")
    assert ((y.cpu().double() - want).abs() <= want.abs() * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150).all()
    assert torch.equal(gh.cpu(), h.to(ref.DT[dt]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,d", [(96, 4096), (40, 5120), (7, 33024)])
def test_norm_codes_equal_the_definition(kind, dt, m, d):
    x, r, w = _norm_rows(m, d, dt, d + 1)
    want, _ = ref.rms_norm(x, w, 1e-6, r)
    _check_codes(st.rms_norm(x.to(DEV), w.to(DEV), eps=1e-6, residual=r.to(DEV), quantize=kind)[0], want)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 544])
def test_norm_of_sums_beyond_fp32(dt, d):
    """x + residual past fp32's largest number: h is infinite in x's type, y is not."""
    x = (3e38 * torch.where(torch.arange(d) % 3 == 0, -1.0, 1.0)).repeat(3, 1).to(ref.DT[dt])
    want, _ = ref.rms_norm(x, None, 1e-6, x)
    y, h = st.rms_norm(x.to(DEV), eps=1e-6, residual=x.to(DEV), out_dtype="f32")
    assert ((y.cpu().double() - want).abs() <= want.abs() * 2.0 ** -23).all() and h.isinf().all()
    for kind in KINDS:
        q, h = st.rms_norm(x.to(DEV), eps=1e-6, residual=x.to(DEV), quantize=kind)
        _check_codes(q, want)
        assert h.isinf().all() and ((_bits(q.data) & 127) != 127).all()


# ------------------------------------------------------------------------------------------------ more rows than one launch takes

@pytest.mark.parametrize("d", [7, 32])
def test_more_rows_than_one_launch_takes(d):
    """Past 2^32 threads and 2^22 workgroups, of one row (odd width) or of four: every form of the output, next to the parts'
    ends against the same rows by themselves."""
    m = (2 ** 24 if d == 32 else 2 ** 22) * 2 + 3
    x = torch.randn(m, d, generator=torch.Generator(DEV).manual_seed(7), device=DEV).to(torch.bfloat16)
    r = x.flip(0)
    w = torch.rand(d, device=DEV)
    parts = [slice(max(0, a - 300), a + 300) for a in range(0, m, 2 ** 22)] + [slice(m - 300, m)]
    if d == 7:
        grid = 2 ** 24 + 3        # past 2^32 threads in workgroups of 256
        big = torch.randn(grid, 1, generator=torch.Generator(DEV).manual_seed(8), device=DEV).to(torch.bfloat16)
        q = st.quantize_activation(big, "FP8_ROW")
        assert torch.equal(q.data.float().abs(), torch.where(big == 0, 0.0, 448.0)) and torch.equal(q.scale, torch.where(big == 0, 1.0, big.double().abs() / 448)[:, 0].float())
    for kind in (None, "FP8_ROW", "FP8_GROUP128") + (("MXFP8",) if d == 32 else ()):
        print(f"many rows {kind} {d}", flush=True)
        y, h = st.rms_norm(x, w, eps=1e-6, residual=r, quantize=kind)
        q = None if kind is None else st.quantize_activation(x, kind)
        assert torch.equal(h, x + r)
        for p in parts:
            y1, _ = st.rms_norm(x[p].contiguous(), w, eps=1e-6, residual=r[p].contiguous(), quantize=kind)
            if kind is None:
                assert torch.equal(y[p], y1)
                continue
            for whole, one in ((y, y1), (q, st.quantize_activation(x[p].contiguous(), kind))):
                assert torch.equal(whole.data[p].view(torch.uint8), one.data.view(torch.uint8))
                assert torch.equal(whole.scale[p].view(torch.uint8), one.scale.view(torch.uint8))


# ------------------------------------------------------------------------------------------------ layouts

@pytest.mark.parametrize("d", [512, 333])
def test_one_row_for_all_and_an_input_in_two_places(d):
    """Rows, residuals and gates broadcast from one row, rows far apart, and x as its own residual and gate."""
    m = 9
    g = torch.Generator().manual_seed(9)
    x, r = (torch.randn(m, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    far = torch.zeros(m, 2 ** 21 + 24, dtype=torch.bfloat16, device=DEV)
    far[:, 8: 8 + d] = x
    for kind in (None, "FP8_ROW", "FP8_GROUP128") + (("MXFP8",) if d % 32 == 0 else ()):
        for a, b in ((x[:1].expand(m, d), r), (x, r[:1].expand(m, d)), (x, x), (far[:, 8: 8 + d], r)):
            ca, cb = a.contiguous(), b.contiguous().clone()
            y, h = st.rms_norm(a, residual=b, quantize=kind)
            z, hz = st.rms_norm(ca, residual=cb, quantize=kind)
            assert torch.equal(h, hz)
            pairs = [(y, z)] if kind is None else [(y.data, z.data), (y.scale, z.scale)]
            if kind is not None:
                q, p = st.quantize_activation(a, kind, gate=b), st.quantize_activation(ca, kind, gate=cb)
                pairs += [(q.data, p.data), (q.scale, p.scale)]
            for s, t in pairs:
                assert torch.equal(_bits(s), _bits(t))
