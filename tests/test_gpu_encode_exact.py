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
