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
