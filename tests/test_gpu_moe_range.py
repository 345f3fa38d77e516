"""GPU: experts whose act(gate) * up lies between bf16's largest number and fp32's."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import moe_reference as mref
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("m", [1, 2, 40, 300])
def test_between_the_largest_bf16_and_the_largest_fp32(m):
    """1023 * 2^118 rounds to an infinite bf16 number; down brings it back into range."""
    i, k, n = 32, 16, 24

    def weight(rows, cols, values, scale):
        w = torch.zeros(rows, cols)
        w[:, :len(values)] = torch.tensor(values)
        return st.QuantizedWeight("w", "FP8_TENSOR", (rows, cols), w.to(torch.float8_e4m3fn), torch.tensor(scale))
    down = weight(n, i, [1.0, -0.5, 0.25], 2.0 ** -100)
    lists = [[weight(i, k, [448.0, 448.0, 120.0, 7.0], 2.0 ** 59)] * 2, [weight(i, k, [0.0, 0.0, 0.0, 1.0], 2.0 ** 59)] * 2, [down] * 2]
    x = torch.ones(m, k, dtype=torch.bfloat16)
    x[1::2, 3] = -1.0                 # 1009 * 2^59 and -2^59
    ids, w = torch.arange(m, dtype=torch.int32).view(m, 1) % 2, torch.full((m, 1), 0.5)
    print(f"moe range {m}", flush=True)
    ex = st.MoeExperts(*([ref.to(a, DEV) for a in ws] for ws in lists))
    got = st.moe(x.to(DEV), ex, ids.to(DEV), w.to(DEV), activation=None, out_dtype="f32")
    want, tol = mref.moe(x, lists, ids, w, activation=None)
    assert (want.abs() > 2.0 ** 16).all() and (want.abs() < 2.0 ** 40).all()
    mref.check(got, want, tol)
