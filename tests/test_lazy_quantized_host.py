"""CPU: modules that compute on quantised weights as stored (LazyModuleLoader(quantized=...)), with a state dict held in
memory and the operators' 64-bit forms in place of the kernels: what the replaced forwards pass on, and what attaching,
detaching and evicting leave behind."""
from types import SimpleNamespace

import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from device_checkpoint_dequantisation_amd import ops
from tests import ops_reference as ref


class _Memory(dict):
    """name -> QuantizedWeight or bf16 tensor, with a lazy state dict's methods."""

    def meta(self, name):
        t = self[name]
        return SimpleNamespace(shape=tuple(t.shape), kind=getattr(t, "kind", "PASS_BF16"))

    def meta_tensor(self, name):
        return torch.empty(tuple(self[name].shape), dtype=torch.bfloat16, device="meta")

    def load(self, names, stream=None):
        return {n: t if torch.is_tensor(t) else ref.weight_value(t).to(torch.bfloat16) for n, t in ((n, self[n]) for n in names)}

    def load_quantized(self, names, stream=None, copy=False):
        return {n: self[n] for n in names}


@pytest.fixture(autouse=True)
def _operators_in_64_bits(monkeypatch):
    def linear(x, w, bias=None, out_dtype=None):
        return ref.linear(x, w, bias=bias)[0].to(ref.DT[out_dtype])

    def rms_norm(x, weight=None, eps=1e-6):
        return ref.rms_norm(x, weight, eps, None)[0].to(x.dtype)
    monkeypatch.setattr(ops, "linear", linear)
    monkeypatch.setattr(ops, "rms_norm", rms_norm)


def _x(*shape, seed=1, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("eps", [None, 1e-5, 0.0])
def test_norm_uses_the_modules_eps(dtype, eps):
    """Rows from much smaller to much larger than the square root of any default eps, against the module's own forward."""
    weight = (1 + 0.1 * _x(64, seed=2, dtype=torch.float32)).to(torch.bfloat16)
    norm = torch.nn.RMSNorm(64, eps=eps, dtype=dtype)
    norm.weight.data.copy_(weight)
    x = torch.cat([_x(3, 64, dtype=torch.float32) * 10.0 ** e for e in (-4, -3, -2, -1, 0, 1)]).to(dtype)
    with torch.no_grad():
        want = norm(x).double()
    st.LazyModuleLoader(norm, _Memory(weight=weight), quantized="weights")
    got = norm(x).double()
    # both are rounded to x's type; torch's 32-bit form takes a handful of roundings of its own
    step = torch.finfo(dtype).eps / 2
    assert ((got - want).abs() <= want.abs() * (2 * step + 16 * 2.0 ** -24) + torch.finfo(dtype).smallest_normal * step * 2).all()
