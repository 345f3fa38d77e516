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


def _checkpoint(seed, bias=True):
    sd = _Memory(weight=ref.random_weight(st, "FP8_TENSOR", 24, 64, seed))
    if bias:
        sd["bias"] = _x(24, seed=seed + 100)
    return sd


def _linear(bias=True):
    return torch.nn.Linear(64, 24, bias=bias, device="meta", dtype=torch.bfloat16)


def _decoded(sd, x):
    return torch.nn.functional.linear(x, ref.weight_value(sd["weight"]).to(torch.bfloat16), sd.get("bias"))


def test_another_checkpoint_after_detach():
    """A module that another checkpoint is attached to computes with that checkpoint's weight, whichever loader it had before."""
    a, b = _checkpoint(1), _checkpoint(2)
    lin, x = _linear(), _x(5, 64, seed=3)
    for evict in (False, True):
        loader = st.LazyModuleLoader(lin, a, quantized="weights")
        want = ops.linear(x, a["weight"], bias=a["bias"], out_dtype="bf16")
        assert torch.equal(lin(x), want)
        if evict:
            loader.evict_all()
        loader.detach()
        assert "forward" not in lin.__dict__
        plain = st.LazyModuleLoader(lin, b)
        assert torch.equal(lin(x), _decoded(b, x))
        plain.detach()
        assert torch.equal(lin(x), _decoded(b, x))


def test_detach_leaves_a_meta_weight_and_counts_it_out():
    a = _checkpoint(1)
    lin, x = _linear(), _x(5, 64, seed=3)
    loader = st.LazyModuleLoader(lin, a, quantized="weights")
    lin(x)
    stored = a["weight"].data.numel() + 4
    assert loader.resident_bytes == stored + 48
    loader.detach()
    assert lin.weight.is_meta and not lin.bias.is_meta and loader.resident_bytes == 48
    loader.materialize(lin)                      # by hand: decoded, as without `quantized`
    assert torch.equal(lin(x), _decoded(a, x)) and loader.resident_bytes == 48 + 2 * 24 * 64
    lin.weight = torch.nn.Parameter(torch.zeros(24, 64, dtype=torch.bfloat16), requires_grad=False)
    assert torch.equal(lin(x), a["bias"].expand(5, 24))


def test_a_weight_assigned_while_attached_is_used():
    a = _checkpoint(1)
    lin, x = _linear(), _x(5, 64, seed=3)
    loader = st.LazyModuleLoader(lin, a, quantized="weights")
    lin(x)
    lin.weight = torch.nn.Parameter(torch.zeros(24, 64, dtype=torch.bfloat16), requires_grad=False)
    assert torch.equal(lin(x), a["bias"].expand(5, 24))
    loader.detach()


def test_a_module_takes_one_quantized_loader_at_a_time():
    a, b = _checkpoint(1), _checkpoint(2)
    lin, x = _linear(), _x(5, 64, seed=3)
    loader = st.LazyModuleLoader(lin, a, quantized="weights")
    want = lin(x)
    for mode in (None, "weights", "activations"):
        with pytest.raises(ValueError, match="detach"):
            st.LazyModuleLoader(lin, b, quantized=mode)
    assert torch.equal(lin(x), want)
    loader.detach()
    st.LazyModuleLoader(lin, b, quantized="weights")
    assert torch.equal(lin(x), ops.linear(x, b["weight"], bias=b["bias"], out_dtype="bf16"))


def test_a_copy_of_a_module_is_its_own():
    """copy.deepcopy copies the loader along: copy and original stay apart, and neither outlives its detach."""
    import copy
    a = _checkpoint(1)
    root = torch.nn.Sequential(_linear())
    loader = st.LazyModuleLoader(root, _Memory({"0." + k: v for k, v in a.items()}), quantized="weights")
    x = _x(5, 64, seed=3)
    want = root(x)
    twin = copy.deepcopy(root)
    twin[0].bias.data.zero_()
    assert torch.equal(root(x), want)
    assert torch.equal(twin(x), ops.linear(x, a["weight"], out_dtype="bf16"))
    loader.detach()
    root[0].weight = torch.nn.Parameter(torch.zeros(24, 64, dtype=torch.bfloat16), requires_grad=False)
    assert torch.equal(root(x), a["bias"].expand(5, 24)) and torch.equal(twin(x), ops.linear(x, a["weight"], out_dtype="bf16"))


def test_a_forward_kept_by_a_wrapper_is_the_modules_own_after_detach():
    a = _checkpoint(1)
    lin, x = _linear(), _x(5, 64, seed=3)
    loader = st.LazyModuleLoader(lin, a, quantized="weights")
    inner = lin.forward
    lin.forward = lambda t: 2 * inner(t)
    assert torch.equal(lin(x), 2 * ops.linear(x, a["weight"], bias=a["bias"], out_dtype="bf16"))
    loader.detach()
    with pytest.raises(RuntimeError, match="not loaded"):
        inner(x)
    loader.materialize(lin)
    assert torch.equal(lin(x), 2 * _decoded(a, x))


def test_a_failed_attach_replaces_no_forward():
    sd = _Memory({"0.weight": ref.random_weight(st, "FP8_TENSOR", 24, 64, 1), "1.weight": ref.random_weight(st, "FP8_TENSOR", 24, 32, 1)})
    root = torch.nn.Sequential(_linear(bias=False), torch.nn.Linear(24, 8, bias=False, device="meta"))
    with pytest.raises(ValueError, match="checkpoint shape"):
        st.LazyModuleLoader(root, sd, quantized="weights")
    assert "forward" not in root[0].__dict__


def test_norms_forward_goes_with_its_loader():
    weight = torch.full((64,), 2.0, dtype=torch.bfloat16)
    norm, x = torch.nn.RMSNorm(64, eps=1e-6, device="meta", dtype=torch.bfloat16), _x(3, 64)
    loader = st.LazyModuleLoader(norm, _Memory(weight=weight), quantized="weights")
    assert "forward" in norm.__dict__ and torch.equal(norm(x), ops.rms_norm(x, weight))
    loader.detach()
    assert "forward" not in norm.__dict__ and not norm.weight.is_meta


def test_a_forward_of_the_instance_is_left_alone():
    """An adapter's forward, set on the module itself, runs as before, on the decoded weight."""
    a = _checkpoint(1)
    lin, x = _linear(), _x(5, 64, seed=3)
    lin.forward = lambda t: 3 * torch.nn.functional.linear(t, lin.weight, lin.bias)
    patched = lin.forward
    loader = st.LazyModuleLoader(lin, a, quantized="weights")
    assert lin.forward is patched and torch.equal(lin(x), 3 * _decoded(a, x))
    loader.detach()
    assert lin.forward is patched
    norm = torch.nn.RMSNorm(64, eps=1e-6, device="meta", dtype=torch.bfloat16)
    norm.forward = lambda t: t
    st.LazyModuleLoader(norm, _Memory(weight=torch.ones(64, dtype=torch.bfloat16)), quantized="weights")
    assert norm(x) is x


def test_inputs_by_name():
    """nn.Linear.forward names its argument input, nn.RMSNorm.forward x."""
    a = _checkpoint(1)
    lin, x = _linear(), _x(5, 64, seed=3)
    st.LazyModuleLoader(lin, a, quantized="weights")
    assert torch.equal(lin(input=x), lin(x))
    norm = torch.nn.RMSNorm(64, eps=1e-6, device="meta", dtype=torch.bfloat16)
    st.LazyModuleLoader(norm, _Memory(weight=torch.ones(64, dtype=torch.bfloat16)), quantized="weights")
    assert torch.equal(norm(x=x), norm(x))


def test_a_failed_load_counts_nothing():
    """A stored weight that cannot be read leaves its module as it was, bias and byte counts included."""
    a = _checkpoint(1)
    lin, x = _linear(), _x(5, 64, seed=3)
    loader = st.LazyModuleLoader(lin, a, quantized="weights")

    def broken(names, stream=None, copy=False):
        raise OSError("short read")
    a.load_quantized = broken
    with pytest.raises(OSError, match="short read"):
        lin(x)
    assert lin.bias.is_meta and loader.resident_bytes == 0
    del a.load_quantized
    assert torch.equal(lin(x), ops.linear(x, a["weight"], bias=a["bias"], out_dtype="bf16"))
    assert loader.resident_bytes == a["weight"].data.numel() + 4 + 48
    loader.evict_all()
    assert loader.resident_bytes == 0 and lin.bias.is_meta


def test_inputs_of_any_layout(monkeypatch):
    """nn.Linear and nn.RMSNorm take transposed and overlapping rows; the operators get adjacent ones."""
    inner = {n: getattr(ops, n) for n in ("linear", "rms_norm")}

    def adjacent(name):
        def call(x, *args, **kw):
            rows, pitch = ops._rows(x, x.shape[-1], "x", name)      # refuses what the operator refuses
            assert rows.shape[0] == 1 or pitch == 0 or pitch >= x.shape[-1]
            return inner[name](x, *args, **kw)
        return call
    for n in inner:
        monkeypatch.setattr(ops, n, adjacent(n))
    a = _checkpoint(1)
    lin, norm = _linear(), torch.nn.RMSNorm(64, eps=1e-6, device="meta", dtype=torch.bfloat16)
    st.LazyModuleLoader(lin, a, quantized="weights")
    st.LazyModuleLoader(norm, _Memory(weight=torch.ones(64, dtype=torch.bfloat16)), quantized="weights")
    long = _x(64 * 8)
    for x in (_x(64, 5).t(), long.unfold(0, 64, 8), long[::8], long[:64].expand(3, 64), _x(2, 64, 5).transpose(1, 2)):
        for mod in (lin, norm):
            assert torch.equal(mod(x), mod(x.contiguous()))


@pytest.mark.parametrize("mode", [None, "weights"])
def test_a_module_left_without_its_weight_refuses_to_run(mode):
    """torch computes with a meta weight without a word, and returns memory nobody wrote: a detached module whose weight is not
    loaded says so instead, until it has one again."""
    a, b = _checkpoint(1), _checkpoint(2)
    lin, x = _linear(), _x(5, 64, seed=3)
    for again in ("by hand", "assigned", "another loader", "another quantized loader"):
        loader = st.LazyModuleLoader(lin, a, quantized=mode)
        lin(x)
        loader.evict_all()
        loader.detach()
        for _ in range(2):
            with pytest.raises(RuntimeError, match="weight.*not loaded"):
                lin(x)
        if again == "by hand":
            loader.materialize(lin)
            assert torch.equal(lin(x), _decoded(a, x))
        elif again == "assigned":
            lin.weight = torch.nn.Parameter(torch.zeros(24, 64, dtype=torch.bfloat16), requires_grad=False)
            lin.bias = torch.nn.Parameter(a["bias"], requires_grad=False)
            assert torch.equal(lin(x), a["bias"].expand(5, 24))
        else:
            other = st.LazyModuleLoader(lin, b, quantized="weights" if "quantized" in again else None)
            lin(x)
            assert len(lin._forward_pre_hooks) == 1
            other.materialize(lin)
            other.detach()
            if other.quantized is None:
                assert torch.equal(lin(x), _decoded(b, x))
        if again != "another quantized loader":
            assert not lin._forward_pre_hooks
    del lin._forward_pre_hooks[next(iter(lin._forward_pre_hooks))]


def test_a_fully_loaded_module_keeps_no_hook_after_detach():
    a = _checkpoint(1)
    lin, x = _linear(), _x(5, 64, seed=3)
    loader = st.LazyModuleLoader(lin, a)
    lin(x)
    loader.detach()
    assert not lin._forward_pre_hooks and torch.equal(lin(x), _decoded(a, x))


def test_attention_whose_projection_is_read_by_its_owner():
    """nn.MultiheadAttention reads its out_proj's weight and never calls that module: it stays a decoded weight."""
    attn = torch.nn.MultiheadAttention(64, 4, bias=False, batch_first=True, device="meta", dtype=torch.bfloat16)
    sd = _Memory({"in_proj_weight": _x(192, 64, seed=4), "out_proj.weight": ref.random_weight(st, "FP8_TENSOR", 64, 64, 5)})
    x = _x(2, 3, 64, seed=6)
    got = []
    for mode in (None, "weights", "activations"):
        loader = st.LazyModuleLoader(attn, sd, quantized=mode)
        loader.materialize(attn.out_proj)
        assert not attn.out_proj.weight.is_meta
        with torch.no_grad():
            got.append(attn(x, x, x, need_weights=False)[0])
        loader.evict_all()
        loader.detach()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2]) and got[0].isfinite().all()
