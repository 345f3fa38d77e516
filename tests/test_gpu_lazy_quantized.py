"""GPU: modules that compute on quantised weights as stored (LazyModuleLoader(quantized=...)): linears and norms
against 64-bit forms of the checkpoint's own bytes, residency and eviction, prefix views and sharded checkpoints,
modules that are left alone, and refusals."""
import pytest
import torch

import synth
import device_checkpoint_dequantisation_amd as st
from tests import ops_reference as ref
from tests.st_files import write_sharded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# config -> (prefix of a linear, shape, weight kind), with the kind its inputs take
LINEARS = {2: ("blocks.1.attn.q", (320, 320), "FP8_TENSOR", "FP8_ROW"),
           3: ("model.layers.1.mlp.down_proj", (320, 960), "FP8_BLOCK128", "FP8_GROUP128"),
           4: ("model.layers.0.mlp.up_proj", (400, 208), "NVFP4", None),
           6: ("model.layers.0.mlp.gate_proj", (960, 320), "MXFP8", "MXFP8"),
           7: ("model.layers.1.mlp.down_proj", (224, 416), "MXFP4", "MXFP8")}


def _module(k):
    name, (n, kk), _, _ = LINEARS[k]
    root = torch.nn.Module()
    at = root
    parts = name.split(".")
    for p in parts[:-1]:
        nxt = torch.nn.Module()
        at.add_module(p, nxt)
        at = nxt
    at.add_module(parts[-1], torch.nn.Linear(kk, n, bias=k == 2, device="meta", dtype=torch.bfloat16))
    return root, getattr(at, parts[-1])


def _file(tmp_path, k):
    path = tmp_path / f"c{k}.safetensors"
    path.write_bytes(synth.config_bytes(k, small=True))
    return str(path)


@pytest.mark.parametrize("k", sorted(LINEARS))
@pytest.mark.parametrize("mode", ["weights", "activations"])
def test_linear_runs_on_stored_weights(k, mode, tmp_path):
    name, (n, kk), kind, encode = LINEARS[k]
    sd = st.StreamStateDict(_file(tmp_path, k), DEV)
    root, lin = _module(k)
    loader = st.LazyModuleLoader(root, sd, quantized=mode)
    assert lin.weight.is_meta and loader.resident_bytes == 0
    stored = ref.to(sd.load_quantized([name + ".weight"])[name + ".weight"], "cpu")
    assert stored.kind == kind
    bias = sd[name + ".bias"].cpu() if k == 2 else None
    print(f"stored linear c{k} {mode}", flush=True)
    for shape in ((1,), (3, 5), (70,)):
        x = torch.randn(*shape, kk, generator=torch.Generator().manual_seed(k)).to(torch.bfloat16)
        y = lin(x.to(DEV))
        assert y.shape == (*shape, n) and y.dtype == torch.bfloat16 and lin.weight.is_meta
        rows = x.reshape(-1, kk)
        if mode == "activations" and encode:
            rows = ref.to(st.quantize_activation(rows.to(DEV), encode), "cpu")
        want, s = ref.linear(rows, stored, bias=bias)
        tol = ref.linear_tolerance(want, s, kk, torch.bfloat16)
        if not torch.is_tensor(rows):
            tol = tol + ref.f8_tolerance(rows, stored)
        assert ((y.cpu().double().reshape(want.shape) - want).abs() <= tol).all()
    size = sum(t.numel() * t.element_size() for t in (stored.data, stored.scale, stored.scale2) if t is not None)
    assert loader.resident_bytes == size + (2 * n if k == 2 else 0)
    loader.evict_all()
    assert loader.resident_bytes == 0 and all(p.is_meta for p in root.parameters())
    again = lin(x.to(DEV))                    # loads once more
    assert torch.equal(again, y) and loader.stats["evicted"] == 1
    loader.detach()


def test_norms_run_through_the_operator_and_others_are_left_alone(tmp_path):
    sd = st.StreamStateDict(_file(tmp_path, 3), DEV)

    class Scaled(torch.nn.Linear):
        def forward(self, x):
            return 2 * torch.nn.functional.linear(x, self.weight)

    root = torch.nn.Module()
    root.norm = torch.nn.RMSNorm(320, eps=1e-5, device="meta", dtype=torch.bfloat16)
    root.q = Scaled(320, 320, bias=False, device="meta", dtype=torch.bfloat16)
    root.embed = torch.nn.Linear(320, 1000, bias=False, device="meta", dtype=torch.bfloat16)      # a bf16 weight
    names = {"norm.weight": "model.layers.0.input_layernorm.weight", "q.weight": "model.layers.0.self_attn.q_proj.weight",
             "embed.weight": "model.embed_tokens.weight"}
    view = st.RenameViewStateDict(sd, {v: k for k, v in names.items()})
    loader = st.LazyModuleLoader(root, view, quantized="weights")
    x = torch.randn(7, 320, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    with torch.no_grad():
        y = root.norm(x)
        w = sd[names["norm.weight"]]
        assert torch.equal(y, st.rms_norm(x, w, eps=1e-5))
        q = sd[names["q.weight"]]
        assert torch.equal(root.q(x), 2 * torch.nn.functional.linear(x, q)) and not root.q.weight.is_meta
        e = sd[names["embed.weight"]]
        assert torch.equal(root.embed(x), torch.nn.functional.linear(x, e))
    loader.detach()


def test_bound_counts_stored_bytes(tmp_path):
    sd = st.StreamStateDict(_file(tmp_path, 6), DEV)
    root = torch.nn.ModuleDict({"gate_proj": torch.nn.Linear(320, 960, bias=False, device="meta", dtype=torch.bfloat16),
                                "up_proj": torch.nn.Linear(320, 960, bias=False, device="meta", dtype=torch.bfloat16)})
    view = st.PrefixViewStateDict(sd, "model.layers.0.mlp.")
    one = 960 * 320 + 960 * 10
    loader = st.LazyModuleLoader(root, view, max_resident_bytes=one, quantized="weights")
    x = torch.randn(2, 320, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    a = [root[n](x) for n in ("gate_proj", "up_proj", "gate_proj")]
    assert torch.equal(a[0], a[2]) and not torch.equal(a[0], a[1])
    assert loader.resident_bytes == one and loader.stats["evicted"] == 2
    loader.detach()


def test_sharded_checkpoint(tmp_path):
    write_sharded(tmp_path, 3)
    sd = st.ShardedStateDict(str(tmp_path), DEV)
    root, lin = _module(3)
    loader = st.LazyModuleLoader(root, sd, quantized="weights")
    x = torch.randn(4, 960, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(DEV)
    name = LINEARS[3][0] + ".weight"
    assert torch.equal(lin(x), st.linear(x, sd.load_quantized([name], copy=True)[name]))
    loader.detach()


def test_refusals(tmp_path):
    sd = st.StreamStateDict(_file(tmp_path, 6), DEV)
    root, lin = _module(6)
    with pytest.raises(ValueError, match="quantized"):
        st.LazyModuleLoader(root, sd, quantized="fp8")
    loader = st.LazyModuleLoader(root, sd, quantized="weights")
    with pytest.raises(ValueError, match="bf16, fp16"):
        lin(torch.zeros(2, 320, device=DEV))
    with pytest.raises(RuntimeError, match="no backward"):
        lin(torch.zeros(2, 320, device=DEV, dtype=torch.bfloat16, requires_grad=True))
    loader.detach()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_norm_without_an_eps_of_its_own(dtype, tmp_path):
    """nn.RMSNorm's default eps against torch's norm, over rows from 1e-4 to 10."""
    sd = st.StreamStateDict(_file(tmp_path, 3), DEV)
    root = torch.nn.Module()
    root.norm = torch.nn.RMSNorm(320, device="meta", dtype=torch.bfloat16)
    loader = st.LazyModuleLoader(root, st.RenameViewStateDict(sd, {"model.layers.0.input_layernorm.weight": "norm.weight"}),
                                 strict=False, quantized="weights")
    g = torch.Generator().manual_seed(4)
    x = torch.cat([torch.randn(3, 320, generator=g) * 10.0 ** e for e in range(-4, 2)]).to(dtype)
    w = sd["model.layers.0.input_layernorm.weight"].cpu()
    want = torch.nn.functional.rms_norm(x.float(), (320,), w.float()).double()
    got = root.norm(x.to(DEV)).cpu().double()
    # one rounding to the rows' type, and the 32-bit form's own handful
    t = torch.finfo(dtype)
    assert ((got - want).abs() <= want.abs() * (t.eps / 2 + 16 * 2.0 ** -24) + t.smallest_normal * t.eps / 2).all()
    loader.detach()


def test_inputs_of_any_layout(tmp_path):
    """Transposed, strided, overlapping and broadcast rows through the modules, and through the operator where they are
    no matrix, for one image as for two."""
    sd = st.StreamStateDict(_file(tmp_path, 3), DEV)
    root, lin = _module(3)
    loader = st.LazyModuleLoader(root, sd, quantized="activations")
    g = torch.Generator().manual_seed(5)
    long = torch.randn(960 * 8, generator=g).to(torch.bfloat16).to(DEV)
    t = torch.randn(2, 960, 3, 4, generator=g).to(torch.bfloat16).to(DEV)
    for x in (t[0, :, 0].t(), long.unfold(0, 960, 8), long[::8], long[:960].expand(3, 960), t.flatten(2).transpose(1, 2),
              t[:1].flatten(2).transpose(1, 2)):
        assert torch.equal(lin(x), lin(x.contiguous()))
    w = sd.load_quantized([LINEARS[3][0] + ".weight"], copy=True)[LINEARS[3][0] + ".weight"]
    for x in (t.flatten(2).transpose(1, 2), t[:1].flatten(2).transpose(1, 2)):
        flat = x.contiguous()
        assert torch.equal(st.linear(x, w), st.linear(flat, w)) and torch.equal(st.rms_norm(x, residual=x)[0], st.rms_norm(flat, residual=flat)[0])
        q, p = st.quantize_activation(x, "MXFP8", gate=x), st.quantize_activation(flat, "MXFP8", gate=flat)
        assert torch.equal(q.data.view(torch.uint8), p.data.view(torch.uint8)) and torch.equal(q.scale.view(torch.uint8), p.scale.view(torch.uint8))
    loader.detach()


@pytest.mark.parametrize("k", [3, 6])
def test_a_captured_forward_replays(k, tmp_path):
    """A resident module's forward captured into a graph, replayed between eager work, new inputs and another module's loads."""
    sd = st.StreamStateDict(_file(tmp_path, k), DEV)
    root, lin = _module(k)
    loader = st.LazyModuleLoader(root, sd, quantized="activations")
    xs = [torch.randn(5, lin.in_features, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).to(DEV) for i in range(3)]
    want = [lin(x) for x in xs]
    x = xs[0].clone()
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lin(x)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lin(x)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i])
        assert torch.equal(lin(xs[2 - i]), want[2 - i])
    loader.detach()
    with pytest.raises(RuntimeError, match="not loaded"):
        lin(xs[0])
    loader.materialize(lin)
    assert torch.equal(lin(xs[0]), torch.nn.functional.linear(xs[0], sd[LINEARS[k][0] + ".weight"]))
