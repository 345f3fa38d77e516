"""CPU: what the operators on the 8-bit cache and on mixtures of experts refuse, before anything reaches a GPU, and the plain forms of
their tests against torch."""
import ctypes as C

import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from device_checkpoint_dequantisation_amd import _lib
from tests import kv_reference as kv
from tests import moe_reference as mref
from tests import ops_reference as ref

P = 0x10000     # a well-aligned address that is never followed
I32 = torch.int32


@pytest.fixture
def as_gpu(monkeypatch):
    """CPU tensors pass as GPU ones, and nothing is launched."""
    from device_checkpoint_dequantisation_amd import experts, kv_cache, ops
    check = ops._on_device
    gpu = type("Device", (), {"type": "cuda", "__eq__": lambda a, b: True, "__ne__": lambda a, b: False})()
    for m in (ops, kv_cache, experts):
        monkeypatch.setattr(m, "_on_device", lambda device, tensors, who: check(gpu, tensors, who))
        monkeypatch.setattr(m, "_launch", lambda *a: None)


def _cache(pages=4, heads=2, dim=64, block=16):
    return st.QuantizedKvCache.empty(pages, heads, dim, block, "cpu")


def _kv(tokens=3, heads=2, dim=64, dt=torch.bfloat16):
    return torch.zeros(tokens, heads, dim, dtype=dt)


def _t(seqs=3, blocks=2):
    return torch.zeros(seqs, blocks, dtype=I32), torch.ones(seqs, dtype=I32)


def test_they_need_a_gpu():
    t, n = _t()
    with pytest.raises(ValueError, match="GPU"):
        st.kv_append(_cache(), _kv(), _kv(), t, n)
    with pytest.raises(ValueError, match="GPU"):
        st.kv_attention(_kv(), _cache(), t, n)
    with pytest.raises(ValueError, match="GPU"):
        st.moe_route(torch.zeros(2, 8), torch.zeros(4, 8), 2)
    w = [ref.random_weight(st, "FP8_TENSOR", 32, 32, 1)]
    with pytest.raises(ValueError, match="GPU"):
        st.MoeExperts(w, w, w)


def test_cache_refusals(as_gpu):
    t, n = _t()
    k, v = _kv(), _kv()
    st.kv_append(_cache(), k, v, t, n)
    assert st.kv_attention(torch.zeros(3, 6, 64, dtype=torch.bfloat16), _cache(), t, n).shape == (3, 6, 64)

    def no(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)
    for f, a in ((st.kv_append, (k, v)), (st.kv_attention, (k,))):
        call = (lambda c=None, t=t, n=n, **kw: f(c or _cache(), *a, t, n, **kw)) if f is st.kv_append else (lambda c=None, t=t, n=n, **kw: f(*a, c or _cache(), t, n, **kw))
        no("QuantizedKvCache", call, c=3)
        for field, bad in (("k", torch.zeros(4, 2, 16, 64)), ("v", _cache().k), ("k_scale", torch.zeros(4, 2)), ("v_scale", _cache().k_scale.view(torch.uint8)),
                           ("k", _cache(block=24).k), ("k", _cache().k.transpose(0, 1).contiguous().transpose(0, 1))):
            c = _cache()
            setattr(c, field, bad)
            no("cache's|pages of", call, c=c)
        no("pages of 24", call, c=_cache(block=24))
        no("table", call, t=t.long())
        no("table", call, t=t[0])
        no("table", call, t=torch.zeros(2, 3, dtype=I32).t())
        no("lengths", call, n=n.long())
        no("lengths", call, n=n[:2])
        no("equal parts", call, t=t[:2], n=n[:2])
        no("equal parts", call, t=t[:0], n=n[:0])
        no("max_new goes", call, max_new=3)
        no("starts", call, starts=torch.zeros(3, dtype=I32))
        no("starts", call, starts=torch.zeros(4))
        no("max_new", call, starts=torch.zeros(4, dtype=I32), max_new=-1)
        no("max_new", call, starts=torch.zeros(4, dtype=I32), max_new=2.0)
    no("head_dim", st.kv_append, _cache(dim=48), _kv(dim=48), _kv(dim=48), t, n)
    no("k is", st.kv_append, _cache(), _kv(heads=3), v, t, n)
    no("v is", st.kv_append, _cache(), k, _kv(dim=32), t, n)
    no("one shape", st.kv_append, _cache(), k, v.half(), t, n)
    no("one shape", st.kv_append, _cache(), k.double(), v.double(), t, n)
    no("one shape", st.kv_append, _cache(), k, _kv(tokens=6), t, n)
    no("contiguous", st.kv_append, _cache(), torch.zeros(3, 64, 2, dtype=torch.bfloat16).transpose(1, 2), v, t, n)
    c = _cache()
    inside = c.k.view(torch.uint8).view(torch.bfloat16).view(-1)[:384].view(3, 2, 64)
    no("overlaps", st.kv_append, c, inside, v, t, n)
    no("head_dim 96", st.kv_attention, _kv(dim=96), _cache(dim=96), t, n)
    no("q is", st.kv_attention, k.float(), _cache(), t, n)
    no("q is", st.kv_attention, k[0], _cache(), t, n)
    no("query heads", st.kv_attention, _kv(heads=3), _cache(), t, n)
    for s in (0.0, -1.0, float("nan"), float("inf")):
        no("scale", st.kv_attention, k, _cache(), t, n, scale=s)
    for w in (0, -3, 2.5):
        no("window", st.kv_attention, k, _cache(), t, n, window=w)
    no("window", st.kv_attention, k, _cache(), t, n, window=4, causal=False)
    no("out", st.kv_attention, k, _cache(), t, n, out=k.half())
    no("strides", st.kv_attention, k, _cache(), t, n, out=torch.zeros(1, 2, 64, dtype=torch.bfloat16).expand(3, 2, 64))
    no("overlaps", st.kv_attention, k, _cache(), t, n, out=k)
    no("cache of 0 pages", st.kv_attention, k, _cache(pages=0), t, n)
    no("table of 0", st.kv_attention, k, _cache(), t[:, :0], n)
    with pytest.raises(RuntimeError, match="no backward"):
        st.kv_attention(k.clone().requires_grad_(), _cache(), t, n)
    # nothing to do
    st.kv_append(_cache(), k[:0], v[:0], t, n)
    st.kv_append(_cache(pages=0), k, v, t, n)
    assert st.kv_attention(k[:0], _cache(), t, n).shape == (0, 2, 64)
    s = torch.zeros(4, dtype=I32)
    assert (st.kv_attention(k, _cache(), t, n, starts=s, max_new=0) == 0).all()


def test_moe_refusals(as_gpu):
    def lists(**kw):
        out = []
        for n, k, kind in ((32, 64, kw.get("up", "FP8_TENSOR")), (32, 64, kw.get("up", "FP8_TENSOR")), (kw.get("n", 16), 32, kw.get("down", "FP8_TENSOR"))):
            out.append([ref.random_weight(st, kind, n, k, e) for e in range(3)])
        return out

    def no(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)
    ex = st.MoeExperts(*lists())
    assert len(ex) == 3 and ex.shape == (32, 64) and ex.width == 16 and ex.table.shape == (9, 3)
    assert st.MoeExperts(*lists(up="MXFP4", down="NVFP4")).down_kind == "NVFP4"
    g, u, d = lists()
    no("one of each", st.MoeExperts, g, u[:2], d)
    no("one of each", st.MoeExperts, [], [], [])
    no("expert 1's up", st.MoeExperts, g, [u[0], ref.random_weight(st, "FP8_TENSOR", 32, 32, 1), u[2]], d)
    no("expert 2's gate", st.MoeExperts, g[:2] + [ref.random_weight(st, "MXFP8", 32, 64, 1)], u, d)
    no("expert 0's down", st.MoeExperts, g, u, [ref.random_weight(st, "FP8_TENSOR", 16, 64, 1)] * 3)
    g[1].data = g[1].data.view(torch.uint8)
    no("holds", st.MoeExperts, g, u, d)
    x, ids, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=I32), torch.zeros(2, 2)
    assert st.moe(x, ex, ids, w).shape == (2, 16) and st.moe(x[:0], ex, ids[:0], w[:0]).shape == (0, 16)
    no("MoeExperts", st.moe, x, lists(), ids, w)
    no("x is", st.moe, x.float(), ex, ids, w)
    no("x is", st.moe, x[:, :32], ex, ids, w)
    no("ids", st.moe, x, ex, ids.long(), w)
    no("ids", st.moe, x, ex, ids[:1], w)
    no("ids", st.moe, x, ex, ids.t().contiguous().t(), w)
    no("experts a row", st.moe, x, ex, torch.zeros(2, 33, dtype=I32), torch.zeros(2, 33))
    no("experts a row", st.moe, x, ex, ids[:, :0].contiguous(), w[:, :0].contiguous())
    no("weights", st.moe, x, ex, ids, w.half())
    no("weights", st.moe, x, ex, ids, w[:, :1])
    no("activation", st.moe, x, ex, ids, w, activation="swish")
    no("residual", st.moe, x, ex, ids, w, residual=x)
    no("out_dtype", st.moe, x, ex, ids, w, out_dtype="f64")
    no("out ", st.moe, x, ex, ids, w, out=torch.zeros(2, 15))
    no("out is", st.moe, x, ex, ids, w, out=torch.zeros(2, 16), out_dtype="bf16")
    no("strides", st.moe, x, ex, ids, w, out=torch.zeros(1, 16).expand(2, 16))
    no("overlaps", st.moe, x, ex, ids, w, out=x[:, :16])
    r = torch.zeros(4, 64)
    no("x is", st.moe_route, x.double(), r, 2)
    no("router", st.moe_route, x, r[:, :32], 2)
    no("router", st.moe_route, x, torch.zeros(64, 4).t(), 2)
    no("router", st.moe_route, x, r[0], 2)
    for k in (0, 5, 1.0):
        no("of 4 experts", st.moe_route, x, r, k)
    no("at most 1024", st.moe_route, x, torch.zeros(1025, 64), 2)
    no("score", st.moe_route, x, r, 2, score="tanh")
    no("bias", st.moe_route, x, r, 2, bias=torch.zeros(4).half())
    no("bias", st.moe_route, x, r, 2, bias=torch.zeros(3))
    assert [t.shape for t in st.moe_route(x, r, 2)] == [(2, 2), (2, 2)]


def _args(cls, **base):
    return lambda **kw: cls(**{**base, **kw})


_append = _args(_lib.KvAppendArgs, k_new=P, v_new=P, k=P, v=P, k_scale=P, v_scale=P, table=P, lengths=P, starts=None, pages=9, tokens=4, seqs=2,
                max_new=2, table_blocks=3, table_pitch=3, k_pitch=128, k_head_pitch=64, v_pitch=128, v_head_pitch=64, heads=2,
                head_dim=64, block=16, x_type=0)
_attention = _args(_lib.KvAttentionArgs, q=P, out=P, k=P, v=P, k_scale=P, v_scale=P, table=P, lengths=P, starts=None, workspace=None,
                   workspace_bytes=0, pages=9, tokens=4, seqs=2, max_new=2, table_blocks=3, table_pitch=3, q_pitch=256, q_head_pitch=64,
                   out_pitch=256, out_head_pitch=64, window=0, scale=0.1, heads=2, group=2, head_dim=64, block=16, causal=1, q_type=0)
_route = _args(_lib.MoeRouteArgs, x=P, router=P, bias=None, weights=P, ids=P, workspace=P, workspace_bytes=1 << 20, t=4, k=64, x_pitch=64,
               router_pitch=64, scaling=1.0, experts=8, top=2, score=0, renormalize=1, x_type=0, router_type=2)
_moe = _args(_lib.MoeArgs, x=P, ids=P, weights=P, experts_dev=P, residual=None, out=P, workspace=P, workspace_bytes=1 << 20, t=4, k=64, i=32,
             n=64, x_pitch=64, residual_pitch=0, out_pitch=64, experts=8, top=2, x_type=0, up_kind=3, down_kind=3, activation=2, residual_type=0,
             out_type=0)


@pytest.mark.parametrize("kw,code", [(dict(x_type=3), -1), (dict(head_dim=0), -6), (dict(head_dim=48), -6), (dict(head_dim=288), -6), (dict(block=8), -6),
                                     (dict(block=48), -6), (dict(tokens=1 << 31), -6), (dict(seqs=65536), -6), (dict(heads=65536), -6),
                                     (dict(pages=1 << 31), -6), (dict(table_blocks=1 << 27), -6), (dict(tokens=5), -6), (dict(k_new=None), -1),
                                     (dict(v_scale=None), -1), (dict(table=None), -1), (dict(k_new=P + 1), -1), (dict(v=P + 8), -1),
                                     (dict(lengths=P + 2), -1), (dict(starts=P + 2), -1), (dict(table_pitch=2), -6),
                                     (dict(tokens=1 << 30, max_new=1 << 30, starts=P), -6)])
def test_append_abi_refusals(kw, code):
    assert _lib.lib().st_kv_append(C.byref(_append(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [(dict(q_type=2), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(causal=2), -1),
                                     (dict(causal=0, window=3), -1), (dict(head_dim=96), -6), (dict(block=256), -6), (dict(seqs=65536), -6),
                                     (dict(group=65536), -6), (dict(table_blocks=1 << 27), -6), (dict(tokens=5), -6), (dict(pages=0), -6),
                                     (dict(table_blocks=0), -6), (dict(q=None), -1), (dict(k_scale=None), -1), (dict(q=P + 1), -1),
                                     (dict(k=P + 4), -1), (dict(table=P + 1), -1), (dict(table_pitch=1), -6),
                                     (dict(tokens=1 << 30, seqs=1, max_new=1 << 30), -6), (dict(tokens=1 << 26, seqs=1, max_new=1 << 26, heads=64), -6)])
def test_attention_abi_refusals(kw, code):
    L, a, need = _lib.lib(), _attention(**kw), C.c_uint64(7)
    assert L.st_kv_attention(C.byref(a), None) == code
    assert L.st_kv_attention_workspace_bytes(C.byref(a), C.byref(need)) == code and need.value == 0


@pytest.mark.parametrize("kw,code", [(dict(x_type=3), -1), (dict(router_type=3), -1), (dict(score=2), -1), (dict(renormalize=2), -1), (dict(experts=0), -6),
                                     (dict(experts=1025), -6), (dict(top=0), -6), (dict(top=9), -6), (dict(t=1 << 17), -6), (dict(k=1 << 31), -6),
                                     (dict(weights=None), -1), (dict(x=None), -1), (dict(x_pitch=63), -6), (dict(router_pitch=63), -6),
                                     (dict(x=P + 1), -1), (dict(router=P + 2), -1), (dict(bias=P + 2), -1), (dict(workspace=None), -1),
                                     (dict(workspace_bytes=8), -1), (dict(workspace=P + 8), -1)])
def test_route_abi_refusals(kw, code):
    assert _lib.lib().st_moe_route(C.byref(_route(**kw)), None) == code


@pytest.mark.parametrize("kw,code", [(dict(x_type=2), -1), (dict(activation=5), -1), (dict(out_type=3), -1), (dict(residual_type=3), -1), (dict(up_kind=2), -1),
                                     (dict(down_kind=8), -1), (dict(up_kind=5, k=72, x_pitch=72), -6), (dict(down_kind=7, i=40), -6), (dict(k=1 << 31), -6),
                                     (dict(experts=16385), -6), (dict(top=33), -6), (dict(t=1 << 23), -6), (dict(k=0), -6), (dict(i=0), -6),
                                     (dict(experts=0), -6), (dict(top=0), -6), (dict(x=None), -1), (dict(ids=None), -1), (dict(experts_dev=None), -1),
                                     (dict(x_pitch=63), -6), (dict(out_pitch=63), -6), (dict(residual=P, residual_pitch=63), -6), (dict(x=P + 1), -1),
                                     (dict(experts_dev=P + 4), -1), (dict(out=P + 1), -1), (dict(workspace=None), -1), (dict(workspace_bytes=64), -1),
                                     (dict(workspace=P + 8), -1), (dict(n=(1 << 31) - 1, out_pitch=1 << 31), -6)])
def test_moe_abi_refusals(kw, code):
    assert _lib.lib().st_moe(C.byref(_moe(**kw)), None) == code


def test_abi_null_and_empty():
    L, need = _lib.lib(), C.c_uint64(7)
    for f in (L.st_kv_append, L.st_kv_attention, L.st_moe_route, L.st_moe):
        assert f(None, None) == -1
    for f, a in ((L.st_kv_attention_workspace_bytes, _attention()), (L.st_moe_route_workspace_bytes, _route()), (L.st_moe_workspace_bytes, _moe())):
        assert f(C.byref(a), None) == -1 and f(None, C.byref(need)) == -1 and need.value == 0
    for f, a in ((L.st_kv_append, _append(tokens=0, k_new=None)), (L.st_kv_append, _append(pages=0)), (L.st_kv_append, _append(max_new=0, starts=P)),
                 (L.st_kv_attention, _attention(tokens=0, q=None)), (L.st_kv_attention, _attention(group=0)), (L.st_kv_attention, _attention(max_new=0, starts=P)),
                 (L.st_moe_route, _route(t=0, x=None, workspace=None)), (L.st_moe, _moe(t=0, x=None, workspace=None)), (L.st_moe, _moe(n=0, out=None))):
        assert f(C.byref(a), None) == 0
    # parts of a long context pass through memory
    a = _attention(table_blocks=1 << 13, table_pitch=1 << 13)
    assert L.st_kv_attention_workspace_bytes(C.byref(a), C.byref(need)) == 0 and need.value
    assert L.st_kv_attention(C.byref(a), None) == -1
    a.workspace, a.workspace_bytes = P, need.value - 1
    assert L.st_kv_attention(C.byref(a), None) == -1
    a.workspace, a.workspace_bytes = P + 8, need.value
    assert L.st_kv_attention(C.byref(a), None) == -1


def test_attention_refuses_more_results_than_sizes_hold():
    """Rows without end (a pitch of 0 takes no memory) must not make the workspace's size wrap around."""
    a, need = _attention(tokens=(1 << 31) - 2, max_new=1, seqs=2, heads=64, group=65535, starts=P, q_pitch=0, out_pitch=0,
                         table_blocks=1 << 20, table_pitch=1 << 20), C.c_uint64(7)
    assert _lib.lib().st_kv_attention_workspace_bytes(C.byref(a), C.byref(need)) == -6 and need.value == 0
    assert _lib.lib().st_kv_attention(C.byref(a), None) == -6


def test_moe_out_among_the_weights(as_gpu):
    """Experts that are views of one buffer: every place for out that touches one of them is refused, those between are not."""
    buf, at, lists = torch.zeros(1 << 16, dtype=torch.uint8), 512, ([], [], [])
    used = torch.zeros(1 << 16, dtype=torch.bool)
    for e in range(5):
        for which, shape in enumerate(((32, 64), (32, 64), (16, 32))):
            w = ref.random_weight(st, "FP8_TENSOR", *shape, 1)
            n = shape[0] * shape[1]
            w.data = buf[at:at + n].view(torch.float8_e4m3fn).view(shape)
            used[at:at + n] = True
            at += n + 64 * ((3 * e + which) % 4)
            lists[which].append(w)
    ex = st.MoeExperts(*lists)
    x, ids, weights = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=I32), torch.zeros(2, 2)
    refused = 0
    for o in range(0, at + 512, 64):
        out = buf[o:o + 64].view(torch.bfloat16).view(2, 16)
        if used[o:o + 64].any():
            refused += 1
            with pytest.raises(ValueError, match="overlaps"):
                st.moe(x, ex, ids, weights, out=out)
        else:
            st.moe(x, ex, ids, weights, out=out)
    assert refused == 5 * (2048 + 2048 + 512) // 64


def test_reference_append_matches_torch():
    """Scales and codes of whole pages against torch's own conversion."""
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn(2, 32, 2, 64, generator=g) * torch.exp(2 * torch.randn(2, 32, 2, 1, generator=g))
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    kc, vc, ks, vs = kv.append(kv.random_cache(st, 2, 2, 64, 16, 2), k, v, [[1, 0]], [32])
    for x, c, e in ((k, kc, ks), (v, vc.transpose(2, 3), vs)):
        for b, page in ((0, 1), (1, 0)):
            rows = x[16 * b:16 * b + 16].transpose(0, 1).float()
            s = torch.exp2(torch.ceil(torch.log2(rows.abs().amax((1, 2)) / 448)))
            assert torch.equal(torch.exp2(e[page].float()), s)
            assert torch.equal(c[page].float(), (rows / s[:, None, None]).to(torch.float8_e4m3fn).float())


def test_reference_attention_matches_torch():
    g = torch.Generator().manual_seed(3)
    cache = kv.random_cache(st, 5, 2, 64, 16, 4)
    q = torch.randn(6, 4, 64, generator=g)
    table, n = [[3, 1, 0]], 37
    got, _ = kv.attention(q, cache, table, [n])
    for h in range(4):
        k, v = (ref.e4m3(c)[[3, 1, 0]][:, h // 2] * ref.e8m0(s)[[3, 1, 0]][:, h // 2, None, None] for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        k, v = k.reshape(-1, 64)[:n], v.transpose(1, 2).reshape(-1, 64)[:n]
        mask = torch.ones(6, n, dtype=torch.bool).tril(n - 6)
        want = torch.nn.functional.scaled_dot_product_attention(q[None, :, h].double(), k[None], v[None], attn_mask=mask)[0]
        assert (got[:, h] - want).abs().max() < 1e-12 * want.abs().max()


def test_reference_moe_matches_loops():
    lists = mref.random_experts(st, "MXFP8", "NVFP4", 3, 32, 64, 16, 5)
    x = torch.randn(4, 64, generator=torch.Generator().manual_seed(6))
    ids = torch.tensor([[0, 2], [1, 1], [2, -1], [9, 0]], dtype=I32)
    w = torch.rand(4, 2, generator=torch.Generator().manual_seed(7))
    got, _ = mref.moe(x, lists, ids, w)
    for t in range(4):
        y = torch.zeros(16, dtype=torch.float64)
        for j in range(2):
            e = int(ids[t, j])
            if 0 <= e < 3:
                a, b, d = (ref.weight_value(ws[e]) for ws in lists)
                y += w[t, j].double() * (d @ (torch.nn.functional.silu(a @ x[t].double()) * (b @ x[t].double())))
        assert (got[t] - y).abs().max() <= 1e-12 * y.abs().max() + 1e-12
