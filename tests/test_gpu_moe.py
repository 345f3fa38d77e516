"""GPU: the router and the experts of a mixture against 64-bit forms: every weight kind, from one row to hundreds, ragged sizes and odd rows,
experts that nobody, everybody or one row twice has, ids that are none, ties and NaN; graphs, streams; a decoding step of all operators."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import kv_reference as kv
from tests import moe_reference as mref
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KINDS = ("FP8_TENSOR", "FP8_BLOCK128", "NVFP4", "MXFP8", "MXFP4")


def _gpu(lists):
    return st.MoeExperts(*([ref.to(w, DEV) for w in ws] for ws in lists))


def _ids(m, top, experts, seed):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(m, experts, generator=g) + torch.linspace(2, 0, experts)
    w, ids = torch.softmax(z, 1).topk(top, 1)
    return ids.to(torch.int32), w.contiguous()


def _rows(m, k, dt, seed):
    return torch.randn(m, k, generator=torch.Generator().manual_seed(seed)).to(ref.DT[dt])


def _check(x, lists, experts, ids, w, **kw):
    got = st.moe(x.to(DEV), experts, ids.to(DEV), w.to(DEV), **{a: b.to(DEV) if torch.is_tensor(b) else b for a, b in kw.items()})
    kw.pop("out_dtype", None)
    want, tol = mref.moe(x, lists, ids, w, **kw)
    mref.check(got, want, tol)
    return got


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("experts,top,i,k,n", [(4, 2, 96, 160, 96), (9, 3, 320, 1280, 200), (2, 1, 32, 64, 1), (6, 6, 160, 576, 130)])
def test_experts(dt, kind, experts, top, i, k, n):
    lists = mref.random_experts(st, kind, kind, experts, i, k, n, 1)
    ex = _gpu(lists)
    for m in (1, 2, 7, 16, 17, 40, 150):
        print(f"moe {dt} {kind} {experts} {top} {i} {k} {n} rows {m}", flush=True)
        x = _rows(m, k, dt, m)
        ids, w = _ids(m, top, experts, m)
        _check(x, lists, ex, ids, w, out_dtype="f32")
        r = _rows(m, n, "f32", m + 1)
        _check(x, lists, ex, ids, w, residual=r.to(ref.DT[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("kind", ["FP8_TENSOR", "FP8_BLOCK128"])
@pytest.mark.parametrize("i,k,n", [(1, 1, 1), (33, 131, 70), (131, 257, 5), (259, 1001, 129), (16, 15, 3)])
def test_odd_sizes(dt, kind, i, k, n):
    lists = mref.random_experts(st, kind, kind, 5, i, k, n, 3)
    ex = _gpu(lists)
    for m in (1, 5, 16, 30, 90):
        print(f"moe odd {dt} {kind} {i} {k} {n} rows {m}", flush=True)
        ids, w = _ids(m, 2, 5, m)
        _check(_rows(m, k, dt, m), lists, ex, ids, w, out_dtype="f32")


@pytest.mark.parametrize("kind,down", [("NVFP4", "FP8_BLOCK128"), ("MXFP4", "MXFP8"), ("FP8_TENSOR", "NVFP4")])
@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
def test_mixed_kinds_and_activations(kind, down, act):
    lists = mref.random_experts(st, kind, down, 4, 160, 288, 72, 5)
    ex = _gpu(lists)
    for m in (3, 33):
        ids, w = _ids(m, 2, 4, m)
        _check(_rows(m, 288, "bf16", m), lists, ex, ids, w, activation=act, out_dtype="f32")


@pytest.mark.parametrize("kind", ["FP8_BLOCK128", "MXFP4"])
def test_who_has_whom(kind):
    """All rows at one expert (several tiles), an expert twice in a row, ids that are none, experts that nobody has."""
    lists = mref.random_experts(st, kind, kind, 7, 96, 128, 64, 7)
    ex = _gpu(lists)
    g = torch.Generator().manual_seed(8)
    for m, top in ((1, 8), (4, 3), (16, 32), (20, 8), (200, 3), (700, 2)):
        print(f"moe ids {kind} {m} {top}", flush=True)
        x, w = _rows(m, 128, "bf16", m), torch.rand(m, top, generator=g)
        every = torch.randint(-2, 9, (m, top), generator=g, dtype=torch.int32)
        one = torch.full((m, top), 4, dtype=torch.int32)
        none = torch.full((m, top), -1, dtype=torch.int32)
        none[0, 0], none[0, top - 1] = 2 ** 31 - 1, -2 ** 31
        few = torch.where(torch.rand(m, top, generator=g) < 0.9, torch.full((m, top), 5, dtype=torch.int32), every)
        for ids in (every, one, none, few):
            _check(x, lists, ex, ids.contiguous(), w, out_dtype="f32")
        got = st.moe(x.to(DEV), ex, none.to(DEV), w.to(DEV))
        assert (got == 0).all()


def test_many_pairs():
    """More ids than one turn of the search reads, and expert rows in several tiles that start anywhere."""
    lists = mref.random_experts(st, "FP8_TENSOR", "FP8_TENSOR", 3, 32, 64, 48, 9)
    ex = _gpu(lists)
    for m, top in ((4099, 2), (1367, 7)):
        ids = torch.randint(-1, 3, (m, top), generator=torch.Generator().manual_seed(m), dtype=torch.int32)
        ids[:, 1:][:1000] = -1
        w = torch.rand(m, top, generator=torch.Generator().manual_seed(m + 1))
        print(f"moe pairs {m} {top}", flush=True)
        _check(_rows(m, 64, "bf16", m), lists, ex, ids, w, out_dtype="f32")


def test_many_experts_few_rows():
    """Fewer pairs than experts: workgroups go by pair; as many tiles with 17 rows and more."""
    lists = mref.random_experts(st, "MXFP8", "MXFP8", 70, 32, 64, 40, 10)
    ex = _gpu(lists)
    for m, top in ((1, 8), (8, 8), (20, 3), (30, 2)):
        ids = torch.randint(0, 70, (m, top), generator=torch.Generator().manual_seed(m), dtype=torch.int32)
        ids[-1, 0] = ids[0, 0]
        _check(_rows(m, 64, "f16", m), lists, ex, ids, torch.rand(m, top, generator=torch.Generator().manual_seed(1)), out_dtype="f32")


@pytest.mark.parametrize("kind", KINDS)
def test_pairs_of_one_wavefront(kind):
    """Up to 16 tokens and 64 pairs, all of them used, with experts that a token has many times."""
    lists = mref.random_experts(st, kind, kind, 6, 96, 288, 72, 12)
    ex = _gpu(lists)
    for m, top in ((2, 32), (16, 4), (9, 7), (3, 21), (16, 1)):
        print(f"moe one wavefront {kind} {m} {top}", flush=True)
        g = torch.Generator().manual_seed(100 * m + top)
        w = torch.rand(m, top, generator=g)
        for ids in (torch.randint(-1, 7, (m, top), generator=g, dtype=torch.int32), torch.full((m, top), 3, dtype=torch.int32),
                    torch.arange(m * top, dtype=torch.int32).view(m, top) % 6):
            _check(_rows(m, 288, "bf16", m), lists, ex, ids.contiguous(), w, out_dtype="f32")


@pytest.mark.parametrize("kind,dt", [("FP8_BLOCK128", "bf16"), ("NVFP4", "f16"), ("MXFP8", "f16")])
def test_few_pairs_on_average(kind, dt):
    """Many experts, most of whose pairs are one's: it has them in many turns of 16."""
    lists = mref.random_experts(st, kind, kind, 40, 64, 288, 40, 13)
    ex = _gpu(lists)
    for m, top in ((30, 4), (17, 8), (70, 3)):
        print(f"moe one busy {kind} {m} {top}", flush=True)
        ids = torch.full((m, top), 31, dtype=torch.int32)
        ids[1::3, 0] = torch.arange(len(ids[1::3]), dtype=torch.int32) % 40
        _check(_rows(m, 288, dt, m), lists, ex, ids, torch.rand(m, top, generator=torch.Generator().manual_seed(m)), out_dtype="f32")


def test_nan_stays_with_its_rows():
    """NaN and infinities in one row, in one expert's weights, in a weight of a slot: nobody else's result changes."""
    for m in (8, 60):
        lists = mref.random_experts(st, "FP8_TENSOR", "FP8_TENSOR", 4, 64, 96, 32, 11)
        x = _rows(m, 96, "bf16", 12)
        ids, w = _ids(m, 2, 3, 13)               # expert 3 is nobody's
        ex = _gpu(lists)
        clean = st.moe(x.to(DEV), ex, ids.to(DEV), w.to(DEV))
        for ws in lists:
            ws[3].data.view(torch.uint8).fill_(0x7F)
            ws[1].data.view(torch.uint8)[0] = 0x7F
        x[2, 5] = float("inf")
        w[4, 0] = float("nan")
        got = st.moe(x.to(DEV), _gpu(lists), ids.to(DEV), w.to(DEV))
        hit = (ids == 1).any(1)
        hit[2] = hit[4] = True
        hit = hit.to(DEV)
        assert torch.equal(got[~hit], clean[~hit])
        assert got[2].isnan().any() and got[4].isnan().all()


def test_views_at_any_byte_strides_and_out():
    """Weights as views into a blob at odd bytes, rows and residuals in wide buffers, out in place of the residual."""
    lists = mref.random_experts(st, "MXFP4", "FP8_TENSOR", 3, 64, 96, 36, 14)

    def odd(t):
        raw = t.contiguous().reshape(-1).view(torch.uint8).to(DEV)
        step = 4 if t.dtype == torch.float32 else 1
        b = torch.zeros(raw.numel() + step, dtype=torch.uint8, device=DEV)
        b[step:] = raw
        return b[step:].view(t.dtype).view(t.shape)
    for ws in lists:
        for w in ws:
            w.odd = type(w)(w.name, w.kind, w.shape, odd(w.data), odd(w.scale))
    ex = st.MoeExperts(*([w.odd for w in ws] for ws in lists))
    for m in (5, 50):
        wide = _rows(m, 96 + 7, "bf16", 15)
        ids, w = _ids(m, 2, 3, 16)
        res = _rows(m, 36 + 3, "f32", 17).to(DEV)
        want, tol = mref.moe(wide[:, 3:99], lists, ids, w, residual=res[:, 1:37].cpu())
        other = res.clone()
        got = st.moe(wide.to(DEV)[:, 3:99], ex, ids.to(DEV), w.to(DEV), residual=res[:, 1:37], out=res[:, 1:37])
        mref.check(got, want, tol)
        assert torch.equal(res[:, :1], other[:, :1]) and torch.equal(res[:, 37:], other[:, 37:])
        x3 = _rows(m * 2, 96, "bf16", 18).view(m, 2, 96)
        ids, w = _ids(m * 2, 2, 3, 19)
        got = st.moe(x3.to(DEV), ex, ids.view(m, 2, 2).to(DEV), w.view(m, 2, 2).to(DEV))
        want, tol = mref.moe(x3.view(-1, 96), lists, ids, w)
        assert got.shape == (m, 2, 36)
        mref.check(got.view(-1, 36), want, tol)


@pytest.mark.parametrize("xt,rt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("experts,top,k", [(1, 1, 8), (4, 4, 64), (65, 6, 131), (128, 8, 4096), (300, 20, 520), (1024, 32, 96)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(xt, rt, experts, top, k, score):
    g = torch.Generator().manual_seed(experts + k)
    router = (torch.randn(experts, k, generator=g) / k ** 0.5).to(ref.DT[rt])
    bias = 0.1 * torch.randn(experts, generator=g)
    for m in (1, 3, 70):
        x = _rows(m, k, xt, m)
        for b in (None, bias):
            for renormalize, scaling in ((True, 1.0), (False, 2.5)):
                print(f"route {xt} {rt} {experts} {top} {k} {score} rows {m}", flush=True)
                w, ids = st.moe_route(x.to(DEV), router.to(DEV), top, score=score, bias=None if b is None else b.to(DEV),
                                      renormalize=renormalize, scaling=scaling)
                want, wids = mref.route(x, router, top, score, b, renormalize, scaling)
                assert torch.equal(ids.cpu(), wids)
                # fp64 throughout, rounded once
                assert ((w.cpu().double() - want).abs() <= want.abs() * (2.0 ** -24 + 2.0 ** -40)).all()


@pytest.mark.parametrize("experts,top,k", [(2, 1, 33), (5, 3, 306), (9, 4, 480), (23, 8, 1412), (61, 6, 317), (127, 7, 100), (513, 5, 64)])
def test_route_any_number_of_experts(experts, top, k):
    """Wavefronts and workgroups that the experts do not fill, for scores that are far apart."""
    g = torch.Generator().manual_seed(experts)
    router, bias = torch.randn(experts, k, generator=g) * 3 / k ** 0.5, 0.1 * torch.randn(experts, generator=g)
    for m in (1, 17, 300):
        x = _rows(m, k, "bf16", m)
        for score in ("softmax", "sigmoid"):
            for b in (None, bias):
                for renormalize in (True, False):
                    print(f"route {experts} {top} {k} {score} rows {m}", flush=True)
                    w, ids = st.moe_route(x.to(DEV), router.to(DEV), top, score=score, bias=None if b is None else b.to(DEV), renormalize=renormalize)
                    want, wids = mref.route(x, router, top, score, b, renormalize)
                    assert torch.equal(ids.cpu(), wids)
                    assert ((w.cpu().double() - want).abs() <= want.abs() * (2.0 ** -24 + 2.0 ** -40)).all()


def test_route_ties_and_nan():
    """Equal scores by their number, NaN last, whatever the sums' order."""
    router = torch.zeros(12, 64)
    router[3:7, 0] = 1.0
    router[9, 1] = float("nan")
    x = torch.zeros(3, 64)
    x[0, 0], x[1, 0] = 2.0, -2.0
    for dt in ("f32", "bf16"):
        for score in ("softmax", "sigmoid"):
            w, ids = st.moe_route(x.to(ref.DT[dt]).to(DEV), router.to(ref.DT[dt]).to(DEV), 12, score=score)
            assert ids.tolist() == [[3, 4, 5, 6, 0, 1, 2, 7, 8, 10, 11, 9], [0, 1, 2, 7, 8, 10, 11, 3, 4, 5, 6, 9],
                                    [0, 1, 2, 3, 4, 5, 6, 7, 8, 10, 11, 9]]
            assert w.isnan().all()                    # the sum they are divided by
    w, ids = st.moe_route(x.to(DEV), router.to(DEV), 11, score="sigmoid", renormalize=False)
    assert not w.isnan().any() and (w[0, :4].cpu() - torch.sigmoid(torch.tensor(2.0))).abs().max() < 1e-7


def test_route_strides():
    wide, r = _rows(9, 100, "bf16", 20), _rows(8, 90, "f32", 21)
    got = st.moe_route(wide.to(DEV)[:, 3:80], r.to(DEV)[:, 5:82], 3)
    want = mref.route(wide[:, 3:80], r[:, 5:82], 3)
    assert torch.equal(got[1].cpu(), want[1])
    got = st.moe_route(wide.to(DEV)[:, 3:80].reshape(3, 3, 77), r.to(DEV)[:, 5:82], 3)
    assert got[0].shape == got[1].shape == (3, 3, 3) and torch.equal(got[1].cpu().view(9, 3), want[1])
    w, ids = st.moe_route(torch.zeros(0, 77, device=DEV), r.to(DEV)[:, 5:82], 3)
    assert w.shape == ids.shape == (0, 3)


def test_graph_and_streams():
    """Router and experts captured once, replayed on other rows with eager work between; then on a side stream."""
    lists = mref.random_experts(st, "NVFP4", "NVFP4", 8, 128, 256, 256, 22)
    ex = _gpu(lists)
    router = _rows(8, 256, "bf16", 23).to(DEV) * 0.1
    for m in (4, 40):
        x = torch.zeros(m, 256, dtype=torch.bfloat16, device=DEV)
        out = torch.empty_like(x)

        def layer():
            w, ids = st.moe_route(x, router, 2)
            st.moe(x, ex, ids, w, residual=x, out=out)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer()
        for i in range(4):
            x.copy_(_rows(m, 256, "bf16", 30 + i))
            g.replay()
            torch.cuda.synchronize()
            w, ids = st.moe_route(x, router, 2)
            eager = st.moe(x, ex, ids, w, residual=x)
            assert torch.equal(out, eager)
            want, tol = mref.moe(x.cpu(), lists, ids.cpu(), w.cpu(), residual=x.cpu())
            mref.check(out, want, tol)
        w2, ids2 = st.moe_route(x, router, 2, stream=side)
        got = None
        with torch.cuda.stream(side):
            got = st.moe(x, ex, ids2, w2, residual=x)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, out) and torch.equal(ids2, ids)
        got = st.moe(x, ex, ids, w, residual=x, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, out)


def test_refusals():
    lists = mref.random_experts(st, "FP8_TENSOR", "FP8_TENSOR", 3, 64, 96, 32, 11)
    ex = _gpu(lists)
    x = torch.zeros(4, 96, dtype=torch.bfloat16, device=DEV)
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    with pytest.raises(ValueError, match="tensors on"):
        st.moe(x, ex, ids.cpu(), w)
    with pytest.raises(RuntimeError, match="no backward"):
        st.moe(x, ex, ids, w.clone().requires_grad_())
    buf = torch.zeros(4, 96, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        st.moe(buf.view(torch.bfloat16)[:, :96], ex, ids, w, out=buf[:, :32])
    with pytest.raises(ValueError, match="overlaps"):
        st.moe(x, ex, ids, w, out=ex.weights[1][0].data.view(torch.uint8).view(-1)[:512].view(torch.float32).view(4, 32))


def test_a_decoding_step():
    """One layer of a small model for a batch of sequences: norm, projections, cache, attention, norm, router, experts, all on quantised
    weights, against the same in 64 bits."""
    hidden, heads, group, dim, seqs, block = 256, 2, 2, 64, 5, 16
    wide = (group + 2) * heads * dim
    qkv, proj = ref.random_weight(st, "FP8_BLOCK128", wide, hidden, 40), ref.random_weight(st, "MXFP4", hidden, group * heads * dim, 41)
    lists = mref.random_experts(st, "NVFP4", "FP8_BLOCK128", 8, 128, hidden, hidden, 42)
    for w in [qkv, proj]:                 # results of ordinary size
        w.scale = (w.scale * 1e-1) if w.kind.startswith("FP8") else (w.scale.view(torch.uint8) - 9).view(torch.float8_e8m0fnu)
    ex, q_gpu, p_gpu = _gpu(lists), ref.to(qkv, DEV), ref.to(proj, DEV)
    router, norm = _rows(8, hidden, "bf16", 43) * 0.1, 1 + 0.1 * _rows(1, hidden, "bf16", 44)[0]
    lengths = [3, 16, 40, 17, 100]
    table = [[7 * s + b for b in range(7)] for s in range(seqs)]
    cache = kv.random_cache(st, 35, heads, dim, block, 45)
    cache.v_scale = torch.full_like(cache.v_scale.view(torch.uint8), 121).view(torch.float8_e8m0fnu)
    dev = kv.to(cache, DEV)
    h = _rows(seqs, hidden, "bf16", 46)
    tb = torch.tensor(table, dtype=torch.int32, device=DEV)
    hd = h.to(DEV)
    for step in range(3):
        lengths = [n + 1 for n in lengths]
        ln = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        x = st.rms_norm(hd, norm.to(DEV))
        y = st.linear(x, q_gpu)
        q, k, v = (t.reshape(seqs, -1, dim) for t in y.split([group * heads * dim, heads * dim, heads * dim], 1))
        q, k, v = (y[:, a:b].unflatten(1, (-1, dim)) for a, b in ((0, group * heads * dim), (group * heads * dim, wide - heads * dim), (wide - heads * dim, wide)))
        before = kv.cpu(dev)
        st.kv_append(dev, k, v, tb, ln)
        o = st.kv_attention(q, dev, tb, ln)
        x2, h2 = st.rms_norm(st.linear(o.flatten(1), p_gpu), norm.to(DEV), residual=hd)
        w, ids = st.moe_route(x2, router.to(DEV), 2)
        out = st.moe(x2, ex, ids, w, residual=h2)
        # each link against its own 64-bit form on what it was given
        wk, wv, wks, wvs = kv.append(before, k.cpu(), v.cpu(), table, lengths)
        assert (ref.e4m3(dev.k.cpu()) == wk).all() and (ref.e4m3(dev.v.cpu()) == wv).all()
        want, tol = kv.attention(q.cpu(), kv.cpu(dev), table, lengths)
        kv.check(o, want, tol)
        rw, rids = mref.route(x2.cpu(), router, 2)
        assert torch.equal(rids, ids.cpu())
        want, tol = mref.moe(x2.cpu(), lists, ids.cpu(), w.cpu(), residual=h2.cpu())
        mref.check(out, want, tol)
        hd = (out / out.float().square().mean(1, keepdim=True).sqrt()).to(torch.bfloat16)
