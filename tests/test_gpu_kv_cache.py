"""GPU: the 8-bit cache.  Appending against its definition, code by code; attention against a 64-bit form: head sizes, groups, pages,
lengths from none to long ones, windows, rows that see nothing, NaN where nobody looks; streams, graphs, offsets past 32 bits."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import kv_reference as kv
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _tables(lengths, block, extra=0, seed=0, spare=3):
    """Pages in random order for sequences of these lengths: (table, pages); entries behind a sequence's end are no pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 0) // block) for n in lengths]
    order = torch.randperm(sum(need) + spare, generator=g).tolist()
    width = max(max(need), 1) + extra
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-7] * (width - n))
        at += n
    return table, sum(need) + spare


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _same(cache, want):
    k, v, ks, vs = want
    for got, w, name in ((cache.k, k, "k"), (cache.v, v, "v")):
        got = ref.e4m3(got.cpu())
        assert ((got == w) | (got.isnan() & w.isnan())).all(), f"{name}: {((got != w) & ~w.isnan()).nonzero()[:4].tolist()}"
    for got, w in ((cache.k_scale, ks), (cache.v_scale, vs)):
        assert torch.equal(kv.raw(got).to(torch.int64) - 127, w)


def _new(tokens, heads, dim, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(2, tokens, heads, dim, generator=g) * torch.exp(torch.randn(tokens, heads, 1, generator=g)) * scale
    return x[0].to(kv.DT[dt]), x[1].to(kv.DT[dt])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,dim,block", [(1, 32, 16), (3, 64, 32), (2, 128, 64), (8, 96, 16), (2, 256, 128), (5, 160, 64)])
def test_append(dt, heads, dim, block):
    counts = [1, block, 0, block + 1, 2 * block - 1, 7]
    had = [0, 3, 5, block - 1, 1, 2 * block]
    lengths = [a + b for a, b in zip(counts, had)]
    starts = [2]
    for c in counts:
        starts.append(starts[-1] + c)
    table, pages = _tables(lengths, block, 1)
    cache = kv.random_cache(st, pages, heads, dim, block, 1, spread=6)
    k, v = _new(starts[-1] + 3, heads, dim, dt, 2, 0.3)
    print(f"append {dt} {heads} {dim} {block}", flush=True)
    want = kv.append(cache, k, v, table, lengths, starts)
    for most in (None, max(counts)):
        d = kv.to(cache, DEV)
        st.kv_append(d, k.to(DEV), v.to(DEV), _i32(table), _i32(lengths), starts=_i32(starts), max_new=most)
        _same(d, want)


@pytest.mark.parametrize("block", [16, 64])
def test_append_grows(block):
    """Token by token, each page's scale growing and its codes following; what the pages held before their first token is no part."""
    heads, dim, seqs = 2, 64, 3
    lengths = [0, 5, block - 2]
    table, pages = _tables([n + 2 * block for n in lengths], block)
    cache = kv.random_cache(st, pages, heads, dim, block, 3)
    d = kv.to(cache, DEV)
    tb = _i32(table)
    for i in range(block + 4):
        lengths = [n + 1 for n in lengths]
        k, v = _new(seqs, heads, dim, "bf16", 100 + i, 1.3 ** i * 1e-3)
        want = kv.append(kv.cpu(d), k, v, table, lengths)
        st.kv_append(d, k.to(DEV), v.to(DEV), tb, _i32(lengths))
        _same(d, want)


def test_append_special_values():
    """NaN and infinities, zeros, the smallest and largest numbers of each type."""
    for dt in ("bf16", "f16", "f32"):
        block, heads, dim = 16, 2, 32
        f = torch.finfo(kv.DT[dt])
        k, v = _new(40, heads, dim, dt, 5)
        k[0] = 0.0
        v[:16] = 0.0
        k[3, 0, 4], k[3, 1, 5], v[20, 0, 1] = float("nan"), float("inf"), float("-inf")
        k[17:] *= 1e-3
        v[18, 1, 3], v[39, 0, 0], k[33, 1, 1] = f.max, -f.max, f.smallest_normal * f.eps
        table, pages = _tables([40], block)
        cache = kv.random_cache(st, pages, heads, dim, block, 6)
        want = kv.append(cache, k, v, table, [40])
        d = kv.to(cache, DEV)
        st.kv_append(d, k.to(DEV), v.to(DEV), _i32(table), _i32([40]))
        _same(d, want)


def test_append_strides_and_missing_pages():
    """Parts of one wide projection at odd offsets; blocks on no page and past the table are left out."""
    heads, dim, block, tokens = 3, 64, 32, 90
    g = torch.Generator().manual_seed(7)
    for shift in (0, 1):
        wide = torch.randn(tokens, 2 * heads * dim + 7 + shift, generator=g).to(torch.bfloat16)
        k = wide[:, shift:shift + heads * dim].view(tokens, heads, dim)
        v = wide[:, shift + heads * dim:shift + 2 * heads * dim].view(tokens, heads, dim)
        table, lengths, pages = [[4, -1, 9], [2, 5, 0]], [100, 45], 6
        starts = [0, 45, 90]
        cache = kv.random_cache(st, pages, heads, dim, block, 8)
        want = kv.append(cache, k, v, table, lengths, starts)
        d = kv.to(cache, DEV)
        w = wide.to(DEV)
        wide_table = torch.full((2, 5), 99, dtype=torch.int32, device=DEV)
        wide_table[:, :3] = _i32(table)
        st.kv_append(d, w[:, shift:shift + heads * dim].view(tokens, heads, dim),
                     w[:, shift + heads * dim:shift + 2 * heads * dim].view(tokens, heads, dim), wide_table[:, :3], _i32(lengths), starts=_i32(starts))
        _same(d, want)


def _case(heads, group, dim, block, lengths, counts, dt, seed=11, gap=0, extra=0):
    starts = [gap]
    for c in counts:
        starts.append(starts[-1] + c)
    table, pages = _tables(lengths, block, extra, seed)
    cache = kv.random_cache(st, pages, heads, dim, block, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = (0.5 * torch.randn(starts[-1] + gap, heads * group, dim, generator=g)).to(kv.DT[dt])
    return q, cache, table, starts


def _attend(q, cache, table, lengths, starts=None, **kw):
    out = st.kv_attention(q.to(DEV), kv.to(cache, DEV), _i32(table), _i32(lengths), starts=None if starts is None else _i32(starts), **kw)
    kw.pop("out", None)
    want, tol = kv.attention(q, cache, table, lengths, starts, **kw)
    kv.check(out, want, tol)
    return out


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,group", [(1, 1), (2, 4), (3, 5), (1, 16), (1, 20)])
def test_single_tokens(dt, dim, block, heads, group):
    lengths = [1, 63, 64, 65, 200, 1031]
    q, cache, table, starts = _case(heads, group, dim, block, lengths, [1] * 6, dt)
    print(f"attention one token {dt} {dim} {block} {heads} {group}", flush=True)
    _attend(q, cache, table, lengths)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim,block,heads,group", [(64, 16, 2, 3), (128, 64, 2, 4), (128, 128, 1, 1), (256, 32, 1, 2), (128, 16, 1, 8)])
@pytest.mark.parametrize("window", [None, 1, 70, 300])
def test_prompts(dt, dim, block, heads, group, window):
    lengths, counts = [150, 64, 333, 90, 5], [150, 3, 40, 0, 5]
    q, cache, table, starts = _case(heads, group, dim, block, lengths, counts, dt, gap=2)
    print(f"attention prompts {dt} {dim} {block} {heads} {group} {window}", flush=True)
    _attend(q, cache, table, lengths, starts, window=window)
    _attend(q, cache, table, lengths, starts, window=window, max_new=40)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim,group", [(64, 2), (128, 7), (256, 1)])
def test_not_causal(dt, dim, group):
    """An encoder's states of another length, none at all among them."""
    lengths, counts = [77, 0, 130, 1], [90, 4, 3, 17]
    q, cache, table, starts = _case(2, group, dim, 16, lengths, counts, dt)
    print(f"attention not causal {dt} {dim} {group}", flush=True)
    out = _attend(q, cache, table, lengths, starts, causal=False)
    assert (out[starts[1]:starts[2]] == 0).all()


@pytest.mark.parametrize("dim,heads,group", [(128, 1, 4), (64, 2, 1)])
def test_long(dim, heads, group):
    """Split over the tokens and joined, unevenly."""
    lengths = [9000, 4100, 70]
    q, cache, table, starts = _case(heads, group, dim, 64, lengths, [2, 1, 3], "bf16")
    print(f"attention long {dim} {heads} {group}", flush=True)
    _attend(q, cache, table, lengths, starts)
    _attend(q, cache, table, lengths, starts, window=5000)


@pytest.mark.parametrize("dim,heads,group,count", [(64, 1, 1, 3), (64, 3, 3, 11), (128, 2, 2, 5), (128, 1, 5, 30), (256, 1, 3, 2), (256, 2, 1, 40)])
@pytest.mark.parametrize("longest", [1100, 2300, 5000, 17000])
def test_parts(dim, heads, group, count, longest):
    """Two parts to many, of sequences that have all of them, some, one and none."""
    lengths, counts = [longest, 0, longest // 2, 40], [count, 2, 1, count]
    q, cache, table, starts = _case(heads, group, dim, 64, lengths, counts, "bf16", gap=1)
    print(f"attention parts {dim} {heads} {group} {count} {longest}", flush=True)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    got = st.kv_attention(q.to(DEV), kv.to(cache, DEV), _i32(table), _i32(lengths), starts=_i32(starts), out=out)
    want, tol = kv.attention(q, cache, table, lengths, starts)
    kv.check(got[1:-1], want[1:-1], tol[1:-1])
    assert (out[0] == 7).all() and (out[-1] == 7).all()


def test_rows_that_see_nothing():
    """More queries than tokens, sequences of no tokens, tokens on no page."""
    lengths, counts = [3, 0, 40], [7, 2, 5]
    q, cache, table, starts = _case(2, 2, 64, 16, lengths, counts, "bf16")
    table[2] = [-1, 10 ** 6, 1]
    out = _attend(q, cache, table, lengths, starts)
    assert (out[:4] == 0).all() and (out[7:9] == 0).all()
    table[2] = [-1, -1, -1]
    out = _attend(q, cache, table, lengths, starts)
    assert (out[9:] == 0).all()
    # a length past the table: its tokens there are seen, by queries whose own place is past it too
    _attend(q, cache, table[:2] + [[1, 2, 0]], [3, 0, 50], starts)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("dim,block", [(64, 16), (128, 64), (256, 128)])
def test_nan_where_nobody_looks(dt, dim, block):
    """Codes of NaN behind a sequence's end, before a window and behind a query's own token change nothing; those a query sees make
    its result NaN, in that head and (for values) that column."""
    lengths, counts = [70, 200], [30, 9]
    q, cache, table, starts = _case(2, 3, dim, block, lengths, counts, dt)
    want = st.kv_attention(q.to(DEV), kv.to(cache, DEV), _i32(table), _i32(lengths), starts=_i32(starts), window=50)
    c = kv.raw(cache.k).clone(), kv.raw(cache.v).clone()
    pages = cache.k.shape[0]

    def place(s, t):
        return table[s][t // block], t % block
    unseen = [(s, t) for s in range(2) for t in list(range(lengths[s], -(-lengths[s] // block) * block)) + list(range(max(0, lengths[s] - counts[s] - 49)))]
    for s, t in unseen:
        p, o = place(s, t)
        c[0][p, :, o] = 0x7F
        c[1][p, :, :, o] = 0xFF
    used = {x for row in table for x in row}
    for p in range(pages):
        if p not in used:
            c[0][p] = 0x7F
    bad = type(cache)(c[0].view(torch.float8_e4m3fn), c[1].view(torch.float8_e4m3fn), cache.k_scale, cache.v_scale)
    print(f"attention nan {dt} {dim} {block}", flush=True)
    got = st.kv_attention(q.to(DEV), kv.to(bad, DEV), _i32(table), _i32(lengths), starts=_i32(starts), window=50)
    assert torch.equal(got, want)
    # one value of a token in the middle of the queries, one key of another
    p, o = place(0, 55)
    c[1][p, 1, 9, o] = 0x7F
    p, o = place(1, 195)
    c[0][p, 0, o, 3] = 0xFF
    bad = type(cache)(c[0].view(torch.float8_e4m3fn), c[1].view(torch.float8_e4m3fn), cache.k_scale, cache.v_scale)
    got = st.kv_attention(q.to(DEV), kv.to(bad, DEV), _i32(table), _i32(lengths), starts=_i32(starts), window=50)
    here = torch.zeros_like(got, dtype=torch.bool)
    here[15:30, 3:, 9] = True             # queries at 55 and behind
    here[30 + 4:, :3] = True              # queries at 195 and behind
    assert torch.equal(got.isnan(), here)
    assert torch.equal(got[~here], want[~here])


def test_scales_far_apart():
    """Values of pages many binades apart; keys too, whose scores then take turns as the largest."""
    block, dim = 16, 64
    q, cache, table, starts = _case(1, 4, dim, block, [400], [6], "bf16")
    g = torch.Generator().manual_seed(3)
    cache.v_scale = (127 + torch.randint(-12, 1, cache.v_scale.shape, generator=g)).to(torch.uint8).view(torch.float8_e8m0fnu)
    cache.k_scale = (120 + torch.randint(-4, 4, cache.k_scale.shape, generator=g)).to(torch.uint8).view(torch.float8_e8m0fnu)
    _attend(q, cache, table, [400], starts)
    # a page of zeros has the smallest scale there is and takes its share of the softmax
    kv.raw(cache.v)[table[0][3]] = 0
    kv.raw(cache.v_scale)[table[0][3]] = 0
    _attend(q, cache, table, [400], starts)


def test_scores_far_apart():
    """Scores that rise and fall by hundreds: the running maximum moves in every step, in either direction."""
    block, dim, n = 64, 128, 1000
    q, cache, table, starts = _case(1, 2, dim, block, [n], [3], "bf16")
    for order in (1, -1):
        e = torch.arange(cache.k.shape[0]) % 7
        for i, p in enumerate(table[0][::order]):
            if 0 <= p:
                e[p] = i % 9
        cache.k_scale = (118 + e[:, None]).to(torch.uint8).view(torch.float8_e8m0fnu)
        _attend(q, cache, table, [n], starts, scale=0.05)
        _attend(q, cache, table, [n], starts, scale=2.0)


def test_strides_and_out():
    """Queries in a wide projection at an odd offset, results into a part of a wide buffer; rows of no sequence stay."""
    lengths, counts = [70, 33], [20, 3]
    q, cache, table, starts = _case(2, 3, 64, 32, lengths, counts, "f16", gap=2)
    tokens, h, dim = q.shape
    wide = torch.zeros(tokens, h * dim + 9, dtype=torch.float16, device=DEV)
    wide[:, 1:1 + h * dim] = q.view(tokens, -1).to(DEV)
    q2 = wide[:, 1:1 + h * dim].view(tokens, h, dim)
    buf = torch.full((tokens, h * dim + 5), 7.0, dtype=torch.float16, device=DEV)
    out = buf[:, 3:3 + h * dim].view(tokens, h, dim)
    wt = torch.full((2, table.__len__() + 6), -1, dtype=torch.int32, device=DEV)
    wt[:, :len(table[0])] = _i32(table)
    got = st.kv_attention(q2, kv.to(cache, DEV), wt[:, :len(table[0])], _i32(lengths), starts=_i32(starts), out=out)
    assert got is out
    want, tol = kv.attention(q, cache, table, lengths, starts)
    kv.check(out[2:25], want[2:25], tol[2:25])
    assert (out[:2] == 7).all() and (out[25:] == 7).all() and (buf[:, :3] == 7).all() and (buf[:, -2:] == 7).all()


def test_offsets_past_32_bits():
    """Pages beyond 4 GiB of codes."""
    heads, dim, block = 8, 128, 128
    pages = 2 ** 32 // (heads * dim * block) + 40
    d = st.QuantizedKvCache.empty(pages, heads, dim, block, DEV)
    table = [[pages - 1, pages - 7, 3]]
    k, v = _new(300, heads, dim, "bf16", 21)
    st.kv_append(d, k.to(DEV), v.to(DEV), _i32(table), _i32([300]))
    small = st.QuantizedKvCache(*(t.view(torch.uint8)[[pages - 1, pages - 7, 3]].cpu().view(t.dtype) for t in (d.k, d.v, d.k_scale, d.v_scale)))
    blank = kv.cpu(st.QuantizedKvCache.empty(3, heads, dim, block, "cpu"))
    _same(small, kv.append(blank, k, v, [[0, 1, 2]], [300]))
    q = (0.3 * torch.randn(2, 8, dim, generator=torch.Generator().manual_seed(22))).to(torch.bfloat16)
    got = st.kv_attention(q.to(DEV), d, _i32(table), _i32([300]))
    want, tol = kv.attention(q, small, [[0, 1, 2]], [300])
    kv.check(got, want, tol)


def test_streams_and_graph():
    """Captured once and replayed while lengths, table and inputs change, with eager work between; then on a side stream."""
    heads, group, dim, block, seqs = 2, 4, 128, 64, 3
    lengths = [60, 200, 63]
    table, pages = _tables([n + 200 for n in lengths], block)
    d = kv.to(kv.random_cache(st, pages, heads, dim, block, 31), DEV)
    start = kv.cpu(d)
    k, v = (torch.zeros(seqs, heads, dim, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros(seqs, heads * group, dim, dtype=torch.bfloat16, device=DEV)
    tb, ln = _i32(table), _i32(lengths)
    out = torch.empty_like(q)

    def step():
        st.kv_append(d, k, v, tb, ln)
        st.kv_attention(q, d, tb, ln, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t, s in zip((d.k, d.v, d.k_scale, d.v_scale), (start.k, start.v, start.k_scale, start.v_scale)):
        t.view(torch.uint8).copy_(s.view(torch.uint8))
    for i in range(5):
        nk, nv = _new(seqs, heads, dim, "bf16", 40 + i)
        nq = torch.randn(seqs, heads * group, dim, generator=torch.Generator().manual_seed(60 + i)).to(torch.bfloat16)
        lengths = [n + 1 for n in lengths]
        before = kv.cpu(d)
        k.copy_(nk), v.copy_(nv), q.copy_(nq), ln.copy_(_i32(lengths))
        g.replay()
        torch.cuda.synchronize()
        _same(d, kv.append(before, nk, nv, table, lengths))
        want, tol = kv.attention(nq, kv.cpu(d), table, lengths)
        kv.check(out, want, tol)
        eager = st.kv_attention(q, d, tb, ln)
        assert torch.equal(eager, out)
    got = st.kv_attention(q, d, tb, ln, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, out)


def test_refusals():
    c = kv.to(kv.random_cache(st, 4, 2, 64, 16, 1), DEV)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    t, n = _i32([[0], [1]]), _i32([3, 4])
    with pytest.raises(ValueError, match="tensors on"):
        st.kv_attention(q, c, t.cpu(), n)
    with pytest.raises(ValueError, match="overlaps"):
        st.kv_attention(q, c, t, n, out=q)
    with pytest.raises(RuntimeError, match="no backward"):
        st.kv_attention(q.clone().requires_grad_(), c, t, n)
    k = c.k.view(torch.uint8).view(torch.bfloat16).view(4, 2, -1)[:2, :, :64]
    with pytest.raises(ValueError, match="overlaps"):
        st.kv_append(c, k, k, t, n)
