"""GPU: attention over the 8-bit cache where the powers of two of pages lie far apart."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import kv_reference as kv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E8M0 = torch.float8_e8m0fnu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _queries(tokens, heads, dim, dt, seed, size=0.5):
    return (size * torch.randn(tokens, heads, dim, generator=torch.Generator().manual_seed(seed))).to(kv.DT[dt])


def _run(q, cache, table, lengths, starts, **kw):
    return st.kv_attention(q.to(DEV), kv.to(cache, DEV), _i32(table), _i32(lengths), starts=_i32(starts), **kw)


def _starts(counts):
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    return starts


# (dim, heads, query heads each): few rows of a sequence's head, and more than 8192 / dim of them
FEW_MANY = [(64, 2, 4, 2), (64, 1, 4, 40), (128, 2, 2, 3), (128, 1, 4, 20), (256, 1, 3, 2), (256, 1, 5, 9)]


@pytest.mark.parametrize("dim,heads,group,count", FEW_MANY)
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("how", ["causal", "window", "all"])
def test_scales_of_pages_nobody_sees(dim, heads, group, count, block, how):
    """Entries behind a sequence's end and before its first query's window name pages of other sequences with any scale: the results
    are bit for bit those of entries that name none."""
    lengths, counts = [count + 17, 203, 70], [count, max(1, count // 2), 1]
    starts = _starts(counts)
    kw = {"causal": dict(), "window": dict(window=40), "all": dict(causal=False)}[how]
    width = -(-max(lengths) // block) + 128 // block + 1
    pages = 3 * width + 1
    cache = kv.random_cache(st, pages, heads, dim, block, 3)
    cache.v_scale = torch.full((pages, heads), 121, dtype=torch.uint8).view(E8M0)
    q = _queries(starts[-1], heads * group, dim, "bf16", 4)
    own = [[s * width + b for b in range(width)] for s in range(3)]
    seen = []
    for s, n in enumerate(lengths):
        first = max(0, n - counts[s] - 40 + 1) if how == "window" else 0          # the first token that a query sees
        seen.append([first // block <= b < -(-n // block) for b in range(width)])
    none = [[p if x else -1 for p, x in zip(*row)] for row in zip(own, seen)]
    assert none != own
    print(f"attention unseen scales {dim} {block} {group} x {count} {how}", flush=True)
    want = _run(q, cache, none, lengths, starts, **kw)
    ref, tol = kv.attention(q, cache, none, lengths, starts, **kw)
    kv.check(want, ref, tol)
    for code in (0, 141, 200, 254, 255):
        other = type(cache)(cache.k, cache.v, cache.k_scale.clone(), cache.v_scale.clone())
        for s in range(3):
            for b in range(width):
                if not seen[s][b]:
                    kv.raw(other.v_scale)[own[s][b]] = code
                    kv.raw(other.k_scale)[own[s][b]] = code
        got = _run(q, other, own, lengths, starts, **kw)
        assert torch.equal(got, want), f"scale code {code}: {int((got != want).sum())} of {got.numel()} results differ"


def _far_apart(dim, heads, group, block, n, count, codes, seed, dt="bf16", **kw):
    """One sequence of n tokens whose pages take their values' scale codes from `codes` in turn."""
    width = -(-n // block)
    cache = kv.random_cache(st, width, heads, dim, block, seed)
    cache.v_scale = torch.tensor([[codes[b % len(codes)]] * heads for b in range(width)], dtype=torch.uint8).view(E8M0)
    q = _queries(count, heads * group, dim, dt, seed + 1)
    table = [list(range(width))]
    got = _run(q, cache, table, [n], [0, count], **kw)
    want, tol = kv.attention(q, cache, table, [n], [0, count], **kw)
    # Values meet the numerators as fp16 numbers relative to a power of two, at most 2^8 times the largest among the pages that a query sees: exact
    # down to 2^-15 of it, below to half of fp16's smallest step, 2^-25 of it, which is 2^-17 of the query's own, and the weights add up to 1.
    for t in range(count):
        pos = n - count + t
        see = [codes[b % len(codes)] for b in range(max(0, pos - (kw.get("window") or n) + 1) // block, pos // block + 1)]
        if max(see) + 8 - min(see) > 15:
            tol[t] += 2.0 ** (max(see) - 127 - 17)
    kv.check(got, want, tol)


@pytest.mark.parametrize("dim,heads,group,count", FEW_MANY)
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("codes", [(127, 107), (97, 127), (127, 100, 112, 90), (140, 20), (1, 125), (0, 127), (60, 128, 59)])
def test_scales_that_only_some_queries_see(dim, heads, group, count, block, codes):
    """Queries whose windows begin and end on different pages: what one sees and another does not leaves the other's result alone."""
    print(f"attention windows over far scales {dim} {block} {group} x {count} {codes}", flush=True)
    for window in (1, block, 2 * block + 5):
        _far_apart(dim, heads, group, block, 5 * block + count // 2 + 1, count, codes, 7, window=window)
    _far_apart(dim, heads, group, block, 5 * block + count // 2 + 1, count, codes, 7)


@pytest.mark.parametrize("dim,heads,group,count", FEW_MANY)
def test_scales_rise_and_fall(dim, heads, group, count):
    """Pages whose scales rise, or fall, by 6 binades each: hundreds of tokens apart they differ by more than any 16-bit number's range."""
    up = list(range(20, 128, 6))
    print(f"attention rising scales {dim} {group} x {count}", flush=True)
    for codes in (up, up[::-1]):
        for window in (1, 30, 100):
            _far_apart(dim, heads, group, 16, 16 * len(codes), count, codes, 9, window=window)
        _far_apart(dim, heads, group, 16, 16 * len(codes), count, codes, 9, dt="f16", window=50)


@pytest.mark.parametrize("dim,heads,group,count", FEW_MANY)
@pytest.mark.parametrize("window", [None, 4500])
def test_far_scales_in_parts(dim, heads, group, count, window):
    """Scales that rise to the last page, which the first queries do not see, or fall from the first of their windows, over tokens that are
    cut into parts."""
    print(f"attention far scales in parts {dim} {group} x {count} {window}", flush=True)
    for codes in (list(range(45, 124)), list(range(123, 44, -1))):
        _far_apart(dim, heads, group, 64, 79 * 64 - 64 + count // 2 + 1, count, codes, 15, window=window)


@pytest.mark.parametrize("dim,heads,group,count", FEW_MANY)
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_far_scales_nan_and_missing_pages(dim, heads, group, count, dt):
    """NaN codes where no query looks, one that only some see, a page of NaN scale that only some see, and a page that is not there."""
    block, pages = 16, 12
    n, window = pages * block - 5, 50
    first = max(0, n - count - window + 1)
    cache = kv.random_cache(st, pages, heads, dim, block, 17)
    cache.v_scale = torch.tensor([[(127, 100, 80, 121)[b % 4]] * heads for b in range(pages)], dtype=torch.uint8).view(E8M0)
    table = [list(range(pages))]
    table[0][pages - 3] = -1
    q = _queries(count, heads * group, dim, dt, 18)
    k, v, vs = kv.raw(cache.k), kv.raw(cache.v), kv.raw(cache.v_scale)
    for t in list(range(first)) + list(range(n, pages * block)):
        k[t // block, :, t % block] = 0x7F
        v[t // block, :, :, t % block] = 0xFF
    t = n - count // 2 - 1                      # the last queries see it, the first ones do not
    v[t // block, heads - 1, 5, t % block] = 0x7F
    print(f"attention far scales with NaN {dim} {group} x {count} {dt}", flush=True)
    for bad in (None, first // block):
        if bad is not None:
            vs[bad] = 255
        got = _run(q, cache, table, [n], [0, count], window=window)
        want, tol = kv.attention(q, cache, table, [n], [0, count], window=window)
        assert (bad is not None or not want.isnan().all()) and (want.isnan() == got.cpu().isnan()).all()
        tol += 2.0 ** (0 - 17)                  # as above: the largest seen is 2^0
        kv.check(got, want, tol)


@pytest.mark.parametrize("dim,heads,group,count", FEW_MANY)
@pytest.mark.parametrize("n", [90, 5000])
def test_values_near_the_largest_number(dim, heads, group, count, n):
    """Values up to 448 * 2^119: sums of their products pass fp32's range, the results, which are their means, do not; and values near
    the smallest."""
    print(f"attention largest values {dim} {group} x {count} of {n}", flush=True)
    for code in (246, 20, 3):
        _far_apart(dim, heads, group, 64, n, count, (code,), 11)
        _far_apart(dim, heads, group, 64, n, count, (code, code - 1, code - 3), 12)


def test_far_scales_in_a_graph():
    """Captured with pages alike, replayed with pages far apart and alike again, into part of a wide buffer; several sequences, some of
    whose rows nobody has."""
    dim, heads, group, block, window = 128, 2, 2, 16, 40
    lengths, counts = [100, 0, 230, 64], [30, 2, 9, 50]
    starts = [3]
    for c in counts:
        starts.append(starts[-1] + c)
    width = -(-max(lengths) // block)
    cache = kv.random_cache(st, 4 * width, heads, dim, block, 19)
    table = [[s * width + b for b in range(width)] for s in range(4)]
    tokens = starts[-1] + 4
    q = _queries(tokens, heads * group, dim, "f16", 20)
    wide = torch.zeros(tokens, 3 * heads * group * dim + 5, dtype=torch.float16, device=DEV)
    part = lambda a: wide[:, a:a + heads * group * dim].unflatten(1, (heads * group, dim))   # noqa: E731
    qd, out = part(1), part(1 + heads * group * dim + 3)
    qd.copy_(q.to(DEV))
    out.fill_(7.0)
    d, tb, ln, sd = kv.to(cache, DEV), _i32(table), _i32(lengths), _i32(starts)

    def step():
        st.kv_attention(qd, d, tb, ln, starts=sd, max_new=50, window=window, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    near = kv.raw(cache.v_scale).clone()
    far = torch.tensor([[(130, 90)[p % 2]] * heads for p in range(4 * width)], dtype=torch.uint8)
    for codes in (near, far, near, far):
        d.v_scale.view(torch.uint8).copy_(codes.to(DEV))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        host = type(cache)(cache.k, cache.v, cache.k_scale, codes.view(E8M0))
        want, tol = kv.attention(q, host, table, lengths, starts, window=window)
        if codes is far:
            # as in _far_apart, for queries that see a page of 2^3 (whose results are not tiny)
            tol[starts[0]:starts[-1]] += 2.0 ** (130 - 127 - 17) * (want[starts[0]:starts[-1]].abs().amax(2, keepdim=True) > 2.0 ** -8)
        kv.check(out[starts[0]:starts[-1]], want[starts[0]:starts[-1]], tol[starts[0]:starts[-1]])
        assert (out[:starts[0]] == 7).all() and (out[starts[-1]:] == 7).all()
        assert torch.equal(st.kv_attention(qd, d, tb, ln, starts=sd, max_new=50, window=window)[starts[0]:starts[-1]], out[starts[0]:starts[-1]])
    assert (wide[:, 0] == 0).all() and (wide[:, -1] == 0).all()
