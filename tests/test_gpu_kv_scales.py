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
