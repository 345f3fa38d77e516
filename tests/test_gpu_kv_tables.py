"""GPU: attention over the 8-bit cache with tables that are much wider than any sequence, as a graph captured once for contexts to come has."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from tests import kv_reference as kv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(dim, heads, group, count, lengths, block, seed):
    """(q, cache, table, lengths) on the GPU, and the first two on the CPU."""
    seqs, tight = len(lengths), -(-max(lengths) // block)
    cache = kv.random_cache(st, seqs * tight, heads, dim, block, seed)
    q = (0.5 * torch.randn(seqs * count, heads * group, dim, generator=torch.Generator().manual_seed(seed + 1))).to(torch.bfloat16)
    table = torch.arange(seqs * tight, dtype=torch.int32, device=DEV).view(seqs, tight)
    return q.to(DEV), kv.to(cache, DEV), table, torch.tensor(lengths, dtype=torch.int32, device=DEV), q, cache


def _widened(table, width):
    wide = torch.zeros(table.shape[0], width, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("dim,heads,group,count", [(64, 2, 4, 2), (128, 8, 4, 1), (256, 1, 3, 2), (128, 1, 4, 40)])
@pytest.mark.parametrize("window", [None, 900])
def test_results(dim, heads, group, count, window):
    lengths = [5000, 70, 2300, 1100, 0, 63]
    q, cache, table, n, q_host, host = _case(dim, heads, group, count, lengths, 64, 13)
    want, tol = kv.attention(q_host, host, table.tolist(), lengths, window=window)
    for width in (table.shape[1], table.shape[1] + 1, 300, 2048, 5000):
        print(f"attention wide table {dim} {count} {window} {width}", flush=True)
        kv.check(st.kv_attention(q, cache, _widened(table, width), n, window=window), want, tol)


def test_cost():
    """The table's width alone makes no call much slower (16 sequences' 4 drafts, 64 queries on 8 heads of 128: 5 times while parts of a sequence
    were cut by it)."""
    q, cache, table, n, _, _ = _case(128, 8, 8, 4, [1000 + 450 * s for s in range(16)], 64, 14)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)

    def fastest(t):
        times = []
        for i in range(6):
            a.record()
            for _ in range(20):
                st.kv_attention(q, cache, t, n)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) / 20)
        return min(times[1:])
    tight, wide = fastest(table), fastest(_widened(table, 2048))
    print(f"tight {1e3 * tight:.1f} us, wide {1e3 * wide:.1f}", flush=True)
    assert wide < 2.5 * tight
