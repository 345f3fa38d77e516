"""CPU: which places for a result beside its inputs are taken for an overlap."""
import pytest
import torch

from device_checkpoint_dequantisation_amd.ops import _overlaps


def _bytes(t):
    i = torch.arange(t.untyped_storage().nbytes() // t.element_size()).as_strided(t.shape, t.stride(), t.storage_offset()).reshape(-1)
    return set(i.tolist())


def test_heads_in_columns_of_one_buffer():
    """Queries, keys and results as parts of one wide buffer: [tokens, heads, head_dim] each."""
    buf = torch.zeros(5, 96, dtype=torch.bfloat16)
    part = lambda a, heads, dim: buf[:, a:a + heads * dim].unflatten(1, (heads, dim))   # noqa: E731
    cases = refused = 0
    for a, ha, da in ((0, 4, 8), (8, 2, 16), (32, 4, 8), (61, 3, 5), (95, 1, 1), (40, 1, 20)):
        for b, hb, db in ((0, 4, 8), (31, 4, 8), (32, 4, 8), (33, 2, 16), (64, 2, 16), (64, 4, 8), (76, 5, 4)):
            x, y = part(a, ha, da), part(b, hb, db)
            cases += 1
            refused += (want := bool(_bytes(x) & _bytes(y)))
            assert _overlaps(x, y) == want, (a, ha, da, b, hb, db)
    assert 0 < refused < cases


@pytest.mark.parametrize("gap", [0, 3])
def test_heads_apart(gap):
    """Every other head of one buffer: as far as the rows tell they overlap, which is refused whether or not they do."""
    buf = torch.zeros(4, 6, 8 + gap)
    x, y = buf[:, 0::2, :8], buf[:, 1::2, :8]
    assert not _bytes(x) & _bytes(y)
    assert _overlaps(x, x) and _overlaps(x, buf) and _overlaps(buf[:, :, :8], y)
    assert not _overlaps(buf[:, :2, :8], buf[:, 2:, :8]) and not _overlaps(buf[:2], buf[2:])


def test_attention_beside_its_queries(monkeypatch):
    """Results into the columns next to the queries of one wide buffer are taken, into the same ones refused."""
    import device_checkpoint_dequantisation_amd as st
    from device_checkpoint_dequantisation_amd import kv_cache
    monkeypatch.setattr(kv_cache, "_on_device", lambda device, tensors, who: None)
    monkeypatch.setattr(kv_cache, "_launch", lambda *a: None)
    cache = st.QuantizedKvCache.empty(2, 2, 64, 16, "cpu")
    table, lengths = torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    wide = torch.zeros(3, 3 * 256, dtype=torch.bfloat16)
    q, out, part = (wide[:, a:a + 256].unflatten(1, (4, 64)) for a in (0, 256, 192))
    assert st.kv_attention(q, cache, table, lengths, out=out) is out
    for bad in (q, part):
        with pytest.raises(ValueError, match="overlaps"):
            st.kv_attention(q, cache, table, lengths, out=bad)
