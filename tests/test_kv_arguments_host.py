"""CPU: what kv_attention hands to the library."""
import pytest
import torch

import device_checkpoint_dequantisation_amd as st
from device_checkpoint_dequantisation_amd import kv_cache


@pytest.mark.parametrize("window,want", [(None, 0), (1, 1), (700, 700), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 64, 2 ** 31 - 1),
                                         (2 ** 64 + 1, 2 ** 31 - 1), (10 ** 30, 2 ** 31 - 1)])
def test_windows_of_any_size(monkeypatch, window, want):
    """A window is at most what the library takes for all of a sequence, never a larger number's low 64 bits."""
    got = []
    monkeypatch.setattr(kv_cache, "_on_device", lambda device, tensors, who: None)
    monkeypatch.setattr(kv_cache, "_launch", lambda f, args, *a: got.append(args.window))
    cache = st.QuantizedKvCache.empty(2, 2, 64, 16, "cpu")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    st.kv_attention(q, cache, torch.zeros(3, 1, dtype=torch.int32), torch.ones(3, dtype=torch.int32), window=window)
    assert got == [want]
