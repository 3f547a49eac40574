"""The attention layer's positions, weights and eviction: what it hands on, without a GPU."""
from types import SimpleNamespace

import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from block_scaled_bit_nvfp4_amd.attention_layer import AttentionLayer


def _layer(freqs):
    layer = object.__new__(AttentionLayer)
    layer.max_tokens, layer.hidden, layer.freqs, layer.heads, layer.device = 4, 16, freqs, 2, torch.device("cpu")
    layer.cache = SimpleNamespace(page_tokens=16)
    return layer


def test_positions_come_with_frequencies():
    batch, x = SimpleNamespace(tokens=3), torch.zeros(3, 16)
    with pytest.raises(ValueError, match="positions"):
        _layer(torch.ones(4, dtype=torch.float64)).step(x, batch)
    with pytest.raises(ValueError, match="positions"):
        _layer(None).step(x, batch, positions=torch.zeros(3, dtype=torch.int32))


def test_weights_cover_the_page_table():
    batch = SimpleNamespace(arrays=(torch.zeros(3, 5, dtype=torch.int32),))
    weights = _layer(None).alloc_weights(batch)
    assert weights.shape == (3, 2, 80) and weights.dtype == torch.float32 and (weights == 0).all()


def test_eviction_cuts_the_batchs_own_lengths(monkeypatch):
    given = {}
    monkeypatch.setattr(nv, "nvfp4_kv_evict", lambda *a, **kw: given.update(args=a, kw=kw))
    layer, past = _layer(None), torch.tensor([9, 3], dtype=torch.int32)
    batch = SimpleNamespace(arrays=(None, None, past))
    layer.evict(batch, "weights", 5, "kept", first=1, recent=2)
    assert given["args"][:5] == (layer.cache, batch, "weights", 5, "kept") and given["args"][5] is past
    assert given["kw"] == {"first": 1, "recent": 2}
