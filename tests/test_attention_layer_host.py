"""The attention layer's own bookkeeping, which needs no GPU: the library's answers
are stood in for."""
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from block_scaled_bit_nvfp4_amd.attention_layer import AttentionLayer


@pytest.fixture
def needs(monkeypatch):
    """A layer without weights, and a function that reserves so many bytes."""
    layer = object.__new__(AttentionLayer)
    layer.q_heads, layer.cache, layer.device = 8, None, torch.device("cpu")
    layer.workspace = torch.empty(0, dtype=torch.uint8)
    layer.retired = []
    monkeypatch.setattr(nv, "nvfp4_kv_attention_workspace_bytes", lambda cache, batch, q_heads: batch)
    return layer, layer.reserve


def test_a_workspace_once_given_out_is_never_freed(needs):
    """A captured step holds its workspace's address: the memory stays the layer's."""
    import weakref
    layer, reserve = needs
    given = []
    for nbytes in (1000, 900, 4000, 1000, 30000, 30001):
        reserve(nbytes)
        assert layer.workspace.numel() >= nbytes
        given.append((weakref.ref(layer.workspace), layer.workspace.data_ptr(), layer.workspace.numel()))
    for ref, at, size in given:
        assert ref() is not None and ref().data_ptr() == at and ref().numel() == size


def test_workspaces_kept_stay_within_twice_the_last(needs):
    """Batches that grow by a little at a time do not pile up memory."""
    layer, reserve = needs
    for nbytes in range(1000, 200000, 500):
        reserve(nbytes)
    assert layer.workspace.numel() < 2 * 200000
    assert sum(w.numel() for w in layer.retired) <= layer.workspace.numel()
