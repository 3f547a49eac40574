"""Layers of one model share a batch, and with it the lengths that their cuts start from."""
from types import SimpleNamespace

import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from tests.test_attention_layer_evict_host import _layer


def test_a_cut_leaves_the_shared_lengths_alone(monkeypatch):
    given = []
    monkeypatch.setattr(nv, "nvfp4_kv_evict", lambda *a, **kw: given.append((a, kw)))
    past, left = torch.tensor([9, 3], dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    batch = SimpleNamespace(arrays=(None, None, past))
    _layer(None).evict(batch, "weights", 5, "kept", first=1, recent=2, left=left)
    _layer(None).evict(batch, "weights", 5, "kept")
    assert given[0][0][5] is left and given[0][1] == {"first": 1, "recent": 2} and given[1][0][5] is past
