"""nvfp4_kv_append and nvfp4_kv_read at the edges of what a step may hold."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from tests import _gpu as G
from tests import _kv as K

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


def test_a_step_of_no_tokens():
    """Every call on a batch of no tokens does nothing, and says so by returning."""
    G.note("kv calls of no tokens")
    cache = nv.alloc_kv_cache(3, 16, 2, 64, device=K.DEV)
    for p in cache.planes:
        p.fill_(0x5A)
    batch = K.batch_gpu(np.array([[0, 1], [2, -1]]), np.array([0, 0, 0]), np.array([4, 0]))
    rows = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=K.DEV)
    q = torch.empty(0, 8, 64, dtype=torch.bfloat16, device=K.DEV)
    nv.nvfp4_kv_append(cache, batch, rows, rows)
    nv.nvfp4_kv_read(cache, batch, rows, rows)
    nv.nvfp4_kv_read(cache, batch, V=rows.float())
    nv.nvfp4_kv_attention(cache, batch, q, 0.125, torch.empty_like(q), lse=torch.empty(0, 8, device=K.DEV),
                          workspace=torch.empty(0, dtype=torch.uint8, device=K.DEV))
    nv.nvfp4_kv_attention(cache, batch, q, 0.125, torch.empty_like(q), tree=torch.empty(0, dtype=torch.int64, device=K.DEV))
    torch.cuda.synchronize()
    assert all((p == 0x5A).all() for p in cache.planes)


@pytest.mark.parametrize("value", [1 << 31, (1 << 32) + 5, -(1 << 31) - 1, -(1 << 32) + 5])
def test_numbers_past_32_bits_are_refused(value):
    """The library's arguments are 32-bit: a larger number must not become another one
    (a window of 2^32 + 5 keys one of 5)."""
    G.note("kv calls with %d" % value)
    table, offsets, past = (torch.zeros(s, dtype=torch.int32, device=K.DEV) for s in ((1, 2), (2,), (1,)))
    with pytest.raises(ValueError):
        nv.KvBatch(table, offsets, past, 1, value, 1)
    with pytest.raises(ValueError):
        nv.KvBatch(table, offsets, past, 1, 1, value)
    cache, batch = nv.alloc_kv_cache(2, 16, 1, 64, device=K.DEV), nv.KvBatch(table, offsets, past, 1, 1, 1)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=K.DEV)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_attention(cache, batch, q, 0.125, torch.empty_like(q), window=value)
    with pytest.raises(ValueError):
        nv.nvfp4_kv_attention_workspace_bytes(cache, batch, value)
    planes = [torch.zeros(1 << 12, dtype=torch.uint8, device=K.DEV) for _ in range(4)]
    for at in range(5):
        numbers = [8, 8, 16, 1, 64]
        numbers[at] += value & ~0xFFFFFFFF or 1 << 32
        with pytest.raises((ValueError, nv.NVFP4Error)):
            nv.KvCache(*planes, *numbers)
