"""nvfp4_kv_append and nvfp4_kv_read at the edges of what a step may hold."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from tests import _gpu as G
from tests import _kv as K
from tests.test_gpu_kv_cache import _want

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


@pytest.mark.parametrize("dim,heads,k_fmt,v_fmt,new", [
    (256, 4, 8, 4, [701, 0, 1, 3, 333, 0, 0, 1011, 4]),          # 2053 rows of 64 threads' work
    (128, 5, 4, 8, [0, 5, 1, 2, 3001, 2, 275]),
    (64, 3, 8, 8, [10913, 0, 11, 2]),
])
def test_read_of_many_rows(dim, heads, k_fmt, v_fmt, new):
    """Enough rows that a thread of the read takes two of them: pairs whose second row is
    another sequence's, has another page or none, or is the last, alone; pages left
    out from an odd row on; rows of no sequence after them."""
    G.note("kv read, %d rows D=%d" % (sum(new), dim))
    rng = np.random.default_rng(dim)
    page, tokens, spare = 16, sum(new), 6
    past = rng.integers(0, 30, len(new))
    past[np.argmax(new)] = 3
    table, keys, values = K.filled(rng, new, past, heads, dim, k_fmt, v_fmt, page)
    table[np.argmax(new), 5], table[np.argmax(new), 9:11] = -1, len(keys.codes)
    offsets, past = K.lengths(new, past)
    assert tokens * heads * (dim // 16) >= 1 << 17 and (offsets[np.argmax(new)] + 5 * page - 3) % 2
    cache = K.cache_gpu(keys, values, page)
    batch = K.batch_gpu(table, offsets, past, tokens=tokens + spare)
    want = [_want(side, table, offsets, past, tokens) for side in (keys, values)]
    for dtype in (torch.bfloat16, torch.float32):
        wide = torch.full((tokens + spare, 2 * heads * dim + 16), float("nan"), dtype=dtype, device=K.DEV)
        k, v = wide[:, :heads * dim].unflatten(1, (heads, dim)), wide[:, heads * dim + 16:].unflatten(1, (heads, dim))
        nv.nvfp4_kv_read(cache, batch, k, v)
        for got, ref in zip((k, v), want):
            assert np.array_equal(got[:tokens].double().cpu().numpy(), ref)
        assert wide[tokens:].isnan().all() and wide[:, heads * dim:heads * dim + 16].isnan().all()
        alone = torch.full((tokens + spare, heads, dim), float("nan"), dtype=dtype, device=K.DEV)
        nv.nvfp4_kv_read(cache, batch, V=alone)
        assert torch.equal(alone[:tokens], v[:tokens]) and alone[tokens:].isnan().all()
