"""Eviction from the cache on the GPU, bit for bit against the oracle."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import evict as oev
from oracle import kv as okv
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


def _planes(rng, past, heads, dim, k_fmt, v_fmt, page):
    """Planes of random bytes: eviction moves them, whatever they mean."""
    table, pages = K.page_table(rng, [0] * len(past), past, page)
    sides = okv.Keys(k_fmt, pages, page, heads, dim), okv.Values(v_fmt, pages, page, heads, dim)
    for side in sides:
        side.codes[:] = rng.integers(0, 256, side.codes.shape)
        side.scales[:] = rng.integers(0, 256, side.scales.shape)
    return table, *sides


def _run(table, keys, values, past, weights, page, budget, first, recent, in_place=False):
    past = np.asarray(past, np.int32)
    seqs, heads = len(past), keys.heads
    cache = K.cache_gpu(keys, values, page)
    batch = K.batch_gpu(table, np.zeros(seqs + 1, np.int32), past, tokens=0, max_new=0)
    w = torch.from_numpy(weights.copy()).to(G.DEV)
    out = w if in_place else torch.full_like(w, -77.0)
    kept = torch.full((seqs, heads, budget), -77, dtype=torch.int32, device=G.DEV)
    left = batch.arrays[2] if in_place else torch.full((seqs,), -77, dtype=torch.int32, device=G.DEV)
    nv.nvfp4_kv_evict(cache, batch, w, budget, kept, left, None if in_place else out, first, recent)
    ref_out = weights.copy() if in_place else np.full_like(weights, -77.0)
    ref_kept, ref_left = oev.evict(keys, values, table, past, weights.copy(), ref_out, budget, first, recent)
    assert np.array_equal(kept.cpu().numpy(), ref_kept)
    assert np.array_equal(left.cpu().numpy(), ref_left)
    assert np.array_equal(out.cpu().numpy(), ref_out, equal_nan=True)
    if not in_place:
        assert np.array_equal(w.cpu().numpy(), weights, equal_nan=True)
        assert np.array_equal(batch.arrays[2].cpu().numpy(), past)
    for plane, ref in zip(cache.planes, (keys.codes, keys.scales, values.codes, values.scales)):
        assert np.array_equal(plane.cpu().numpy(), ref.reshape(-1))
    return ref_kept


@pytest.mark.parametrize("k_fmt,v_fmt", [(4, 4), (8, 8), (4, 8), (8, 4)])
@pytest.mark.parametrize("dim,heads,page", [(64, 3, 16), (128, 2, 64), (256, 1, 32)])
@pytest.mark.parametrize("past,budget,first,recent", [
    ((2,), 1, 0, 0), ((50,), 49, 1, 1), ((100, 7, 64, 65), 64, 4, 16), ((300,), 7, 0, 7), ((33, 0, 200), 40, 40, 0),
    ((500, 129), 128, 0, 0)])
def test_against_the_oracle(past, budget, first, recent, dim, heads, page, k_fmt, v_fmt):
    rng = np.random.default_rng(sum(past) + dim)
    table, keys, values = _planes(rng, past, heads, dim, k_fmt, v_fmt, page)
    weights = rng.random((len(past), heads, table.shape[1] * page + 3)).astype(np.float32)
    G.note("evict %s to %d, %d heads of %d, %d/%d bits" % (past, budget, heads, dim, k_fmt, v_fmt))
    state = [a.copy() for a in (keys.codes, keys.scales, values.codes, values.scales)]
    _run(table, keys, values, past, weights, page, budget, first, recent)
    for a, b in zip((keys.codes, keys.scales, values.codes, values.scales), state):
        a[:] = b
    _run(table, keys, values, past, weights, page, budget, first, recent, in_place=True)


@pytest.mark.parametrize("what", ["equal", "few", "zeros", "special", "rising", "falling", "negative", "tiny"])
def test_orders_of_weights(what):
    """Ties, zeros of both signs, infinities and NaN, weights apart by their last bits."""
    rng = np.random.default_rng(1)
    past, page, budget = (1500, 700), 64, 333
    table, keys, values = _planes(rng, past, 2, 64, 4, 4, page)
    w = rng.random((2, 2, table.shape[1] * page)).astype(np.float32)
    if what == "equal":
        w[:] = 0.25
    elif what == "few":
        w = np.round(w * 4).astype(np.float32)
    elif what == "zeros":
        w = np.where(w < 0.9, np.float32(-0.0), np.where(w < 0.95, np.float32(0.0), w))
    elif what == "special":
        w = np.choose(rng.integers(0, 6, w.shape), [w, np.float32(np.nan), np.float32(np.inf), np.float32(-np.inf), -w,
                                                    np.float32(0)]).astype(np.float32)
        w[1, 1] = np.nan
    elif what in ("rising", "falling"):
        w[:] = np.arange(w.shape[-1]) * (1 if what == "rising" else -1)
    elif what == "negative":
        w = -w
    else:
        w = (w.view(np.uint32) % 512 + 0x3F800000).astype(np.uint32).view(np.float32)
    G.note("evict by %s weights" % what)
    for first, recent in ((0, 0), (4, 32)):
        _run(table, keys, values, past, np.ascontiguousarray(w), page, budget, first, recent, in_place=first > 0)


def test_sequences_that_stay():
    """Within the budget, empty, of negative or too many positions, or with a position that
    has no page: nothing moves."""
    rng = np.random.default_rng(2)
    past, page, budget = (100, 100, 30, 0, 100, 100), 16, 40
    table, keys, values = _planes(rng, past, 2, 128, 8, 8, page)
    table[0, 3], table[4, 6] = -1, len(keys.codes)
    past = np.array(past)
    past[3], past[5] = -5, table.shape[1] * page + 1
    weights = rng.random((6, 2, table.shape[1] * page)).astype(np.float32)
    G.note("evict: sequences that stay")
    kept = _run(table, keys, values, past, weights, page, budget, 2, 5)
    assert (kept[[0, 3, 4, 5]] == -1).all() and (kept[1] >= 0).all() and (kept[2, :, :30] == np.arange(30)).all()
    # entries behind the last position do not matter
    table[1, -1:] = -1 if table.shape[1] * page - 100 >= page else table[1, -1:]
    _run(table, keys, values, past, weights, page, budget, 2, 5)


@pytest.mark.parametrize("length,budget", [(20000, 19000), (20000, 5000), (70001, 4096), (8193, 8000), (12000, 3001),
                                           (16384, 140), (16385, 16384)])
def test_long_sequences(length, budget):
    """Many stretches of tokens, and a page at the end that is filled in part."""
    rng = np.random.default_rng(3)
    page = 1024
    table, keys, values = _planes(rng, (length,), 1, 64, 4, 8, page)
    weights = (rng.random((1, 1, table.shape[1] * page)) ** 8).astype(np.float32)
    G.note("evict %d to %d" % (length, budget))
    _run(table, keys, values, (length,), weights, page, budget, 4, 100, in_place=True)


def test_many_sequences():
    rng = np.random.default_rng(4)
    past = rng.integers(0, 120, 70)
    table, keys, values = _planes(rng, past, 3, 64, 8, 4, 16)
    weights = rng.random((70, 3, table.shape[1] * 16)).astype(np.float32)
    G.note("evict of 70 sequences")
    _run(table, keys, values, past, weights, 16, 48, 1, 8)


def test_graph_replays():
    """Captured with left in the batch's past: appended tokens between the replays; each
    replay as the oracle's step, one that finds nothing to cut among them."""
    rng = np.random.default_rng(5)
    heads, dim, page, budget, seqs = 2, 64, 16, 50, 2
    past = np.array([64, 20], np.int32)
    table, keys, values = _planes(rng, (96, 96), heads, dim, 8, 8, page)
    cache = K.cache_gpu(keys, values, page)
    batch = K.batch_gpu(table, np.zeros(3, np.int32), past, tokens=0, max_new=0)
    w = torch.zeros(seqs, heads, 96, device=G.DEV)
    kept = torch.zeros(seqs, heads, budget, dtype=torch.int32, device=G.DEV)
    call = lambda: nv.nvfp4_kv_evict(cache, batch, w, budget, kept, batch.arrays[2], first=2, recent=10)
    G.note("evict in a graph")
    batch.arrays[2].zero_()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        past = past + (i * 9, 14)
        ref = rng.random((seqs, heads, 96)).astype(np.float32)
        w.copy_(torch.from_numpy(ref))
        batch.arrays[2].copy_(torch.from_numpy(past))
        graph.replay()
        torch.cuda.synchronize()
        out = ref.copy()
        ref_kept, past = oev.evict(keys, values, table, past, ref, out, budget, 2, 10)
        past = past.astype(np.int32)
        assert np.array_equal(kept.cpu().numpy(), ref_kept) and np.array_equal(w.cpu().numpy(), out)
        assert np.array_equal(batch.arrays[2].cpu().numpy(), past)
        for plane, r in zip(cache.planes, (keys.codes, keys.scales, values.codes, values.scales)):
            assert np.array_equal(plane.cpu().numpy(), r.reshape(-1)), i


def test_refusals_of_tensors():
    rng = np.random.default_rng(6)
    table, keys, values = _planes(rng, (40,), 2, 64, 8, 8, 16)
    cache = K.cache_gpu(keys, values, 16)
    batch = K.batch_gpu(table, np.zeros(2, np.int32), np.array([40], np.int32), tokens=0, max_new=0)
    w = torch.zeros(1, 2, 48, device=G.DEV)
    kept, left = torch.zeros(1, 2, 20, dtype=torch.int32, device=G.DEV), torch.zeros(1, dtype=torch.int32, device=G.DEV)
    for bad in (dict(kept=kept[:, :1]), dict(kept=kept.long()), dict(left=left.cpu()), dict(weights=w.double()),
                dict(weights_out=w[..., :40].contiguous()), dict(budget=21), dict(budget=1 << 31)):
        kw = dict(dict(weights=w, budget=20, kept=kept, left=left), **bad)
        with pytest.raises(ValueError):
            nv.nvfp4_kv_evict(cache, batch, **kw)
    for kw in (dict(budget=0), dict(first=21), dict(recent=-1)):
        with pytest.raises(nv.NVFP4Error) as err:
            nv.nvfp4_kv_evict(cache, batch, w, kept=kept, left=left, **dict(dict(budget=20), **kw))
        assert err.value.status == -1
