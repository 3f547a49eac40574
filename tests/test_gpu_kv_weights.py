"""The attention that cached keys receive, gathered on the GPU, against the fp64 oracle,
whose bound of the error is derived beside it."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import evict as oev
from oracle import kv as okv
from tests import _gpu as G
from tests import _kv as K

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


def _words(tree):
    return torch.tensor([int(w) - (1 << 64) if int(w) >> 63 else int(w) for w in tree], dtype=torch.int64, device=G.DEV)


def _tree(rng, new):
    words = []
    for n in new:
        own = []
        for i in range(n):
            own.append((own[rng.integers(i)] if i else 0) | 1 << i)
        words += own
    return words


def _run(rng, table, keys, values, new, past, q_heads, page, decay=1.0, window=0, tree=None, bounds=(None, None),
         scale=None, spoil=None, rows=0):
    """One call against the oracle: q in rows of a wider stride, `rows` more than the
    sequences have; weights hold NaN wherever they must not be read."""
    offsets, past = K.lengths(new, past)
    tokens, dim, heads = int(offsets[-1]) + rows, keys.dim, keys.heads
    scale = float(np.float32(dim ** -0.5 if scale is None else scale))
    q = K.bf16(1.5 * rng.standard_normal((tokens, q_heads, dim)))
    with np.errstate(invalid="ignore"):
        _, lse, _, _ = okv.attention(keys, values, table, offsets, past, q, scale, window, tree)
    lse = lse.astype(np.float32)
    if spoil is not None:
        spoil(q, lse)
    width = table.shape[1] * page + 5
    old = rng.random((len(past), heads, width)).astype(np.float32) * 4
    for s in range(len(past)):
        old[s, :, past[s]:past[s] + new[s]] = np.nan
    if decay == 0:
        old[:] = np.nan
    with np.errstate(invalid="ignore"):
        ref, bound = oev.gather(keys, table, offsets, past, q, scale, lse.astype(np.float64), old.astype(np.float64),
                                float(np.float32(decay)), window, tree)
    wide = torch.full((tokens, (q_heads + 1) * dim), float("nan"), dtype=torch.bfloat16, device=G.DEV)
    qs = wide[:, :q_heads * dim].unflatten(1, (q_heads, dim))
    qs.copy_(K.to_gpu(q, torch.bfloat16))
    w = torch.from_numpy(old.copy()).to(G.DEV)
    batch = K.batch_gpu(table, offsets, past, tokens, *bounds)
    nv.nvfp4_kv_weights(K.cache_gpu(keys, values, page), batch, qs, scale, torch.from_numpy(lse).to(G.DEV), w,
                        decay=decay, window=window, tree=None if tree is None else _words(tree))
    got = w.double().cpu().numpy()
    touched = np.zeros(old.shape, bool)
    for s in range(len(past)):
        if new[s]:
            touched[s, :, :min(past[s] + new[s], table.shape[1] * page)] = True
    # exp2 gives 0 below fp32's normal numbers: at most 2^-126 for each row
    tol = UNIT * bound + 2.0 ** -126 * (tokens * q_heads // heads)
    with np.errstate(invalid="ignore"):
        same = np.where(touched, np.abs(got - ref) <= tol, (got == old) | (np.isnan(got) & np.isnan(old)))
    assert same.all(), "%d of %d weights off, first at %s: %r for %r within %r" % (
        (~same).sum(), same.size, np.argwhere(~same)[0], got[~same][0], ref[~same][0], tol[~same][0])
    return got


BATCHES = [
    ((1,), (0,)), ((1,), (1,)), ((1,), (37,)), ((1, 1, 1), (5, 200, 31)), ((8,), (130,)), ((3, 0, 17), (0, 9, 40)),
    ((70,), (0,)), ((33, 1, 100), (20, 77, 3)), ((150,), (90,))]


@pytest.mark.parametrize("k_fmt", [4, 8])
@pytest.mark.parametrize("dim,heads,q_heads,page", [(64, 2, 2, 16), (128, 2, 10, 32), (256, 1, 7, 64), (64, 1, 40, 128)])
@pytest.mark.parametrize("new,past", BATCHES)
def test_against_the_oracle(new, past, dim, heads, q_heads, page, k_fmt):
    rng = np.random.default_rng(sum(new) + sum(past) + dim)
    table, keys, values = K.filled(rng, new, past, heads, dim, k_fmt, 8, page)
    G.note("weights %s after %s, %d/%d heads of %d, %d bits" % (new, past, q_heads, heads, dim, k_fmt))
    for decay in (1.0, 0.7, 0.0):
        _run(rng, table, keys, values, new, past, q_heads, page, decay=decay)


@pytest.mark.parametrize("context", [None, 40000, 200000])
@pytest.mark.parametrize("dim,heads,q_heads,k_fmt", [(64, 2, 6, 8), (128, 1, 5, 4), (128, 2, 14, 8), (256, 1, 3, 8), (64, 1, 64, 4)])
@pytest.mark.parametrize("new,past,window", [
    ((64,), (0,), 0), ((96, 96), (130, 5), 0), ((333,), (70,), 0), ((500, 400), (0, 33), 0), ((256,), (400,), 90),
    ((289,), (1,), 33), ((64, 64, 64), (0, 1, 200), 1)])
def test_tiles_of_a_heads_tokens(new, past, window, dim, heads, q_heads, k_fmt, context):
    """Sequences whose tokens fill tiles of 32, at the three ways of sharing keys and rows
    among waves that the bound of the context picks."""
    rng = np.random.default_rng(sum(new) + dim + window)
    table, keys, values = K.filled(rng, new, past, heads, dim, k_fmt, 8, 32)
    G.note("weights of tiles, %s after %s, %d/%d heads of %d, window %d" % (new, past, q_heads, heads, dim, window))

    def spoil(q, lse):
        lse[[0, 31, 32, sum(new) - 1], [0, q_heads - 1, 1, 0]] = np.nan, np.inf, -np.inf, np.nan

    _run(rng, table, keys, values, new, past, q_heads, 32, decay=0.6, window=window, bounds=(None, context), spoil=spoil)


@pytest.mark.parametrize("context", [None, 200000])
def test_a_tree_that_fills_its_tiles(context):
    rng = np.random.default_rng(11)
    new, past = (64, 64), (90, 3)
    table, keys, values = K.filled(rng, new, past, 2, 128, 8, 8, 16)
    G.note("weights of full trees")
    _run(rng, table, keys, values, new, past, 10, 16, tree=_tree(rng, new), bounds=(None, context))
    # fewer tokens than the bounds say, in rows of no sequence
    _run(rng, table, keys, values, (64, 32), past, 10, 16, bounds=(64, context), rows=32)


@pytest.mark.parametrize("window", [1, 7, 50, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("new,past", [((1,), (90,)), ((40, 3), (60, 0)), ((130,), (20,))])
def test_windows(new, past, window):
    rng = np.random.default_rng(window % 1000 + sum(new))
    table, keys, values = K.filled(rng, new, past, 2, 64, 8, 8, 16)
    G.note("weights of a window of %d, %s after %s" % (window, new, past))
    _run(rng, table, keys, values, new, past, 6, 16, decay=0.5, window=window)


@pytest.mark.parametrize("new,past", [((8,), (100,)), ((1, 40, 64), (0, 33, 5)), ((64,), (0,)), ((20, 0, 7), (31, 3, 64))])
def test_trees(new, past):
    rng = np.random.default_rng(sum(new))
    table, keys, values = K.filled(rng, new, past, 2, 128, 4, 4, 32)
    tree = _tree(rng, new)
    G.note("weights of trees, %s after %s" % (new, past))
    _run(rng, table, keys, values, new, past, 8, 32, tree=tree)
    # words that name tokens that are not there, none at all, and all
    tree = [int(w) for w in rng.integers(0, 1 << 63, sum(new), dtype=np.int64)]
    tree[0] = 0
    tree[-1] = (1 << 64) - 1
    _run(rng, table, keys, values, new, past, 8, 32, tree=tree)


@pytest.mark.parametrize("bounds", [(1, 1), (1, 100000), (5000, 1), (0, 0), (64, 2 ** 31 - 1), (2 ** 31 - 1, 40)])
def test_bounds_never_change_the_result(bounds):
    rng = np.random.default_rng(2)
    new, past = (40, 1, 9), (300, 200, 0)
    table, keys, values = K.filled(rng, new, past, 2, 64, 8, 8, 16)
    G.note("weights with bounds %s" % (bounds,))
    _run(np.random.default_rng(3), table, keys, values, new, past, 8, 16, decay=0.9, bounds=bounds)


def test_pages_that_are_not_there():
    """Keys without a page gather nothing, their old weight still fades; positions past the
    table have no place."""
    rng = np.random.default_rng(4)
    new, past = (3, 50), (100, 60)
    table, keys, values = K.filled(rng, new, past, 2, 128, 8, 8, 16)
    table[0, 1], table[0, 4], table[1, 0], table[1, 5] = -1, len(keys.codes), 2 ** 31 - 1, -2 ** 31
    G.note("weights: pages that are not there")
    got = _run(rng, table, keys, values, new, past, 4, 16, decay=0.5)
    assert (got[1, :, 80:96] == 0).all()
    _run(rng, np.ascontiguousarray(table[:, :6]), keys, values, new, past, 4, 16, decay=0.5)


def test_rows_without_a_sum_and_keys_without_a_value():
    """Rows whose log-sum-exp is infinite or NaN add nothing, whatever their queries hold;
    keys that hold a NaN gather nothing and spoil no other."""
    rng = np.random.default_rng(5)
    new, past, page = (40, 2), (70, 9), 16
    for dim in (64, 128, 256):
        for fmt in (4, 8):
            table, keys, values = K.filled(rng, new, past, 2, dim, fmt, 8, page)

            def spoil(q, lse):
                for t, h, v in ((0, 1, np.nan), (3, 0, np.inf), (17, 5, -np.inf), (39, 3, np.nan), (40, 2, np.nan)):
                    lse[t, h] = v
                    q[t, h, rng.integers(dim)] = v

            G.note("weights: spoilt rows and keys, heads of %d, %d bits" % (dim, fmt))
            _run(rng, table, keys, values, new, past, 6, page, spoil=spoil)
            # a key's block of NaN, after the attention's sums were taken without it
            for pos in (0, 33, 75):
                keys.scales[table[0, pos // page], 1, 0, keys._scale_bytes(pos % 16)[-1]] = 0xFF
            _run(rng, table, keys, values, new, past, 6, page,
                 spoil=lambda q, lse: lse.__setitem__(slice(None), np.where(np.isfinite(lse), lse, 5.0)))


def test_rows_of_no_sequence():
    rng = np.random.default_rng(6)
    table, keys, values = K.filled(rng, (5,), (20,), 1, 64, 8, 8, 16)
    _run(rng, table, keys, values, (5,), (20,), 4, 16, rows=40)


def test_the_same_bits_again():
    rng = np.random.default_rng(7)
    new, past = (200, 60), (300, 0)
    table, keys, values = K.filled(rng, new, past, 2, 128, 8, 8, 16)
    a, b = [_run(np.random.default_rng(8), table, keys, values, new, past, 8, 16) for _ in range(2)]
    assert np.array_equal(a, b, equal_nan=True)


@pytest.mark.parametrize("k_fmt", [4, 8])
@pytest.mark.parametrize("new,context", [(1, 131072), (3, 70001), (300, 40000)])
def test_long_contexts_by_closed_forms(new, context, k_fmt):
    """Equal keys: each allowed key of a row gets exp(-lse); with lse the logarithm of a
    power of two, an exact share for each row that sees it.  Keys twice as long are told
    apart."""
    heads, dim, page, group = 2, 64, 256, 4
    width = -(-context // page)
    cache = nv.alloc_kv_cache(width, page, heads, dim, k_fmt, 4)
    table = torch.randperm(width, device=G.DEV).to(torch.int32).view(1, width)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=G.DEV)
    k = torch.zeros(context, heads, dim, device=G.DEV)
    far = [0, 31, 32, 4095, context // 2, context - new - 1]
    k[far] = 1.0
    nv.nvfp4_kv_append(cache, nv.KvBatch(table, ints(0, context), ints(0), context, context, context), k, torch.zeros_like(k))
    q = torch.full((new, heads * group, dim), 1 / 64, dtype=torch.bfloat16, device=G.DEV)
    lse = torch.full((new, heads * group), 10 * float(np.log(2)), device=G.DEV)
    w = torch.zeros(1, heads, width * page, device=G.DEV)
    G.note("weights of %d tokens over %d keys of %d bits" % (new, context, k_fmt))
    nv.nvfp4_kv_weights(cache, nv.KvBatch(table, ints(0, new), ints(context - new), new, new, context), q, 1.0, lse, w)
    pos = np.arange(width * page)
    seen = np.clip(context - np.maximum(pos, context - new), 0, None) * group
    ref = seen * np.where(np.isin(pos, far), np.exp(1.0), 1.0) * np.exp(-lse.double().cpu().numpy()[0, 0])
    off = np.abs(w.double().cpu().numpy() - ref)
    # the sums (a step for each 32 rows, and 16), the exponents of 14 at most and their factors
    assert (off <= ref * UNIT * (new * group / 32 + 16 + 3 * 15 + 8 + 2 * dim)).all()


def test_the_weights_of_a_row_sum_to_one():
    """With the attention's own log-sum-exp: gathered over all keys, one for each row."""
    rng = np.random.default_rng(9)
    new, past, q_heads, page = (64, 1), (500, 1000), 16, 64
    table, keys, values = K.filled(rng, new, past, 4, 128, 8, 8, page)
    offsets, past = K.lengths(new, past)
    cache, batch = K.cache_gpu(keys, values, page), K.batch_gpu(table, offsets, past)
    q = K.to_gpu(rng.standard_normal((65, q_heads, 128)), torch.bfloat16)
    _, lse = K.attend(cache, batch, q, 128 ** -0.5, q_heads)
    w = torch.zeros(2, 4, table.shape[1] * page, device=G.DEV)
    G.note("weights after the attention")
    nv.nvfp4_kv_weights(cache, batch, q, 128 ** -0.5, lse, w)
    total = w.double().sum(-1).cpu().numpy()
    want = np.array(new)[:, None] * (q_heads / 4)
    # the attention's log-sum-exp and this call's exponents each within 2^-17 of such scores
    assert (np.abs(total - want) <= want * 2.0 ** -15).all()


def test_graph_replays_follow_the_lengths():
    """A captured decode step: past moves on between replays, weights gather."""
    rng = np.random.default_rng(10)
    heads, q_heads, dim, page, steps = 2, 8, 128, 16, 4
    new, past = (1, 1), (60, 14)
    table, keys, values = K.filled(rng, (1 + steps, 1 + steps), past, heads, dim, 8, 8, page)
    cache = K.cache_gpu(keys, values, page)
    offsets, start = K.lengths(new, past)
    batch = K.batch_gpu(table, offsets, start, max_context=100)
    q = torch.zeros(2, q_heads, dim, dtype=torch.bfloat16, device=G.DEV)
    lse = torch.zeros(2, q_heads, device=G.DEV)
    w = torch.zeros(2, heads, table.shape[1] * page, device=G.DEV)
    call = lambda: nv.nvfp4_kv_weights(cache, batch, q, dim ** -0.5, lse, w, decay=0.75)
    G.note("weights in a graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        batch.arrays[2].add_(1)
    w.zero_()
    batch.arrays[2].copy_(torch.from_numpy(start))
    ref, off = np.zeros(w.shape), np.zeros(w.shape)
    for i in range(steps):
        x = K.bf16(rng.standard_normal((2, q_heads, dim)))
        _, l, _, _ = okv.attention(keys, values, table, offsets, start + i, x, dim ** -0.5)
        q.copy_(K.to_gpu(x, torch.bfloat16))
        lse.copy_(torch.from_numpy(l.astype(np.float32)))
        graph.replay()
        torch.cuda.synchronize()
        scale = float(np.float32(dim ** -0.5))
        ref, bound = oev.gather(keys, table, offsets, start + i, x, scale, l.astype(np.float32).astype(float), ref, 0.75)
        off = 0.75 * off + UNIT * bound + 1e-37
        got = w.double().cpu().numpy()
        assert (np.abs(got - ref) <= off).all(), i


def test_refusals_of_tensors():
    rng = np.random.default_rng(11)
    table, keys, values = K.filled(rng, (2,), (20,), 2, 64, 8, 8, 16)
    offsets, past = K.lengths((2,), (20,))
    cache, batch = K.cache_gpu(keys, values, 16), K.batch_gpu(table, offsets, past)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=G.DEV)
    lse, w = torch.zeros(2, 4, device=G.DEV), torch.zeros(1, 2, 32, device=G.DEV)
    for bad in (dict(lse=lse[:1]), dict(lse=lse.double()), dict(weights=w[:, :1]), dict(weights=w.cpu()),
                dict(weights=w.transpose(1, 2)), dict(Q=q.float()), dict(window=1 << 31),
                dict(tree=torch.zeros(2, device=G.DEV))):
        kw = dict(dict(Q=q, scale=0.1, lse=lse, weights=w), **bad)
        with pytest.raises(ValueError):
            nv.nvfp4_kv_weights(cache, batch, **kw)
    with pytest.raises(nv.NVFP4Error) as err:
        nv.nvfp4_kv_weights(cache, batch, q, 0.1, lse, w[..., :31].contiguous())
    assert err.value.status == -2
