"""nvfp4_kv_attention against the fp64 oracle, at the sizes and masks where it can
go wrong.  Planes hold NaN codes and NaN scales wherever no token was written."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
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


# The batch's host numbers only shape the launch: the same cases run with bounds that
# are exact, with a context bound far above (the long splits of many rows), and among
# many rows that no sequence has (whole tiles of the kernel for many rows).
@pytest.fixture(params=["exact", "far", "spare"], autouse=True)
def _shape(request, monkeypatch):
    monkeypatch.setattr(K, "shape", request.param)


def _run(rng, new, past, heads, group, dim, k_fmt=8, v_fmt=8, page=16, window=0, tree=None, pad=0, q_scale=1.5,
         edit=None, **bounds):
    table, keys, values = K.filled(rng, new, past, heads, dim, k_fmt, v_fmt, page)
    if edit:
        edit(table, keys, values)
    offsets, past = K.lengths(new, past)
    tokens, q_heads = int(offsets[-1]), heads * group
    wide = K.to_gpu(q_scale * rng.standard_normal((tokens, q_heads * dim + pad)), torch.bfloat16)
    if K.shape == "far":
        bounds = {"max_context": 100000, **bounds}
    if K.shape == "spare":
        wide = torch.cat([wide, wide.new_zeros(400000 // q_heads, wide.shape[1])])
        bounds = {"tokens": wide.shape[0], **bounds}
    q = wide[:, :q_heads * dim].unflatten(1, (q_heads, dim))
    scale = dim ** -0.5
    cache, batch = K.cache_gpu(keys, values, page), K.batch_gpu(table, offsets, past, **bounds)
    kw = {"window": window}
    if tree is not None:
        words = [int(w) - (1 << 64) if int(w) >> 63 else int(w) for w in tree]
        kw["tree"] = torch.tensor(words + [0] * (len(q) - tokens), dtype=torch.int64, device=K.DEV)
    out, lse = K.attend(cache, batch, q, scale, q_heads, **kw)
    assert out[tokens:].isnan().all() and lse[tokens:].isnan().all()     # rows of no sequence are left alone
    q, out, lse = q[:tokens], out[:tokens], lse[:tokens]
    ref = okv.attention(keys, values, table, offsets, past, q.double().cpu().numpy(), scale, window, tree)
    what = "new %s past %s heads %dx%d D %d formats %d/%d page %d window %d" % (
        list(new)[:6], list(past)[:6], heads, group, dim, k_fmt, v_fmt, page, window)
    K.check(out, lse, ref, dim, what)
    q = wide[:, :q_heads * dim].unflatten(1, (q_heads, dim))
    again, lse2 = (t[:tokens] for t in K.attend(cache, batch, q, scale, q_heads, **kw))
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), what + ": another run, other bits"
    assert torch.equal(lse.view(torch.int32), lse2.view(torch.int32))
    return out, lse, ref


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("k_fmt,v_fmt", [(8, 8), (4, 8), (8, 4), (4, 4)])
@pytest.mark.parametrize("new,past,heads,group", [
    ([1], [0], 1, 1),                      # a single key
    ([1], [300], 2, 4),
    ([8], [130], 2, 5),                    # a verify's columns, an odd group
    ([70], [45], 1, 4),                    # a chunk that ends inside a tile
])
def test_formats_and_dims(dim, k_fmt, v_fmt, new, past, heads, group):
    G.note("attention D=%d %d/%d new %s past %s" % (dim, k_fmt, v_fmt, new, past))
    rng = np.random.default_rng(dim + 3 * k_fmt + v_fmt + new[0])
    _run(rng, new, past, heads, group, dim, k_fmt, v_fmt)


@pytest.mark.parametrize("past", [0, 1, 15, 16, 30, 31, 32, 33, 62, 63, 64, 65, 127, 128, 255, 256, 257, 1000])
@pytest.mark.parametrize("page", [16, 128])
def test_one_token_at_every_edge(past, page):
    G.note("attention, one token after %d, pages of %d" % (past, page))
    _run(np.random.default_rng(past), [1], [past], 2, 8, 128, page=page)


@pytest.mark.parametrize("new", [2, 3, 15, 16, 17, 31, 32, 33, 64, 65, 127, 129, 200])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_chunks_from_nothing(new, group):
    G.note("attention, %d tokens from nothing, group %d" % (new, group))
    _run(np.random.default_rng(new), [new], [0], 1, group, 64, 8, 4, page=32)


@pytest.mark.parametrize("group", [1, 7, 16, 17, 48, 128])
def test_groups(group):
    G.note("attention, group %d" % group)
    _run(np.random.default_rng(group), [3, 1, 9], [40, 7, 0], 1, group, 64)


@pytest.mark.parametrize("dim,k_fmt,v_fmt", [(64, 8, 8), (128, 4, 8), (256, 8, 4)])
def test_ragged_batch_with_empty_sequences(dim, k_fmt, v_fmt):
    G.note("attention, ragged D=%d" % dim)
    rng = np.random.default_rng(dim)
    _run(rng, [0, 5, 1, 0, 33, 90, 0], [3, 100, 0, 0, 64, 31, 900], 2, 3, dim, k_fmt, v_fmt, page=64, pad=24)


def test_many_sequences():
    G.note("attention, 70 sequences")
    rng = np.random.default_rng(70)
    _run(rng, rng.integers(0, 3, 70), rng.integers(0, 90, 70), 1, 4, 64, 4, 4)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 100, 5000])
def test_windows(window):
    G.note("attention, window %d" % window)
    rng = np.random.default_rng(window)
    _run(rng, [1, 70, 9], [200, 150, 0], 2, 4, 128, 8, 4, page=16, window=window)


def test_long_context_is_split():
    """Enough keys that several workgroups share a row's, with bounds that say so."""
    G.note("attention, split keys")
    rng = np.random.default_rng(12)
    new, past = [1, 4, 0, 2], [2999, 1500, 10, 0]
    out, lse, ref = _run(rng, new, past, 1, 5, 64, 8, 8, page=64)
    # the bounds only shape the launch: far too large and far too small ones
    rng = np.random.default_rng(12)
    _run(rng, new, past, 1, 5, 64, 8, 8, page=64, max_context=100000, max_new=64)
    rng = np.random.default_rng(12)
    _run(rng, new, past, 1, 5, 64, 8, 8, page=64, max_context=1, max_new=1)


@pytest.mark.parametrize("dim,k_fmt,v_fmt", [(64, 8, 8), (128, 8, 4), (256, 4, 8)])
def test_many_rows_in_splits(dim, k_fmt, v_fmt):
    """A chunk whose keys several workgroups share, beside a short sequence and one
    whose last split has a single key."""
    G.note("attention of a chunk, split keys, D=%d" % dim)
    rng = np.random.default_rng(dim)
    _run(rng, [100, 3, 60], [2600, 900, 837], 1, 5, dim, k_fmt, v_fmt, page=64)


@pytest.mark.parametrize("n", [1, 8, 40, 64])
def test_tree_masks(n):
    G.note("attention, tree of %d" % n)
    rng = np.random.default_rng(n)
    words = []
    for i in range(n):
        words.append((words[rng.integers(i)] if i else 0) | 1 << i)
    words[n // 2] = 0                       # sees the past only
    _run(rng, [n], [77], 2, 4, 128, 4, 4, tree=np.array(words, dtype=object))
    # without a past, a token of no ancestor sees nothing: zeros and -inf
    out, lse, ref = _run(np.random.default_rng(n), [n], [0], 1, 2, 64, tree=np.array(words, dtype=object))
    assert (out[n // 2] == 0).all() and (lse[n // 2] == float("-inf")).all()


def test_missing_pages_are_seen_by_nobody():
    G.note("attention, missing pages")

    def edit(table, keys, values):
        table[0, 1] = -1
        table[0, 4] = len(keys.codes)
        table[1, :] = -1

    rng = np.random.default_rng(13)
    out, lse, ref = _run(rng, [3, 2, 1], [100, 20, 33], 2, 4, 128, edit=edit)
    assert (out[3:5] == 0).all() and (lse[3:5] == float("-inf")).all()


@pytest.mark.parametrize("new,group", [(40, 4), (100, 8)])
def test_nan_in_a_masked_place_stays_there(new, group):
    """A NaN key or value reaches the rows that see its token and no other."""
    G.note("attention, NaN among %d new tokens" % new)

    def edit(table, keys, values):
        for side, pos, block in ((values, 50 + new // 2, 1), (keys, 50 + new - 2, 0), (values, 50 + new - 1, 3)):
            page, at = table[0, pos // 16], pos % 16
            side.scales[page, 0, 0, side._scale_bytes(at)[block]] = 0xFF

    rng = np.random.default_rng(14)
    out, lse, ref = _run(rng, [new], [50], 1, group, 128, edit=edit)
    o = out.float().cpu().numpy()
    assert np.isfinite(o[:new // 2]).all() and np.isnan(o[new // 2, :, 32:64]).all()
    assert np.isfinite(o[new // 2, :, :32]).all() and np.isnan(o[new - 2:]).all()


def test_large_and_tiny_scores():
    """Scores far apart (weights underflow), all equal, and negative throughout."""
    G.note("attention, extreme scores")
    for q_scale in (0.0, 1e-6, 300.0, 3e4):
        _run(np.random.default_rng(15), [2, 20], [90, 5], 1, 4, 128, q_scale=q_scale)


def test_without_lse_and_rows_of_no_sequence():
    G.note("attention, no lse")
    rng = np.random.default_rng(16)
    table, keys, values = K.filled(rng, [3, 2], [40, 0], 2, 64, 8, 8, 16)
    offsets, past = K.lengths([3, 2], [40, 0])
    cache, batch = K.cache_gpu(keys, values, 16), K.batch_gpu(table, offsets, past, tokens=9)
    q = K.to_gpu(rng.standard_normal((9, 4, 64)), torch.bfloat16)
    out, lse = K.attend(cache, batch, q, 0.125, 4)
    assert torch.isnan(out[5:]).all() and torch.isnan(lse[5:]).all()
    out2 = torch.zeros(9, 6, 64, dtype=torch.bfloat16, device=K.DEV)[:, :4]     # strided output
    workspace = torch.empty(max(1, nv.nvfp4_kv_attention_workspace_bytes(cache, batch, 4)), dtype=torch.uint8, device=K.DEV)
    nv.nvfp4_kv_attention(cache, batch, q, 0.125, out2, workspace=workspace)
    assert torch.equal(out2[:5], out[:5]) and (out2[5:] == 0).all()


def test_other_stream_and_graph_follow_the_arrays():
    """On a stream of its own, and captured: replays follow the offsets, lengths and
    table that the arrays hold when they run."""
    G.note("attention, stream and graph")
    rng = np.random.default_rng(17)
    heads, dim, page, width = 2, 128, 16, 40
    cache = nv.alloc_kv_cache(width, page, heads, dim, device=K.DEV)
    for p in cache.planes:
        p.fill_(0xFF)
    table = np.arange(width, dtype=np.int32)[::-1].reshape(1, width).copy()
    keys = okv.Keys(8, width, page, heads, dim, fill=0xFF)
    values = okv.Values(8, width, page, heads, dim, fill=0xFF)
    batch = K.batch_gpu(table, np.array([0, 2]), np.array([0]), max_context=width * page)
    k, v = (torch.empty(2, heads, dim, dtype=torch.bfloat16, device=K.DEV) for _ in range(2))
    q = torch.empty(2, 8, dim, dtype=torch.bfloat16, device=K.DEV)
    out, lse = torch.empty_like(q), torch.empty(2, 8, device=K.DEV)
    need = nv.nvfp4_kv_attention_workspace_bytes(cache, batch, 8)
    workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=K.DEV)
    past = batch.arrays[2]
    side = torch.cuda.Stream()

    def step():
        nv.nvfp4_kv_append(cache, batch, k, v)
        nv.nvfp4_kv_attention(cache, batch, q, dim ** -0.5, out, lse=lse, workspace=workspace)

    def fresh():
        for t in (k, v, q):
            t.copy_(torch.from_numpy(rng.standard_normal(tuple(t.shape))).to(torch.bfloat16))

    def verify(at, what):
        off, pst = np.array([0, 2]), np.array([at])
        okv.append(keys, table, off, pst, k.double().cpu().numpy())
        okv.append(values, table, off, pst, v.double().cpu().numpy())
        ref = okv.attention(keys, values, table, off, pst, q.double().cpu().numpy(), dim ** -0.5)
        K.check(out, lse, ref, dim, what)

    at = 0
    with torch.cuda.stream(side):
        for _ in range(3):
            fresh()
            past.fill_(at)
            step()
            side.synchronize()
            verify(at, "eager at %d" % at)
            at += 2
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(8):
        fresh()
        past.fill_(at)
        graph.replay()
        torch.cuda.synchronize()
        verify(at, "replay at %d" % at)
        at += 2
        if i == 3:                          # an eager pass between replays
            fresh()
            past.fill_(at)
            step()
            torch.cuda.synchronize()
            verify(at, "eager between replays")
            at += 2


def test_a_workspace_that_is_too_small_is_refused():
    rng = np.random.default_rng(18)
    table, keys, values = K.filled(rng, [1], [3000], 1, 64, 8, 8, 64)
    cache, batch = K.cache_gpu(keys, values, 64), K.batch_gpu(table, np.array([0, 1]), np.array([3000]))
    need = nv.nvfp4_kv_attention_workspace_bytes(cache, batch, 4)
    assert need > 0
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=K.DEV)
    for workspace in (None, torch.empty(need - 1, dtype=torch.uint8, device=K.DEV)):
        with pytest.raises(nv.NVFP4Error) as e:
            nv.nvfp4_kv_attention(cache, batch, q, 0.125, torch.empty_like(q), workspace=workspace)
        assert e.value.status == -4
