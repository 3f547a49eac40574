"""nvfp4_kv_append and nvfp4_kv_read: the bytes of the planes and the values read
back, exactly the oracle's."""
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


def _append_case(rng, new, past, heads, dim, k_fmt, v_fmt, page, f32, pad=16, table=None, pages=None, mangle=None):
    """Append into planes of a known fill, strided inputs; returns what is compared."""
    if table is None:
        table, pages = K.page_table(rng, new, past, page)
    offsets, past = K.lengths(new, past)
    tokens = int(offsets[-1])
    keys = okv.Keys(k_fmt, pages, page, heads, dim, fill=0xA5)
    values = okv.Values(v_fmt, pages, page, heads, dim, fill=0x5A)
    cache, batch = K.cache_gpu(keys, values, page), K.batch_gpu(table, offsets, past)
    wide = rng.standard_normal((tokens, 2 * heads * dim + pad)) * np.exp2(rng.integers(-20, 20, (tokens, 1)))
    if mangle:
        mangle(wide)
    dtype = torch.float32 if f32 else torch.bfloat16
    wide = K.to_gpu(wide, dtype)
    k = wide[:, :heads * dim].unflatten(1, (heads, dim))
    v = wide[:, heads * dim + pad:].unflatten(1, (heads, dim))
    nv.nvfp4_kv_append(cache, batch, k, v)
    okv.append(keys, table, offsets, past, k.double().cpu().numpy())
    okv.append(values, table, offsets, past, v.double().cpu().numpy())
    return cache, batch, table, offsets, past, keys, values, tokens


def _same_planes(cache, keys, values):
    for got, want in zip(cache.planes, (keys.codes, keys.scales, values.codes, values.scales)):
        assert np.array_equal(got.cpu().numpy(), want.reshape(-1))


def _want(side, table, offsets, past, tokens):
    want = np.zeros((tokens, side.heads, side.dim))
    for s in range(len(past)):
        n = offsets[s + 1] - offsets[s]
        want[offsets[s]:offsets[s + 1]] = okv.held(side, table, s, past[s] + n)[0][past[s]:]
    return want


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("k_fmt,v_fmt", [(8, 8), (4, 8), (8, 4), (4, 4)])
@pytest.mark.parametrize("page,heads,f32", [(16, 3, False), (64, 1, True), (32, 5, True)])
def test_append_and_read(dim, k_fmt, v_fmt, page, heads, f32):
    G.note("kv append D=%d %d/%d page %d heads %d f32 %d" % (dim, k_fmt, v_fmt, page, heads, f32))
    rng = np.random.default_rng(dim + page + 7 * k_fmt + v_fmt)
    new, past = [1, 0, 37, 5, 16, 0], [0, 9, 14, 63, 16, 0]
    cache, batch, table, offsets, past, keys, values, tokens = _append_case(
        rng, new, past, heads, dim, k_fmt, v_fmt, page, f32)
    _same_planes(cache, keys, values)
    for dtype in (torch.bfloat16, torch.float32):
        kout = torch.full((tokens, heads, dim), float("nan"), dtype=dtype, device=K.DEV)
        vout = torch.full_like(kout, float("nan"))
        nv.nvfp4_kv_read(cache, batch, kout, vout)
        assert np.array_equal(kout.double().cpu().numpy(), _want(keys, table, offsets, past, tokens))
        assert np.array_equal(vout.double().cpu().numpy(), _want(values, table, offsets, past, tokens))


@pytest.mark.parametrize("seqs", [64, 65, 130])
def test_many_sequences_with_empty_ones(seqs):
    G.note("kv append, %d sequences" % seqs)
    rng = np.random.default_rng(seqs)
    new, past = rng.integers(0, 3, seqs), rng.integers(0, 40, seqs)
    new[[0, -1]] = 0
    new[seqs // 2] = 2
    cache, *_, keys, values, _ = _append_case(rng, new, past, 2, 64, 8, 4, 16, False)
    _same_planes(cache, keys, values)


def test_tokens_without_a_page_are_dropped_and_read_as_zeros():
    G.note("kv append, missing pages")
    rng = np.random.default_rng(5)
    table = np.array([[2, -1, 0], [7, 1 << 30, 3]], np.int32)       # 6 pages: 7 and 2^30 name none
    new, past = [40, 60], [6, 1]                                    # and the second runs past its table
    cache, batch, table, offsets, past, keys, values, tokens = _append_case(
        rng, new, past, 2, 128, 8, 4, 16, False, table=table, pages=6)
    _same_planes(cache, keys, values)
    out = torch.full((tokens, 2, 128), float("nan"), device=K.DEV)
    nv.nvfp4_kv_read(cache, batch, V=out)
    want = _want(values, table, offsets, past, tokens)
    assert (want[12:20] == 0).all() and np.array_equal(out.double().cpu().numpy(), want)


def test_rows_past_the_last_offset_are_left_alone():
    G.note("kv read, rows of no sequence")
    rng = np.random.default_rng(6)
    table, keys, values = K.filled(rng, [3], [4], 2, 64, 8, 8, 16)
    cache = K.cache_gpu(keys, values, 16)
    batch = K.batch_gpu(table, np.array([0, 3]), np.array([4]), tokens=9)
    out = torch.full((9, 2, 64), 7.0, device=K.DEV)
    nv.nvfp4_kv_read(cache, batch, K=out)
    assert (out[3:] == 7).all() and np.array_equal(out[:3].double().cpu().numpy(), okv.held(keys, table, 0, 7)[0][4:])
    before = [p.clone() for p in cache.planes]
    nv.nvfp4_kv_append(cache, batch, out, out)
    again = [p.clone() for p in cache.planes]
    out[3:] = 1.0
    nv.nvfp4_kv_append(cache, batch, out, out)
    assert all(torch.equal(a, b) for a, b in zip(again, cache.planes))
    assert not torch.equal(before[0], again[0])


def test_block_edges():
    """Zeros of both signs, the largest magnitude at, just under and just over a
    step of the scale, ties, subnormals, the largest floats."""
    G.note("kv append, block edges")

    def mangle(x):
        x[0] = 0.0
        x[1] = -0.0
        for i, top in enumerate([448.0, np.float32(448.00003), np.nextafter(np.float32(448), np.float32(0)), 6.0, 7.99,
                                 8.0, 3.0e38, 2.0 ** -126, 2.0 ** -140, 2.0 ** -149]):
            x[2 + i] = rng.uniform(-1, 1, x.shape[1]) * top
            x[2 + i, ::32] = top
        # every midpoint between two codes, at a block whose unit is 1
        for row, fmt, amax in ((12, 8, 448), (13, 4, 6)):
            mags = okv.code_values(fmt)[:8 if fmt == 4 else 127]
            mid = (mags[1:] + mags[:-1]) / 2
            x[row] = np.resize(np.concatenate((mid, -mid)), x.shape[1])
            x[row, ::32] = amax

    rng = np.random.default_rng(8)
    for k_fmt, v_fmt in ((8, 4), (4, 8)):
        rng = np.random.default_rng(8)
        cache, *_, keys, values, _ = _append_case(rng, [14], [3], 2, 256, k_fmt, v_fmt, 16, True, mangle=mangle)
        _same_planes(cache, keys, values)


def test_infinities_and_nans_mark_their_block_only():
    G.note("kv append, not finite")

    def mangle(x):
        x[1, 5], x[2, 40], x[3, 64 + 3], x[3, 100] = np.inf, -np.inf, np.nan, np.nan

    rng = np.random.default_rng(9)
    cache, batch, table, offsets, past, keys, values, tokens = _append_case(
        rng, [5], [2], 1, 128, 8, 4, 16, True, pad=0, mangle=mangle)
    _same_planes(cache, keys, values)
    out = torch.empty(tokens, 1, 128, dtype=torch.bfloat16, device=K.DEV)
    nv.nvfp4_kv_read(cache, batch, K=out)
    nan = torch.isnan(out[:, 0]).cpu().numpy().reshape(5, 4, 32)
    want = np.zeros((5, 4), bool)
    want[1, 0] = want[2, 1] = want[3, 2] = want[3, 3] = True
    assert np.array_equal(nan.all(-1), want) and np.array_equal(nan.any(-1), want)


def test_mxfp4_codes_are_mxfp4_quantize_s():
    G.note("kv append against mxfp4_quantize")
    rng = np.random.default_rng(10)
    W = K.to_gpu(rng.standard_normal((16, 128)), torch.float32)
    codes = torch.empty(16, 64, dtype=torch.uint8, device=K.DEV)
    scales = torch.empty(16, 4, dtype=torch.uint8, device=K.DEV)
    nv.mxfp4_quantize(W, 16, 128, 1.0, codes, scales)
    cache = nv.alloc_kv_cache(1, 16, 1, 128, nv.NVFP4_KV_MXFP4, nv.NVFP4_KV_MXFP4, device=K.DEV)
    batch = K.batch_gpu(np.zeros((1, 1)), np.array([0, 16]), np.array([0]))
    nv.nvfp4_kv_append(cache, batch, W[:, None], W[:, None])
    # one unit: pieces of 16 bytes
    assert torch.equal(cache.planes[0].view(4, 16, 16).permute(1, 0, 2).reshape(16, 64), codes)
    assert torch.equal(cache.planes[1].view(16, 4), scales)


def test_planes_past_4_gib():
    """Pages whose byte offsets pass 32 bits."""
    G.note("kv append, a pool of more than 4 GiB")
    heads, dim, page = 8, 256, 128
    pages = (1 << 32) // (heads * dim * page) + 3
    cache = nv.alloc_kv_cache(pages, page, heads, dim, device=K.DEV)
    new, past = [21], [page - 10]
    table = np.array([[pages - 1, 1]], np.int32)
    offsets, past = K.lengths(new, past)
    batch = K.batch_gpu(table, offsets, past)
    rng = np.random.default_rng(11)
    x = K.to_gpu(rng.standard_normal((21, heads, dim)), torch.float32)
    nv.nvfp4_kv_append(cache, batch, x, 2 * x)
    small, pages2 = nv.alloc_kv_cache(2, page, heads, dim, device=K.DEV), np.array([[0, 1]], np.int32)
    nv.nvfp4_kv_append(small, K.batch_gpu(pages2, offsets, past), x, 2 * x)
    a, b = torch.empty_like(x), torch.empty_like(x)
    nv.nvfp4_kv_read(cache, batch, a, b)
    c, d = torch.empty_like(x), torch.empty_like(x)
    nv.nvfp4_kv_read(small, K.batch_gpu(pages2, offsets, past), c, d)
    assert torch.equal(a, c) and torch.equal(b, d) and torch.equal(b, 2 * a)
    assert np.array_equal(a.double().cpu().numpy(), okv.dequantise(*okv.quantise(x.double().cpu().numpy(), 8), 8))
    # and attention over them
    q = K.to_gpu(rng.standard_normal((21, heads, dim)), torch.bfloat16)
    big, _ = K.attend(cache, batch, q, 0.0625, heads)
    # positions before the appended ones hold whatever the pool held: compare a window of the new tokens only
    win, _ = K.attend(cache, batch, q, 0.0625, heads, window=1)
    win2, _ = K.attend(small, K.batch_gpu(pages2, offsets, past), q, 0.0625, heads, window=1)
    assert torch.equal(win, win2) and big.shape == win.shape
