"""Host-side checks of the key/value cache's entry points that need no GPU: sizes,
and the refusals, which come before anything touches the device; and the oracle's
own pins."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import kv as okv

OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE = 0, -1, -2, -3, -4
A = 1 << 20          # an address that is aligned and never followed


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def cache(**kw):
    d = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, k_format=8, v_format=4, pages=4, page_tokens=64, heads=2,
             head_dim=128)
    d.update(kw)
    return nv._KvCache(*d.values())


def batch(**kw):
    d = dict(page_table=A, offsets=A, past=A, tokens=6, seqs=2, table_width=2, max_new=3, max_context=100)
    d.update(kw)
    return nv._KvBatch(*d.values())


def append(lib, c, b, dtype=0, k=A, ks=256, v=A, vs=256):
    return lib.nvfp4_kv_append(ctypes.byref(c), ctypes.byref(b), dtype, k, ks, v, vs, None)


def attention(lib, c, b, q=A, qs=1024, q_heads=8, scale=0.1, window=0, tree=None, out=A, os_=1024, lse=A, ws=None, nbytes=0):
    return lib.nvfp4_kv_attention(ctypes.byref(c), ctypes.byref(b), q, qs, q_heads, scale, window, tree, out, os_, lse,
                                  ws, nbytes, None)


def test_sizes():
    assert nv.nvfp4_kv_code_bytes(8, 3, 64, 5, 128) == 3 * 64 * 5 * 128
    assert nv.nvfp4_kv_code_bytes(4, 3, 64, 5, 128) == 3 * 64 * 5 * 64
    assert nv.nvfp4_kv_scale_bytes(4, 3, 64, 5, 128) == 3 * 64 * 5 * 4
    for bad in ((5, 1, 16, 1, 64), (8, 0, 16, 1, 64), (8, 1, 8, 1, 64), (8, 1, 48, 1, 64), (8, 1, 2048, 1, 64),
                (8, 1, 16, 0, 64), (8, 1, 16, 1, 96), (8, 1, 16, 1, 0), (8, (1 << 30) + 1, 16, 1, 64)):
        assert nv.nvfp4_kv_code_bytes(*bad) == 0 and nv.nvfp4_kv_scale_bytes(*bad) == 0, bad
    assert nv.nvfp4_kv_code_bytes(8, 1 << 24, 1024, 8, 256) == (1 << 24) * 1024 * 8 * 256      # past 32 bits


SHARED = [
    (dict(k_codes=0), {}, EINVAL), (dict(v_scales=0), {}, EINVAL), (dict(k_format=5), {}, ESHAPE),
    (dict(v_format=0), {}, ESHAPE), (dict(pages=0), {}, ESHAPE), (dict(page_tokens=24), {}, ESHAPE),
    (dict(page_tokens=8), {}, ESHAPE), (dict(heads=0), {}, ESHAPE), (dict(head_dim=192), {}, ESHAPE),
    (dict(k_codes=A + 8), {}, EALIGN), (dict(v_scales=A + 4), {}, EALIGN),
    ({}, dict(page_table=0), EINVAL), ({}, dict(offsets=0), EINVAL), ({}, dict(past=0), EINVAL),
    ({}, dict(seqs=0), EINVAL), ({}, dict(table_width=0), EINVAL), ({}, dict(tokens=-1), EINVAL),
    ({}, dict(max_new=-1), EINVAL), ({}, dict(max_context=-1), EINVAL),
    ({}, dict(table_width=1 << 25), ESHAPE), ({}, dict(tokens=1 << 30), ESHAPE), ({}, dict(offsets=A + 2), EALIGN),
]


@pytest.mark.parametrize("c,b,status", SHARED)
def test_cache_and_batch_refusals(lib, c, b, status):
    assert append(lib, cache(**c), batch(**b)) == status
    assert attention(lib, cache(**c), batch(**b)) == status
    assert lib.nvfp4_kv_attention_workspace_bytes(ctypes.byref(cache(**c)), ctypes.byref(batch(**b)), 8) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(dtype=2), EINVAL), (dict(ks=255), ESHAPE),
    (dict(vs=1 << 41), ESHAPE), (dict(k=A + 8), EALIGN), (dict(ks=260), EALIGN), (dict(dtype=1, vs=258), EALIGN)])
def test_append_refusals(lib, kw, status):
    assert append(lib, cache(), batch(), **kw) == status


def test_read_refusals(lib):
    c, b = cache(), batch()
    assert lib.nvfp4_kv_read(ctypes.byref(c), ctypes.byref(b), 0, None, 0, None, 0, None) == EINVAL
    assert lib.nvfp4_kv_read(ctypes.byref(c), ctypes.byref(b), 0, None, 0, A, 8, None) == ESHAPE
    assert lib.nvfp4_kv_read(None, ctypes.byref(b), 0, A, 256, A, 256, None) == EINVAL
    assert lib.nvfp4_kv_read(ctypes.byref(c), None, 0, A, 256, A, 256, None) == EINVAL


@pytest.mark.parametrize("kw,b,status", [
    (dict(q=None), {}, EINVAL), (dict(out=None), {}, EINVAL), (dict(scale=0.0), {}, EINVAL),
    (dict(scale=-1.0), {}, EINVAL), (dict(scale=float("nan")), {}, EINVAL), (dict(scale=float("inf")), {}, EINVAL),
    (dict(window=-1), {}, EINVAL), (dict(tree=A, window=5), {}, EINVAL), (dict(tree=A), dict(max_new=65), EINVAL),
    (dict(q_heads=0), {}, ESHAPE), (dict(q_heads=7), {}, ESHAPE), (dict(qs=1023), {}, ESHAPE),
    (dict(os_=512), {}, ESHAPE), (dict(q=A + 2), {}, EALIGN), (dict(out=A + 8), {}, EALIGN),
    (dict(qs=1028), {}, EALIGN), (dict(lse=A + 2), {}, EALIGN), (dict(tree=A + 4), {}, EALIGN),
    (dict(), dict(max_context=100000, table_width=2000), EWORKSPACE),
    (dict(ws=A, nbytes=64), dict(max_context=100000, table_width=2000), EWORKSPACE),
    (dict(ws=A + 8, nbytes=1 << 40), dict(max_context=100000, table_width=2000), EALIGN)])
def test_attention_refusals(lib, kw, b, status):
    assert attention(lib, cache(), batch(**b), **kw) == status


def test_nothing_to_do_is_no_error(lib):
    assert append(lib, cache(), batch(tokens=0)) == OK
    assert attention(lib, cache(), batch(tokens=0)) == OK


def test_workspace_grows_with_the_batch_and_not_past_need(lib):
    size = lambda **kw: lib.nvfp4_kv_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch(**kw)), 8)
    long = dict(max_context=100000, table_width=2000)
    assert size(max_context=1) == 0                                  # whole tiles, nothing to join
    assert size(**long) > 0
    assert size(tokens=600, max_new=300, **long) > size(**long)
    assert size(tokens=1300, max_new=700, **long) > size(**long)     # both kernels' parts


def test_binding_refuses_before_the_library():
    t = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        nv.KvCache(t, t, t, t, 8, 8, 16, 1, 64)                      # too small
    with pytest.raises(nv.NVFP4Error):
        nv.KvCache(t, t, t, t, 8, 8, 17, 1, 64)
    big = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        nv.KvCache(big, big, big, big, 8, 8, 16, 1, 64)              # not on a GPU
    with pytest.raises(ValueError):
        nv.KvBatch(torch.zeros(4, dtype=torch.int32), None, None, 1, 1, 1)
    with pytest.raises(TypeError):
        nv.nvfp4_kv_append(None, None, big, big)
    with pytest.raises(nv.NVFP4Error):
        nv.alloc_kv_cache(0, 16, 1, 64)


def test_oracle_code_values():
    e4m3 = okv.code_values(okv.MXFP8)
    assert e4m3[0] == 0 and e4m3[1] == 2.0 ** -9 and e4m3[8] == 2.0 ** -6 and e4m3[56] == 1 and e4m3[126] == 448
    assert np.isnan(e4m3[127]) and np.isnan(e4m3[255]) and e4m3[128 + 56] == -1
    assert list(okv.code_values(okv.MXFP4)) == [0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6]


@pytest.mark.parametrize("fmt", [4, 8])
def test_oracle_quantises_to_the_nearest_value(fmt):
    """By brute force over every code."""
    rng = np.random.default_rng(fmt)
    x = rng.standard_normal((40, 64)) * np.exp2(rng.integers(-12, 12, (40, 1)))
    codes, scales = okv.quantise(x, fmt)
    amax = np.abs(x.reshape(40, 2, 32)).max(-1)
    unit = np.exp2(scales.astype(float) - 127)
    if fmt == 8:
        assert (amax <= 448 * unit).all() and (amax > 448 * unit / 2).all()
    else:
        assert (amax < 8 * unit).all() and (amax >= 4 * unit).all()
    grid = okv.code_values(fmt)
    grid = grid[np.isfinite(grid)]
    y = x.reshape(40, 2, 32) / unit[..., None]
    best = np.abs(grid - np.clip(y, -grid.max(), grid.max())[..., None]).min(-1)
    got = np.abs(okv.code_values(fmt)[codes].reshape(40, 2, 32) - np.clip(y, -grid.max(), grid.max()))
    assert np.array_equal(got, best)


@pytest.mark.parametrize("kind", [okv.Keys, okv.Values])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("fmt", [4, 8])
def test_oracle_layout_is_a_permutation(kind, dim, fmt):
    side = kind(fmt, 1, 16, 1, dim)
    at = np.concatenate([side._code_bytes(r) for r in range(16)])
    assert sorted(at) == list(range(16 * dim * fmt // 8))
    at = np.concatenate([side._scale_bytes(r) for r in range(16)])
    assert sorted(at) == list(range(16 * dim // 32))


def test_oracle_attention_closed_forms():
    """One key: its value.  Equal keys: the mean.  A key far above the rest: its value."""
    keys, values = okv.Keys(8, 2, 16, 1, 64), okv.Values(8, 2, 16, 1, 64)
    table, off, past = np.array([[1, 0]]), np.array([0, 4]), np.array([0])
    k, v = np.zeros((4, 1, 64)), np.arange(4.0)[:, None, None] * np.ones((4, 1, 64))
    k[2] = 8.0
    okv.append(keys, table, off, past, k)
    okv.append(values, table, off, past, v)
    q = np.ones((4, 1, 64))
    out, lse, spread, zmax = okv.attention(keys, values, table, off, past, q, 1.0)
    assert np.allclose(out[0], 0) and np.allclose(out[1], 0.5) and np.allclose(out[2], 2) and np.allclose(out[3], 2)
    assert np.allclose(lse[:, 0], [0, np.log(2), 512, 512]) and zmax[3, 0] == 512 and np.array_equal(out, spread)
