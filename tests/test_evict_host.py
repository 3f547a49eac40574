"""Host-side checks of the gathered weights and of eviction that need no GPU: the
refusals, which come before anything touches the device, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import evict as oev
from oracle import kv as okv
from tests import test_kv_host as H

OK, EINVAL, ESHAPE, EALIGN = 0, -1, -2, -3
A = H.A


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def weigh(lib, c, b, q=A, qs=1024, q_heads=8, scale=0.1, window=0, tree=None, lse=A, decay=1.0, weights=A, width=128):
    return lib.nvfp4_kv_weights(ctypes.byref(c), ctypes.byref(b), q, qs, q_heads, scale, window, tree, lse, decay,
                                weights, width, None)


def evict(lib, c, b, budget=50, first=4, recent=8, weights=A, out=A, width=128, kept=A, left=A):
    return lib.nvfp4_kv_evict(ctypes.byref(c), ctypes.byref(b), budget, first, recent, weights, out, width, kept, left,
                              None)


@pytest.mark.parametrize("c,b,status", H.SHARED)
def test_cache_and_batch_refusals(lib, c, b, status):
    assert weigh(lib, H.cache(**c), H.batch(**b), width=1 << 35) == status
    assert evict(lib, H.cache(**c), H.batch(**b), width=1 << 35) == status


@pytest.mark.parametrize("kw,b,status", [
    (dict(q=None), {}, EINVAL), (dict(lse=None), {}, EINVAL), (dict(weights=None), {}, EINVAL),
    (dict(scale=0.0), {}, EINVAL), (dict(scale=float("nan")), {}, EINVAL), (dict(scale=float("inf")), {}, EINVAL),
    (dict(window=-1), {}, EINVAL), (dict(tree=A, window=5), {}, EINVAL), (dict(tree=A), dict(max_new=65), EINVAL),
    (dict(decay=-0.1), {}, EINVAL), (dict(decay=1.1), {}, EINVAL), (dict(decay=float("nan")), {}, EINVAL),
    (dict(q_heads=0), {}, ESHAPE), (dict(q_heads=7), {}, ESHAPE), (dict(qs=1023), {}, ESHAPE),
    (dict(width=127), {}, ESHAPE), (dict(width=1 << 41), {}, ESHAPE), (dict(q=A + 2), {}, EALIGN),
    (dict(qs=1028), {}, EALIGN), (dict(lse=A + 2), {}, EALIGN), (dict(weights=A + 2), {}, EALIGN),
    (dict(tree=A + 4), {}, EALIGN)])
def test_weights_refusals(lib, kw, b, status):
    assert weigh(lib, H.cache(), H.batch(**b), **kw) == status


@pytest.mark.parametrize("kw,b,status", [
    (dict(weights=None), {}, EINVAL), (dict(out=None), {}, EINVAL), (dict(kept=None), {}, EINVAL),
    (dict(left=None), {}, EINVAL), (dict(budget=0, first=0, recent=0), {}, EINVAL), (dict(first=-1), {}, EINVAL),
    (dict(recent=-1), {}, EINVAL), (dict(first=43), {}, EINVAL), (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), {}, EINVAL),
    (dict(width=127), {}, ESHAPE), (dict(budget=(1 << 28) + 1), {}, ESHAPE), (dict(), dict(seqs=1 << 20), ESHAPE),
    (dict(weights=A + 2), {}, EALIGN), (dict(out=A + 1), {}, EALIGN), (dict(kept=A + 2), {}, EALIGN),
    (dict(left=A + 2), {}, EALIGN)])
def test_evict_refusals(lib, kw, b, status):
    assert evict(lib, H.cache(), H.batch(**b), **kw) == status


def test_no_tokens_is_no_error(lib):
    assert weigh(lib, H.cache(), H.batch(tokens=0), q=None, lse=None, weights=None) == OK


def test_binding_refuses_before_the_library():
    t = torch.zeros(64)
    with pytest.raises(TypeError):
        nv.nvfp4_kv_weights(None, None, t, 1.0, t, t)
    with pytest.raises(TypeError):
        nv.nvfp4_kv_evict(None, None, t, 1, t, t)


def test_oracle_chooses():
    nan = float("nan")
    w = np.array([9, 1, 5, 5, nan, 7, -1, 5, 0, 2.0])
    assert list(oev.choose(w, 10, 10, 0, 0)) == list(range(10)) and list(oev.choose(w, 4, 9, 1, 1)) == [0, 1, 2, 3]
    assert list(oev.choose(w, 10, 4, 0, 0)) == [0, 2, 3, 5]              # ties: the lowest
    assert list(oev.choose(w, 10, 4, 1, 2)) == [0, 5, 8, 9]
    assert list(oev.choose(w, 10, 3, 2, 1)) == [0, 1, 9]                 # no choice left
    assert list(oev.choose(w, 10, 9, 0, 0)) == [0, 1, 2, 3, 5, 6, 7, 8, 9]   # NaN goes first


def test_oracle_gathers_closed_forms():
    """Equal keys: each allowed key of a row gets the same share, and a row's shares sum to
    one; rows without a sum add nothing."""
    keys = okv.Keys(8, 2, 16, 1, 64)
    table, off, past = np.array([[1, 0]]), np.array([0, 3]), np.array([2])
    okv.append(keys, table, np.array([0, 5]), np.array([0]), np.ones((5, 1, 64)))
    q = np.zeros((3, 2, 64))
    lse = np.log(np.array([[3.0, 3], [4, 4], [5, np.inf]]))
    old = np.full((1, 1, 32), 8.0)
    got, bound = oev.gather(keys, table, off, past, q, 1.0, lse, old, 0.5)
    assert np.allclose(got[0, 0, :6], [4 + 2 / 3 + 2 / 4 + 1 / 5] * 2 + [2 / 3 + 2 / 4 + 1 / 5, 2 / 4 + 1 / 5, 1 / 5, 8])
    assert (bound[0, 0, :5] > 0).all() and (bound[0, 0, 5:] == 0).all()
    got, _ = oev.gather(keys, table, off, past, q, 1.0, lse, old, 0.0, tree=[1, 2, 4])
    assert np.allclose(got[0, 0, :5], [2 / 3 + 2 / 4 + 1 / 5] * 2 + [2 / 3, 2 / 4, 1 / 5])


def test_oracle_evicts():
    """Tokens that stay hold the bytes they had, in order, in the first slots."""
    rng = np.random.default_rng(3)
    keys, values = okv.Keys(4, 4, 16, 2, 64), okv.Values(8, 4, 16, 2, 64)
    table, past = np.array([[2, 0, 3]]), np.array([40])
    x = rng.standard_normal((40, 2, 64))
    for side in (keys, values):
        okv.append(side, table, np.array([0, 40]), np.array([0]), x)
    before, _ = okv.held(keys, table, 0, 40)
    w = rng.random((1, 2, 48))
    out = np.zeros_like(w)
    kept, left = oev.evict(keys, values, table, past, w, out, 20, 1, 3)
    assert left[0] == 20 and (np.diff(kept[0], axis=1) > 0).all() and (kept[0, :, 0] == 0).all() and (kept[0, :, 17:] == [37, 38, 39]).all()
    after, _ = okv.held(keys, table, 0, 20)
    for h in range(2):
        assert np.array_equal(after[:, h], before[kept[0, h], h]) and np.array_equal(out[0, h, :20], w[0, h, kept[0, h]])
