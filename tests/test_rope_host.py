"""Host-side checks of the rotary positions that need no GPU: the refusals, which come
before anything touches the device, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import rope as orope

OK, EINVAL, ESHAPE, EALIGN = 0, -1, -2, -3
A = 1 << 20          # an address that is aligned and never followed
B = 2 << 20


class Rows(ctypes.Structure):
    """struct nvfp4_rope_rows of nvfp4.h."""
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("in_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("heads", ctypes.c_int32), ("out_type", ctypes.c_int32)]


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def call(lib, rows=((A, B, 1024, 1024, 8, 0),), count=None, dtype=0, tokens=5, dim=128, rotary=128, adjacent=0,
         positions=A, axes=3, freqs=A, axis=A, factor=1.0):
    arr = None if rows is None else (Rows * 8)(*[Rows(*r) for r in rows])
    return lib.nvfp4_rope(arr, len(rows or ()) if count is None else count, dtype, tokens, dim, rotary, adjacent,
                          positions, axes, freqs, axis, factor, None)


def rows(**kw):
    d = dict(in_=A, out=B, in_stride=1024, out_stride=1024, heads=8, out_type=0)
    d.update(kw)
    return (tuple(d.values()),)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=None, count=1), EINVAL), (dict(count=0), EINVAL), (dict(count=5), EINVAL), (dict(dtype=2), EINVAL),
    (dict(tokens=-1), EINVAL), (dict(axes=0), EINVAL), (dict(positions=None), EINVAL), (dict(freqs=None), EINVAL),
    (dict(factor=0.0), EINVAL), (dict(factor=-1.0), EINVAL), (dict(factor=float("nan")), EINVAL),
    (dict(factor=float("inf")), EINVAL), (dict(rows=rows(in_=None)), EINVAL), (dict(rows=rows(out=None)), EINVAL),
    (dict(rows=rows(out_type=2)), EINVAL), (dict(rows=rows(out=A, out_type=1)), EINVAL),
    (dict(rows=rows(out=A, out_stride=2048)), EINVAL),
    (dict(dim=4), ESHAPE), (dict(dim=132), ESHAPE), (dict(dim=1032), ESHAPE), (dict(rotary=0), ESHAPE),
    (dict(rotary=136), ESHAPE), (dict(rotary=100), ESHAPE), (dict(tokens=1 << 31), ESHAPE), (dict(axes=257), ESHAPE),
    (dict(rows=rows(heads=0)), ESHAPE), (dict(rows=rows(heads=65536, in_stride=1 << 30, out_stride=1 << 30)), ESHAPE),
    (dict(rows=rows(in_stride=1023)), ESHAPE), (dict(rows=rows(out_stride=1016)), ESHAPE),
    (dict(rows=rows(in_stride=1 << 41)), ESHAPE), (dict(tokens=1 << 30), ESHAPE),
    (dict(rows=rows(in_=A + 8)), EALIGN), (dict(rows=rows(out=B + 8)), EALIGN), (dict(rows=rows(in_stride=1028)), EALIGN),
    (dict(rows=rows(out_stride=1028)), EALIGN), (dict(rows=rows(out_stride=1026, out_type=1)), EALIGN),
    (dict(freqs=A + 4), EALIGN), (dict(positions=A + 2), EALIGN),
    # the same set twice, and outputs that another set reads or writes
    (dict(rows=rows(out=A) * 2), EINVAL), (dict(rows=rows() * 2), EINVAL), (dict(rows=rows() + rows(in_=B, out=B + 4096)), EINVAL),
    (dict(rows=rows(in_=B, out=B + 4096) + rows()), EINVAL)])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status


def test_nothing_to_do_is_no_error(lib):
    assert call(lib, tokens=0) == OK
    assert call(lib, rows=rows(in_=None, out=None), tokens=0, positions=None) == OK


def test_binding_packs_the_struct():
    assert nv._rope_rows.size == ctypes.sizeof(Rows)
    assert nv._rope_rows.pack(A, B, 1 << 35, -3, 7, 1) == bytes(Rows(A, B, 1 << 35, -3, 7, 1))


def test_binding_refuses_before_the_library():
    x, pos, freqs = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32), torch.ones(32, dtype=torch.float64)
    for bad in ([], [x], [(x,)], [(x[0], x[0])], [(None, x)]):
        with pytest.raises(ValueError):
            nv.nvfp4_rope(bad, pos, freqs)
    with pytest.raises(ValueError):
        nv.nvfp4_rope([(x, x)], pos, freqs)                          # not on a GPU
    with pytest.raises(ValueError):
        nv.nvfp4_rope([(x, x)], pos.long(), freqs)
    with pytest.raises(ValueError):
        nv.nvfp4_rope([(x, x)], pos, freqs.float())


@pytest.mark.parametrize("adjacent", [False, True])
def test_oracle_turns_pairs(adjacent):
    """A quarter turn takes (a, b) to (-b, a); position 0 changes nothing; two turns add up;
    each pair follows its own axis."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 10))
    quarter = np.full(4, np.pi / 2)
    got, _, _ = orope.rope(x, [[1, 0]], quarter, adjacent=adjacent)
    even, odd = (slice(0, 8, 2), slice(1, 8, 2)) if adjacent else (slice(0, 4), slice(4, 8))
    assert np.allclose(got[0, :, even], -x[0, :, odd]) and np.allclose(got[0, :, odd], x[0, :, even])
    assert np.array_equal(got[1], x[1]) and np.array_equal(got[..., 8:], x[..., 8:])
    freqs, axis = rng.random(4), np.array([0, 1, 7, 1])
    once, _, _ = orope.rope(x, [[3, 4], [5, -6]], freqs, axis, adjacent)
    back, _, far = orope.rope(once, [[-3, -4], [-5, 6]], freqs, axis, adjacent)
    assert np.allclose(back, x) and far > 0
    assert np.array_equal(once[:, :, even][..., 2], x[:, :, even][..., 2])      # no such axis
