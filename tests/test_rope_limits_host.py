"""Rope calls whose workgroups would pass the largest launch are refused on the host."""
import pytest

from tests import test_rope_host as H

lib = H.lib


def set_of(at, heads, dim, dtype):
    return (at, at, heads * dim, heads * dim, heads, dtype)       # in place


# 2^24 workgroups of 256 threads each: a workgroup has at most 512 pairs of sines and
# cosines, so that few heads leave it few elements.
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("heads,dim,rotary,tokens", [
    ((1,), 128, 128, 1 << 27),          # 8 tokens a workgroup
    ((1,), 1024, 1024, 1 << 24),        # one token
    ((1, 1), 1024, 1024, 1 << 23), ((1, 1, 1, 1), 520, 520, 1 << 22)])
def test_too_many_workgroups(lib, heads, dim, rotary, tokens, dtype):
    rows = tuple(set_of(H.A + (i << 40), h, dim, dtype) for i, h in enumerate(heads))
    assert H.call(lib, rows=rows, dtype=dtype, tokens=tokens, dim=dim, rotary=rotary, axes=1, axis=None) == H.ESHAPE
