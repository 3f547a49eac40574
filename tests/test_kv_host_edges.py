"""Host-side edges of the key/value cache's entry points that need no GPU."""
import ctypes

from tests.test_kv_host import A, EINVAL, OK, append, attention, batch, cache, lib      # noqa: F401


def test_a_step_of_no_tokens_needs_no_rows(lib):      # noqa: F811
    """An empty tensor's address is null; what else is wrong is still refused."""
    none = batch(tokens=0)
    assert append(lib, cache(), none, k=None, v=None) == OK
    assert lib.nvfp4_kv_read(ctypes.byref(cache()), ctypes.byref(none), 0, None, 256, None, 256, None) == OK
    assert attention(lib, cache(), none, q=None, out=None, lse=None) == OK
    assert append(lib, cache(), none, dtype=2, k=None, v=None) == EINVAL
    assert attention(lib, cache(), none, q=None, out=None, lse=None, scale=0.0) == EINVAL
    one = batch(tokens=1)
    assert append(lib, cache(), one, k=None) == EINVAL and append(lib, cache(), one, v=None) == EINVAL
    assert lib.nvfp4_kv_read(ctypes.byref(cache()), ctypes.byref(one), 0, None, 256, None, 256, None) == EINVAL
    assert attention(lib, cache(), one, q=None) == EINVAL and attention(lib, cache(), one, out=None) == EINVAL
