"""nvfp4_kv_attention on values that are not finite, against the fp64 oracle, at
every head size and with both kernels."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import kv as okv
from tests import _gpu as G
from tests import _kv as K
from tests.test_gpu_kv_attention import _run, _shape      # noqa: F401  (every case at three launch shapes)

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")]


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dim,k_fmt", [(64, 8), (128, 4), (256, 8)])
@pytest.mark.parametrize("new,past,tree", [(3, 200, False), (100, 300, False), (40, 0, True)])
def test_infinities_in_queries(dim, k_fmt, new, past, tree, monkeypatch):
    """A query with an infinity has no softmax: its row is NaN, also where every score
    is minus infinity; one that may see nothing gets zeros all the same, and the
    other rows are as ever."""
    G.note("attention, infinite queries D=%d, %d after %d" % (dim, new, past))
    heads, group = 2, 4
    rng = np.random.default_rng(dim + new)
    at = [(0, 1, 0, -np.inf), (new - 1, 6, dim - 1, -np.inf), (new - 1, 0, 17, np.inf), (new // 2, 3, 40, np.nan),
          (1, 5, 8, -np.inf)]

    def edit(table, keys, values):
        # keys above zero: a query of minus infinity scores minus infinity everywhere
        k = np.abs(rng.standard_normal((new + past, heads, dim))) + 0.25
        okv.append(keys, table, np.array([0, new + past]), np.array([0]), k)

    to_gpu = K.to_gpu

    def with_infinities(x, dtype):
        for t, h, d, v in at:
            x[t, h * dim + d] = v
        return to_gpu(x, dtype)

    monkeypatch.setattr(K, "to_gpu", with_infinities)
    words = None
    if tree:
        words = [(1 << (i + 1)) - 1 for i in range(new)]
        words[1] = 0                                # sees nothing: no past either
    out, lse, ref = _run(rng, [new], [past], heads, group, dim, k_fmt, 8, page=32, edit=edit,
                         tree=None if words is None else np.array(words, dtype=object))
    o = out.float().cpu().numpy()
    for t, h, _, _ in at:
        if tree and t == 1:
            assert (o[t, h] == 0).all() and lse[t, h] == float("-inf")
        else:
            assert np.isnan(o[t, h]).all()
    assert np.isnan(o).any(-1).sum() == len(at) - tree


def _nan(side, table, pos, head, block, page):
    """One block of one token becomes NaN."""
    unit, r = divmod(pos % page, 16)
    side.scales[table[0, pos // page], head, unit, side._scale_bytes(r)[block]] = 0xFF


@pytest.mark.parametrize("dim,k_fmt,v_fmt", [(64, 8, 8), (64, 4, 4), (128, 8, 4), (128, 4, 8), (256, 4, 8), (256, 8, 4)])
@pytest.mark.parametrize("new,group", [(40, 4), (100, 8)])
def test_nan_blocks_of_new_tokens(new, group, dim, k_fmt, v_fmt):
    """A NaN block of a value reaches its elements, a NaN block of a key everything, in
    the rows that see the token and no other."""
    G.note("attention, NaN among %d new tokens D=%d %d/%d" % (new, dim, k_fmt, v_fmt))
    past, last = 50, dim // 32 - 1

    def edit(table, keys, values):
        _nan(values, table, past + new // 2, 0, 1, 32)
        _nan(values, table, past + new // 2 + 3, 1, 0, 32)
        _nan(keys, table, past + new - 2, 0, last, 32)
        _nan(values, table, past + new - 1, 0, last, 32)

    out, lse, ref = _run(np.random.default_rng(dim), [new], [past], 2, group, dim, k_fmt, v_fmt, page=32, edit=edit)
    o, half = out.float().cpu().numpy(), new // 2
    assert np.isfinite(o[:half]).all() and np.isnan(o[half:, :group, 32:64]).all() and np.isnan(o[new - 2:, :group]).all()
    assert np.isfinite(o[half:new - 2, :group, :32]).all() and np.isfinite(o[half:new - 2, :group, 64:]).all()
    assert np.isnan(o[half + 3:, group:, :32]).all() and np.isfinite(o[:, group:, 32:]).all()


@pytest.mark.parametrize("dim,k_fmt,v_fmt", [(64, 8, 4), (128, 4, 8), (256, 8, 8)])
@pytest.mark.parametrize("new,window", [(3, 0), (100, 0), (100, 60)])
def test_nan_blocks_of_the_past(new, window, dim, k_fmt, v_fmt):
    """The same in tiles that every row sees, and where the rows' windows pass them."""
    G.note("attention, NaN in the past of %d new tokens D=%d window %d" % (new, dim, window))
    past = 300

    def edit(table, keys, values):
        _nan(values, table, 140 if window == 0 else past - 20, 0, 1, 32)
        _nan(keys, table, 170 if window == 0 else past - 10, 1, 0, 32)

    out, lse, ref = _run(np.random.default_rng(dim), [new], [past], 3, 4, dim, k_fmt, v_fmt, page=32, edit=edit, window=window)
    o = out.float().cpu().numpy()
    v_rows, k_rows = (new, new) if window == 0 else (window - 20, window - 10)        # the rows that see them
    assert np.isnan(o[:v_rows, :4, 32:64]).all() and np.isfinite(o[:, :4, :32]).all() and np.isfinite(o[v_rows:, :4]).all()
    assert np.isnan(o[:k_rows, 4:8]).all() and np.isfinite(o[k_rows:, 4:8]).all() and np.isfinite(o[:, 8:]).all()
