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
