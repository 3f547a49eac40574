"""nvfp4_kv_attention over long contexts and many splits, by closed forms that a
single key left out, or taken twice, would change; no oracle."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
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


@pytest.mark.parametrize("dim,k_fmt,v_fmt", [(64, 8, 8), (128, 4, 8), (256, 8, 4)])
@pytest.mark.parametrize("new,past,bound", [
    (1, 65535, 65536),                     # 256 splits of 256 keys
    (1, 131071, 131072), (7, 40000, 40007),
    (1, 9000, 1 << 30), (3, 70, 131072),   # bounds far above the context
    (300, 30001, 30301),                   # many rows, in splits
    (300, 3000, 1 << 30), (1100, 4500, 5600),
])
def test_every_key_counts_once(new, past, bound, dim, k_fmt, v_fmt):
    """Keys of zeros weigh the same: token i's log-sum-exp is log(past + i + 1).  fp32:
    counts are exact, log2 within a unit in the last place of 17 (2^-19), the
    product with log 2 within half a one of 12 (2^-21): 2^-18 in all, and a key more
    or less is 2^-17 of 131072.  Values that are zero but for element d of one
    token each give 2^16 / (past + i + 1) where the token is seen, to bf16's 2^-8."""
    G.note("attention, %d tokens after %d bounded by %d, D=%d" % (new, past, bound, dim))
    heads, group, page, n = 2, 4, 256, new + past
    rng = np.random.default_rng(dim + n)
    pages = -(-n // page)
    cache = nv.alloc_kv_cache(pages + 1, page, heads, dim, k_fmt, v_fmt, device=K.DEV)
    for p in cache.planes:
        p.fill_(0xFF)                      # what no token owns is NaN
    table = rng.permutation(pages + 1)[:pages].reshape(1, -1)
    # marked tokens: the first and last keys, either side of tiles' and splits' ends, and any others
    at = [0, n - 1, n - new, max(0, n - new - 1)] + [k + e for k in (32, 64, 128, 256, 512, 2048, 8192, 32768) for e in (-1, 0)]
    at = np.array([a for a in dict.fromkeys(at) if a < n][:dim])
    rest = np.setdiff1d(np.arange(n), at)
    at = np.concatenate((at, rng.choice(rest, min(dim, n) - len(at), replace=False)))
    values = torch.zeros(n, heads, dim, dtype=torch.bfloat16, device=K.DEV)
    for h in range(heads):
        values[torch.from_numpy(at), h, torch.arange(len(at))] = float(1 << 16)
    everything = K.batch_gpu(table, np.array([0, n]), np.array([0]))
    nv.nvfp4_kv_append(cache, everything, torch.zeros_like(values), values)
    batch = K.batch_gpu(table, np.array([0, new]), np.array([past]), max_context=bound)
    q = K.to_gpu(rng.standard_normal((new, heads * group, dim)), torch.bfloat16)
    out, lse = K.attend(cache, batch, q, dim ** -0.5, heads * group)
    seen = past + 1 + np.arange(new)
    off = np.abs(lse.double().cpu().numpy() - np.log(seen)[:, None])
    assert off.max() <= 2.0 ** -18, "log-sum-exp %.3g off" % off.max()
    want = np.where(at[None, :] < seen[:, None], 65536.0 / seen[:, None], 0.0)[:, None, :]
    o = out.double().cpu().numpy()
    assert (np.abs(o[..., :len(at)] - want) <= 2.0 ** -8 * want).all()
    assert (o[..., len(at):] == 0).all()
