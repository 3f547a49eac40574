"""Host-side checks of the log probabilities that need no GPU: sizes, the refusals, which
come before anything touches the device, and the oracle's own pins."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import logprobs as olp

OK, EINVAL, ESHAPE, EALIGN, EWORKSPACE = 0, -1, -2, -3, -4
A = 1 << 20          # an address that is aligned and never followed


@pytest.fixture(scope="module")
def lib():
    return nv.load()


def call(lib, dtype=1, logits=A, n=3, vocab=1000, stride=1000, scale=1.0, tokens=A, given=2, logp=A, lse=A, entropy=A,
         top=5, top_logp=A, top_index=A, ws=None, nbytes=0):
    return lib.nvfp4_logprobs(dtype, logits, n, vocab, stride, scale, tokens, given, logp, lse, entropy, top, top_logp,
                              top_index, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), EINVAL), (dict(logits=None), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL), (dict(given=-1), EINVAL),
    (dict(given=(1 << 20) + 1), EINVAL), (dict(tokens=None), EINVAL), (dict(logp=None), EINVAL),
    (dict(top_logp=None), EINVAL), (dict(top_index=None), EINVAL),
    (dict(given=0, tokens=None, logp=None, top=0, lse=None, entropy=None), EINVAL),
    (dict(n=-1), ESHAPE), (dict(n=(1 << 30) + 1), ESHAPE), (dict(vocab=0), ESHAPE),
    (dict(vocab=(1 << 30) + 1, stride=1 << 31), ESHAPE), (dict(n=1 << 30, vocab=100000, stride=100000), ESHAPE),
    (dict(top=-1), ESHAPE), (dict(top=65), ESHAPE), (dict(vocab=4, top=5), ESHAPE), (dict(stride=999), ESHAPE),
    (dict(stride=1 << 41), ESHAPE), (dict(logits=A + 2), EALIGN), (dict(dtype=0, logits=A + 1), EALIGN),
    (dict(tokens=A + 2), EALIGN), (dict(logp=A + 1), EALIGN), (dict(lse=A + 2), EALIGN), (dict(entropy=A + 2), EALIGN),
    (dict(top_logp=A + 2), EALIGN), (dict(top_index=A + 2), EALIGN),
    (dict(), EWORKSPACE), (dict(ws=A, nbytes=3 * (16 + 40) - 1), EWORKSPACE), (dict(ws=A + 8, nbytes=1 << 20), EALIGN)])
def test_refusals(lib, kw, status):
    assert call(lib, **kw) == status


def test_no_rows_are_no_error(lib):
    assert call(lib, n=0, logits=None, tokens=None, logp=None, lse=None, entropy=None, top_logp=None, top_index=None) == OK


def test_workspace_sizes():
    size = nv.nvfp4_logprobs_workspace_bytes
    # four numbers a chunk, of 2048 logits for a few rows and 8192 for many, and its keys
    assert size(3, 1000, 5) == 3 * (16 + 5 * 8) and size(3, 8192, 0) == 3 * 4 * 16 and size(3, 8193, 0) == 3 * 5 * 16
    assert size(2, 151936, 20) == 2 * 75 * (16 + 160) and size(512, 151936, 20) == 512 * 19 * (16 + 160)
    assert size(0, 1000, 5) == 0 and size(1, 0, 0) == 0 and size(1, 10, 11) == 0 and size(1, 100, 65) == 0


def test_binding_refuses_before_the_library():
    x = torch.zeros(2, 100)
    with pytest.raises(TypeError):
        nv.nvfp4_logprobs(None)
    for bad in (x[0], x.half(), x.t()):
        with pytest.raises(ValueError):
            nv.nvfp4_logprobs(bad, lse=torch.zeros(2))
    tokens, logp = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3)
    for kw in (dict(tokens=tokens), dict(logp=logp), dict(tokens=tokens, logp=logp[:1]), dict(tokens=tokens[0], logp=logp),
               dict(top_index=tokens), dict(top_index=tokens, top_logp=logp[:, :2]), dict(tokens=tokens, logp=logp)):
        with pytest.raises(ValueError):
            nv.nvfp4_logprobs(x, **kw)                               # the last: not on a GPU


def test_oracle_closed_forms():
    """Equal logits, one certain token, masked tokens, rows without a finite sum, ties."""
    inf, nan = float("inf"), float("nan")
    x = np.array([[1.0, 1, 1, 1], [0, 800, 0, 0], [-inf, 2, -inf, 2], [-inf] * 4, [0, inf, 0, 0], [0, nan, 1, -inf],
                  [-0.0, 0.0, -1, 0.0]])
    got = olp.logprobs(x, np.array([[1, 4]] * 7), 4, 1.0)
    assert np.allclose(got["lse"][:3], [1 + np.log(4), 800, 2 + np.log(2)]) and np.allclose(
        got["entropy"][:3], [np.log(4), 0, np.log(2)])
    assert np.isnan(got["logp"][:, 1]).all() and np.allclose(got["logp"][:3, 0], [-np.log(4), 0, -np.log(2)])
    assert got["lse"][3] == -inf and got["entropy"][3] == 0 and (got["top_logp"][3] == -inf).all()
    assert np.isnan(got["lse"][4:6]).all() and np.isnan(got["top_logp"][4:6]).all()
    assert got["top_index"].tolist() == [[0, 1, 2, 3], [1, 0, 2, 3], [1, 3, 0, 2], [0, 1, 2, 3], [1, 0, 2, 3],
                                         [2, 0, 3, 1], [0, 1, 3, 2]]
    assert np.allclose(olp.logprobs(x[1:2] / 100, np.zeros((1, 1), int), 0, 0.5)["lse"], np.log(3 + np.exp(4)))
    long = np.round(np.random.default_rng(0).standard_normal(5000) * 3)
    long[7], long[9] = nan, -0.0
    assert list(olp._best(long, 50)) == sorted(range(5000), key=lambda i: (np.isnan(long[i]), -long[i], i))[:50]
