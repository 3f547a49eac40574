"""A workspace of the log probabilities that serves a batch serves every smaller one."""
import pytest

import block_scaled_bit_nvfp4_amd as nv
from tests import test_logprobs_host as H

size = nv.nvfp4_logprobs_workspace_bytes


@pytest.mark.parametrize("vocab", [1, 50, 2048, 2049, 8192, 8193, 32003, 151936, 262144, 5000000, 1 << 30])
@pytest.mark.parametrize("top", [0, 20, 64])
def test_sizes_never_fall_with_the_rows(vocab, top):
    top = min(top, vocab)
    rows = sorted({*range(1, 700), 1000, 4096, 10000, *(512 * 8192 // vocab + d for d in range(-3, 4) if vocab < 10000)})
    got = [size(n, vocab, top) for n in rows]
    got = got[:next((i for i, b in enumerate(got) if b == 0), len(got))]       # past the largest launch
    assert got and got == sorted(got)


def test_sizes_never_fall_with_the_likeliest():
    for n in (1, 26, 27, 500):
        got = [size(n, 151936, top) for top in range(65)]
        assert got == sorted(got)


@pytest.mark.parametrize("most,vocab,top", [(128, 32003, 20), (27, 151936, 20), (600, 9001, 1)])
def test_smaller_batches_take_the_largest_ones_workspace(most, vocab, top):
    """The workspace is looked at before its alignment, with which the call stops."""
    lib = nv.load()
    for n in range(1, most + 1):
        kw = dict(n=n, vocab=vocab, stride=vocab, top=top, ws=H.A + 8)
        assert H.call(lib, nbytes=size(most, vocab, top), **kw) == H.EALIGN, n
