"""Gathered weights of more sequences than a wave has lanes, and evictions whose moves take
several stretches at every head size and format."""
import numpy as np
import pytest

from tests import _gpu as G
from tests import _kv as K
from tests import test_gpu_kv_evict as E
from tests import test_gpu_kv_weights as W

pytestmark = pytest.mark.gpu
_device = W._device


@pytest.mark.parametrize("seqs", [64, 65, 128, 131, 200])
@pytest.mark.parametrize("most,window,bounds", [(1, 0, (None, None)), (1, 20, (None, 5000)), (3, 0, (1, 1)), (40, 9, (None, None))])
def test_weights_of_many_sequences(seqs, most, window, bounds):
    """Lengths from nothing on, and stretches of sequences that have no new token; with a few
    long ones among them both kernels have their own."""
    rng = np.random.default_rng(seqs + most)
    new, past = rng.integers(0, most + 1, seqs), rng.integers(0, 70, seqs)
    new[5:9], new[60:66], past[62:70:2] = 0, 0, 0
    new[-1], past[-1], past[0] = most, 300, 150
    table, keys, values = K.filled(rng, new, past, 2, 64, 8, 8, 16)
    G.note("weights of %d sequences of up to %d new tokens, window %d" % (seqs, most, window))
    W._run(rng, table, keys, values, tuple(new), tuple(past), 6, 16, decay=0.7, window=window, bounds=bounds)


@pytest.mark.parametrize("dim,k_fmt,v_fmt", [(128, 8, 8), (128, 4, 8), (256, 8, 8), (256, 4, 4), (256, 8, 4)])
@pytest.mark.parametrize("length,budget", [(9000, 8300), (10000, 4097), (4200, 4096)])
def test_moves_of_several_stretches(length, budget, dim, k_fmt, v_fmt):
    rng = np.random.default_rng(length + dim)
    page = 256
    past = (length, 100)
    table, keys, values = E._planes(rng, past, 1, dim, k_fmt, v_fmt, page)
    weights = (rng.random((2, 1, table.shape[1] * page)) ** 8).astype(np.float32)
    weights[0, 0, rng.integers(0, length)] = np.nan
    G.note("evict %d to %d, a head of %d, %d/%d bits" % (length, budget, dim, k_fmt, v_fmt))
    E._run(table, keys, values, past, weights, page, budget, 4, 100, in_place=True)
