"""Log probabilities at scales whose products with the logits are rounded or pass fp32's
range: nothing is lost to that, since all sums refer to the largest logit itself."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from tests import _gpu as G
from tests import test_gpu_logprobs as P

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scale", [0.3, 0.7, 1.1, 1.4286])
@pytest.mark.parametrize("n,vocab", [(1, 151936), (3, 5003), (300, 5003), (600, 9001)])
def test_a_token_that_is_all_but_certain(n, vocab, scale, dtype):
    """As at a scale of 1, in units of 2^-24 of the result: with D = 32 * scale the largest
    |d|, a term e^d is off by 4 D + 2 (the difference and its product with the scale, log2(e)
    and the product with it, exp2), a chunk's weight by 2 more, the logarithm by 4, the
    result by 1: below 4 D + 10.  A term of t is 3 more off and added in at most 64 steps:
    below 4 D + 80.  The sum of exp in 64 bits is 1 and a little: each of its at most 64
    additions is off by half a step of a number in 1 .. 2, 2^-53, so that log l is off by
    64 * 2^-53 = 2^-47 whatever its size.  A probability is never above 1."""
    scale = float(np.float32(scale))
    g = torch.Generator(G.DEV).manual_seed(vocab + n)
    logits = torch.randn(n, vocab, generator=g, device=G.DEV).clamp(-5, 5)
    at = torch.randint(0, vocab, (n,), generator=g, device=G.DEV)
    logits[torch.arange(n, device=G.DEV), at] = 14 + 13 * torch.rand(n, generator=g, device=G.DEV)
    logits = logits.to(dtype)
    G.note("logprobs of all but certain tokens, %d x %d %s, scale %g" % (n, vocab, dtype, scale))
    out = P._run(logits, at.view(n, 1).int(), 1, scale)
    assert torch.equal(out["top_index"][:, 0].long(), at)
    x = logits.double().cpu()
    d = (x - x.amax(1, keepdim=True)) * scale
    little = torch.where(d == 0, torch.zeros_like(d), d.exp()).sum(1)
    logp = -torch.log1p(little)
    entropy = torch.log1p(little) - (d.exp() * d).sum(1) / (1 + little)
    for name, want, units in (("logp", logp, 128 * scale + 10), ("top_logp", logp, 128 * scale + 10),
                              ("entropy", entropy, 128 * scale + 80)):
        got = out[name].double().cpu().view(-1)
        assert ((got - want).abs() <= units * P.UNIT * want.abs() + 2.0 ** -47).all(), name
    assert (out["logp"] <= 0).all() and (out["top_logp"] <= 0).all() and (out["entropy"] >= 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [50, 20000])
@pytest.mark.parametrize("scale,size", [(2.0, 3e38), (1e30, 3e38), (1e30, 1.0), (3e38, 1e-37), (1e-38, 3e38), (0.75, 3e38),
                                        (3e38, 3e38), (1e-40, 3e38)])
def test_finite_logits_whose_products_are_not(scale, size, vocab, dtype):
    """Finite logits are no masked tokens and no infinities, however large their products
    with the scale are: log probabilities and entropy are those of their differences."""
    g = torch.Generator(G.DEV).manual_seed(vocab)
    x = size * (2 * torch.rand(8, vocab, generator=g, device=G.DEV) - 1)
    x[0] = size
    x[1] = -size
    x[2], x[2, ::3] = -float("inf"), -size
    x[3] = x[3].abs()
    x[4] = -x[4].abs()
    x[5], x[5, 7:9] = -size, size
    x[6] = torch.where(x[6] > 0, size, -size)
    logits = x.to(dtype)
    tokens = torch.tensor([[0, 7, vocab - 1]] * 8, dtype=torch.int32, device=G.DEV)
    G.note("logprobs of logits of %g, %d %s, scale %g" % (size, vocab, dtype, scale))
    out = P._run(logits, tokens, 20, scale)
    P._check(out, logits, tokens, 20, scale, "scale %g" % scale)
    assert (out["logp"][:2].isfinite()).all() and out["entropy"].isfinite().all()
