"""Log probabilities on the GPU against the fp64 oracle.

Tolerances, in units of 2^-24.  A term e^d, d = z - m: d is one rounding off, its product
with log2(e) two more, each of d, and exp2 is off by two units: 3 |d| + 2 relative.  Summed
over the row with the probabilities, |d| is at most the entropy, H <= log V; the terms are
added in at most 32 + 2 * 6 + 4 + (chunks / 256 + 1) <= 64 steps, each one unit of the sum,
and joined with weights that are off as the terms are.  So l is off by at most
2 (3 log V + 2) + 64, log l by the same and one rounding, and lse by that and one unit
of itself, of log l and of m:  lse: 70 + 6 log V + 3 (|lse| + log V).
A log probability is d - log l: one rounding of d, at most |logp| + log V, and one of
the difference beside log l's error.  t = sum e^d d is off by
3 sum p d^2 + (2 + 64) H relative to l, twice over for the join's weights; the entropy,
log l - t / l, by the sum of these, of l's error on t / l, and a rounding of each part."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import logprobs as olp
from tests import _gpu as G

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
UNIT = 2.0 ** -24
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


def _run(logits, tokens, top, scale=1.0, stream=None, workspace=None):
    n, vocab = logits.shape
    out = {"logp": torch.full(tokens.shape, 7.0, device=G.DEV), "lse": torch.full((n,), 7.0, device=G.DEV),
           "entropy": torch.full((n,), 7.0, device=G.DEV), "top_logp": torch.full((n, top), 7.0, device=G.DEV),
           "top_index": torch.full((n, top), -7, dtype=torch.int32, device=G.DEV)}
    if workspace is None:
        workspace = torch.full((nv.nvfp4_logprobs_workspace_bytes(n, vocab, top),), 0xFF, dtype=torch.uint8, device=G.DEV)
    nv.nvfp4_logprobs(logits, tokens=tokens, scale=scale, workspace=workspace, stream=stream, **out)
    return out


def _check(out, logits, tokens, top, scale, what):
    x = logits.double().cpu().numpy()
    s = float(np.float32(scale))
    ref = olp.logprobs(x, tokens.cpu().numpy(), top, s)
    assert np.array_equal(out["top_index"].cpu().numpy(), ref["top_index"]), what
    log_v = np.log(x.shape[1])
    finite = np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0)
    l_off = 70 + 6 * log_v
    tol_lse = UNIT * (l_off + 3 * (finite + log_v))
    H = np.where(np.isfinite(ref["entropy"]), ref["entropy"], 0)
    tol_H = UNIT * (l_off + 6 * ref["square"] + (2 * 66 + l_off + 4) * H + 2 * log_v)

    def near(name, tol):
        got, want = out[name].double().cpu().numpy(), ref[name]
        with np.errstate(invalid="ignore", over="ignore"):      # past fp32's range: its infinity
            same = (got == want.astype(np.float32)) | (np.isnan(got) & np.isnan(want)) | (np.abs(got - want) <= tol)
        assert same.all(), "%s: %s: %d of %d off, first %r for %r" % (
            what, name, (~same).sum(), same.size, got[~same][0], want[~same][0])

    near("lse", tol_lse)
    near("entropy", tol_H)
    for name in ("logp", "top_logp"):
        near(name, UNIT * (l_off + 3 * log_v + 2 * np.where(np.isfinite(ref[name]), np.abs(ref[name]), 0)))


def _logits(n, vocab, seed, dtype, extra=0):
    """Rows of a stride of vocab + extra, some tokens of a row likely."""
    g = torch.Generator(G.DEV).manual_seed(seed)
    x = torch.randn(n, vocab + extra, generator=g, device=G.DEV) * 2
    at = torch.randint(0, vocab, (n, 4), generator=g, device=G.DEV)
    x.scatter_add_(1, at, 12 * torch.rand(n, 4, generator=g, device=G.DEV))
    return x.to(dtype)[:, :vocab], at


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,vocab", [(1, 151936), (3, 5003), (600, 9001)])
def test_a_token_that_is_all_but_certain(n, vocab, dtype):
    """Where l is 1 and a little, that little counts: log probability and entropy to a few
    units of themselves.  Terms are 3 |d| + 2 units off, |d| at most 32, and log l four more:
    102, below 128; t's terms are one more off and added in at most 64 steps: below 256."""
    g = torch.Generator(G.DEV).manual_seed(vocab)
    logits = torch.randn(n, vocab, generator=g, device=G.DEV).clamp(-5, 5)
    at = torch.randint(0, vocab, (n,), generator=g, device=G.DEV)
    logits[torch.arange(n, device=G.DEV), at] = torch.linspace(14, 27, n, device=G.DEV)
    logits = logits.to(dtype)
    G.note("logprobs of all but certain tokens, %d x %d %s" % (n, vocab, dtype))
    out = _run(logits, at.view(n, 1).int(), 1)
    assert torch.equal(out["top_index"][:, 0].long(), at)
    z = logits.double().cpu()
    d = z - z.amax(1, keepdim=True)
    little = torch.where(d == 0, torch.zeros_like(d), d.exp()).sum(1)
    logp = -torch.log1p(little)
    entropy = torch.log1p(little) - (d.exp() * d).sum(1) / (1 + little)
    for name, want, units in (("logp", logp, 128), ("top_logp", logp, 128), ("entropy", entropy, 256)):
        got = out[name].double().cpu().view(-1)
        assert ((got - want).abs() <= units * UNIT * want.abs()).all(), name


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,vocab,top,given,extra,scale", [
    (1, 1, 1, 1, 0, 1.0), (3, 2, 1, 2, 0, 1.0), (2, 63, 63, 0, 1, 0.5), (2, 64, 64, 1, 0, 1.0), (5, 100, 20, 3, 3, 2.0),
    (4, 1023, 5, 1, 0, 1.0), (1, 8191, 64, 1, 1, 1.0), (2, 8192, 64, 2, 0, 0.7), (2, 8193, 64, 1, 2, 1.0),
    (3, 8200, 20, 1, 1, 1.0), (7, 32003, 20, 3, 0, 1.25), (1, 151936, 20, 1, 0, 1.0), (2, 262144, 64, 1, 5, 1.0),
    (40, 16411, 0, 600, 0, 1.0), (600, 5003, 3, 1, 0, 1.0)])
def test_against_the_oracle(n, vocab, top, given, extra, scale, dtype):
    logits, likely = _logits(n, vocab, vocab + top, dtype, extra)
    g = torch.Generator(G.DEV).manual_seed(1)
    tokens = torch.randint(-2, vocab + 2, (n, given), generator=g, device=G.DEV, dtype=torch.int32)
    if given:
        tokens[:, 0] = likely[:, 0]
    G.note("logprobs %d x %d %s, top %d, %d given" % (n, vocab, dtype, top, given))
    _check(_run(logits, tokens, top, scale), logits, tokens, top, scale, "plain")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vocab", [50, 8192, 30011])
def test_masks_and_special_values(vocab, dtype):
    """Masked tokens, rows of nothing else, infinities and NaN, alone in a row or in all of
    a chunk of it, huge logits."""
    n, top = 12, 40
    x, _ = _logits(n, vocab, 5, F32)
    x[0] = -INF
    x[1] = -INF
    x[1, vocab - 1] = 3.0
    x[2, torch.rand(vocab, device=G.DEV) < 0.9] = -INF
    x[3, vocab // 2] = INF
    x[4, vocab - 1] = NAN
    x[5] = NAN
    x[6, :vocab // 2] = NAN
    x[7] = -INF
    x[7, 3] = NAN
    x[8] = -3e38
    x[8, 5:9] = 3e38
    x[9, :] = -0.0
    x[9, 7::3] = 0.0
    x[10, 8192:] = -INF
    x[11, :min(vocab - 4, 8192)] = -INF
    logits = x.to(dtype)
    tokens = torch.tensor([[0, vocab - 1, 3]] * n, dtype=torch.int32, device=G.DEV)
    G.note("logprobs of special values, %d %s" % (vocab, dtype))
    _check(_run(logits, tokens, top), logits, tokens, top, 1.0, "special")


@pytest.mark.parametrize("vocab", [600, 20000])
@pytest.mark.parametrize("levels", [1, 2, 40])
def test_ties(vocab, levels):
    """More equal logits than are kept as candidates: the lowest tokens come first."""
    g = torch.Generator(G.DEV).manual_seed(levels)
    logits = torch.randint(0, levels, (5, vocab), generator=g, device=G.DEV).float()
    logits[3] = -logits[3]
    tokens = torch.zeros(5, 1, dtype=torch.int32, device=G.DEV)
    G.note("logprobs of %d levels, %d tokens" % (levels, vocab))
    for top in (1, 13, 64):
        _check(_run(logits, tokens, top), logits, tokens, top, 1.0, "%d levels, top %d" % (levels, top))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [2, 600])
def test_few_threads_hold_the_largest(n, dtype):
    """Runs of four logits 1024 apart, as one thread reads them: 63 such columns are above
    all else, so that the 64th largest of the threads' maxima bounds next to nothing; and
    rows of a few allowed tokens, where all others are equal."""
    vocab, top = 9000, 64
    logits, _ = _logits(n, vocab, 21, dtype)
    at = torch.arange(vocab, device=G.DEV) // 4 % 256
    logits[:, at < 63] += 50
    for r, allowed in ((0, [8999, 17, 4096]), (1, [])):
        logits[r] = -INF
        logits[r, allowed] = 1.5
    tokens = torch.full((n, 1), 17, dtype=torch.int32, device=G.DEV)
    G.note("logprobs, the largest in few threads, %d rows %s" % (n, dtype))
    _check(_run(logits, tokens, top), logits, tokens, top, 1.0, "few threads")


@pytest.mark.parametrize("rising", [True, False])
def test_sorted_rows(rising):
    """The largest logits all in one chunk, one wave, one thread."""
    logits = torch.arange(40000, device=G.DEV).float().div_(1000).expand(3, -1).clone()
    if not rising:
        logits = logits.flip(1).contiguous()
    tokens = torch.tensor([[0], [39999], [20000]], dtype=torch.int32, device=G.DEV)
    _check(_run(logits, tokens, 64), logits, tokens, 64, 1.0, "sorted")


def test_outputs_one_by_one():
    """Each output alone has the bits that it has with all the others."""
    logits, _ = _logits(3, 20011, 4, F32)
    tokens = torch.tensor([[5], [6], [20010]], dtype=torch.int32, device=G.DEV)
    every = _run(logits, tokens, 9)
    wsp = torch.empty(1 << 16, dtype=torch.uint8, device=G.DEV)
    for names in (("lse",), ("entropy",), ("logp",), ("top_logp", "top_index")):
        got = {n: torch.empty_like(every[n]) for n in names}
        nv.nvfp4_logprobs(logits, tokens=tokens if "logp" in got else None, workspace=wsp, **got)
        for n in names:
            assert torch.equal(got[n], every[n]), n


def test_rows_of_large_strides():
    """Offsets past 32 bits: rows far apart in one allocation of 9 GB."""
    stride = (1 << 30) + 12345
    buf = torch.empty(2 * stride + 9000, dtype=F32, device=G.DEV)
    logits = buf.as_strided((3, 9000), (stride, 1))
    logits.copy_(_logits(3, 9000, 8, F32)[0])
    tokens = torch.tensor([[8999]] * 3, dtype=torch.int32, device=G.DEV)
    G.note("logprobs of rows 4 GB apart")
    _check(_run(logits, tokens, 20), logits, tokens, 20, 1.0, "far rows")


def test_refusals():
    logits, _ = _logits(2, 100, 1, F32)
    lse, wsp = torch.empty(2, device=G.DEV), torch.empty(1 << 12, dtype=torch.uint8, device=G.DEV)
    for kw in (dict(lse=lse[:1]), dict(lse=lse.double()), dict(lse=lse.cpu()), dict(entropy=lse[:0])):
        with pytest.raises(ValueError):
            nv.nvfp4_logprobs(logits, workspace=wsp, **kw)
    with pytest.raises(nv.NVFP4Error) as err:
        nv.nvfp4_logprobs(logits, lse=lse)
    assert err.value.status == -4
    with pytest.raises(nv.NVFP4Error) as err:
        nv.nvfp4_logprobs(logits[:1].expand(2, -1), lse=lse, workspace=wsp)      # rows over one another
    assert err.value.status == -2


def test_graph_replays_and_streams():
    """Two captured calls with workspaces of their own, replayed beside eager calls; a call
    on another stream."""
    cases = [(1, 40000, 20), (6, 9001, 5)]
    tokens = [torch.full((n, 2), 17, dtype=torch.int32, device=G.DEV) for n, _, _ in cases]
    bufs = [_logits(n, v, 3, F32)[0].contiguous() for n, v, _ in cases]
    work = [torch.empty(nv.nvfp4_logprobs_workspace_bytes(*c), dtype=torch.uint8, device=G.DEV) for c in cases]
    G.note("logprobs in graphs")
    for b, t, c, w in zip(bufs, tokens, cases, work):
        _run(b, t, c[2], workspace=w)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for b, t, c, w in zip(bufs, tokens, cases, work):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_run(b, t, c[2], workspace=w))
        graphs.append(g)
    for i in range(4):
        for b, (n, v, _) in zip(bufs, cases):
            b.copy_(_logits(n, v, 50 + i, F32)[0])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b, t, c, o in zip(bufs, tokens, cases, outs):
            want = _run(b, t, c[2])
            for name in o:
                assert torch.equal(o[name], want[name]), (i, name)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = _run(bufs[0], tokens[0], 20)
    torch.cuda.synchronize()
    want = _run(bufs[0], tokens[0], 20)
    assert all(torch.equal(got[name], want[name]) for name in got)


def test_with_the_products():
    """A vocabulary projection's logits: the likeliest token is the argmax product's, and a
    greedy token's log probability is the first alternative's."""
    R, K, n = 4099, 512, 4
    wq, ws = G.repack_gpu(*G.quantize_gpu(G.seeded_matrix(R, K, 1)), R, K)
    logits, am = G.gemv_argmax_gpu(wq, ws, 1.0, R, K, G.seeded_x(n, K, 2))
    out = _run(logits, am.view(n, 1), 5)
    assert torch.equal(out["top_index"][:, 0], am) and torch.equal(out["top_logp"][:, 0], out["logp"][:, 0])
    _check(out, logits, am.view(n, 1), 5, 1.0, "products")
