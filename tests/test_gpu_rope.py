"""Rotary positions on the GPU against the fp64 oracle.

Tolerance, in units of 2^-24 of factor * (|a| + |b|) of an element's pair: the angle left
after whole quarter turns is rounded, multiplied by a rounded pi / 2 and that product
rounded (3 of at most pi / 4: 2.4); the series' last steps round once each (1.1, with what
the earlier ones leave); the factor's product (1); the two products and their sum (2).
That is less than 8, 2^-21.  The angle itself, position * (frequency * 2 / pi) in 64 bits,
is off by three roundings of 2^-53 of it, here taken as 2^-50.  An output in bf16 is
rounded by at most 2^-8 of itself."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import rope as orope
from tests import _gpu as G

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


def _freqs(pairs, base=10000.0):
    return base ** -(np.arange(pairs) / pairs)


def _dev(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(G.DEV)


def _check(out, x, positions, freqs, axis, adjacent, factor, what):
    ref, size, far = orope.rope(x.double().cpu().numpy(), positions, freqs, axis, adjacent, factor)
    tol = (2.0 ** -21 + far * 2.0 ** -50) * size
    if out.dtype == BF16:
        tol = tol + 1.01 * 2.0 ** -8 * np.abs(ref) + 1e-38
    got = out.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        same = (np.abs(got - ref) <= tol) | (np.isnan(ref) & np.isnan(got)) | (got == ref)
    assert same.all(), "%s: %d of %d off, first at %s: %r for %r" % (
        what, (~same).sum(), same.size, np.argwhere(~same)[0], got[~same][0], ref[~same][0])


def _qkv(tokens, heads, dim, dtype, seed, more=1):
    """Rows of one projection: the sets' heads, and columns that nobody is to touch."""
    g = torch.Generator(G.DEV).manual_seed(seed)
    return torch.randn(tokens, (sum(heads) + more) * dim, generator=g, device=G.DEV).to(dtype)


def _split(qkv, heads, dim):
    at, out = 0, []
    for h in heads:
        out.append(qkv[:, at * dim:(at + h) * dim].unflatten(1, (h, dim)))
        at += h
    return out


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,heads,dim,rotary,axes", [
    (1, (32, 8), 128, 128, 1), (2, (5,), 8, 8, 2), (63, (3, 1, 2), 72, 72, 2), (300, (16, 16), 80, 40, 3),
    (7, (1, 1, 1, 1), 1024, 64, 1), (1500, (40, 8), 128, 128, 3), (33, (12, 2), 256, 64, 3), (129, (4,), 64, 24, 4),
    (4099, (7,), 72, 72, 2),
    # enough of them for sines and cosines that are shared: heads in ranges, units of every kind
    (1300, (16, 16), 80, 40, 3), (400, (1, 1, 1, 1), 1024, 64, 1), (101, (23, 2), 1024, 1024, 2), (9001, (5,), 64, 24, 4),
    (50001, (5, 1), 8, 8, 2), (1500, (3, 70), 256, 256, 1)])
def test_against_the_oracle(tokens, heads, dim, rotary, axes, dtype, adjacent):
    rng = np.random.default_rng(tokens + dim)
    pairs = rotary // 2
    positions = rng.integers(-5, 1 << 20, (axes, tokens))
    freqs, axis = _freqs(pairs), rng.integers(0, axes, pairs) if axes > 1 else None
    factor = 1.0 if tokens % 2 else 1.25
    qkv = _qkv(tokens, heads, dim, dtype, tokens)
    kept = qkv.clone()
    ins = _split(qkv, heads, dim)
    # outputs of either type, one of them in rows of its own stride
    wide = [torch.full((tokens, h + i, dim), float("nan"), dtype=(BF16, F32)[i % 2], device=G.DEV)
            for i, h in enumerate(heads)]
    outs = [w[:, :h] for w, h in zip(wide, heads)]
    G.note("rope %d tokens, heads %s of %d, %d turn, %d axes, %s" % (tokens, heads, dim, rotary, axes, dtype))
    nv.nvfp4_rope(list(zip(ins, outs)), _dev(positions, torch.int32), _dev(freqs, torch.float64),
                  None if axis is None else _dev(axis, torch.uint8), adjacent, factor)
    assert torch.equal(qkv, kept)
    for i, (x, out) in enumerate(zip(ins, outs)):
        _check(out, x, positions, freqs, axis, adjacent, factor, "set %d" % i)
        assert wide[i][:, heads[i]:].isnan().all()


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype,dim,rotary", [(BF16, 128, 128), (BF16, 72, 72), (F32, 128, 96)])
def test_a_token_alone_and_among_many(dtype, dim, rotary, adjacent):
    """A token's result does not depend on how many others the call has."""
    tokens, heads = 2500, (12, 3)
    rng = np.random.default_rng(dim)
    positions = _dev(rng.integers(0, 1 << 16, (2, tokens)), torch.int32)
    freqs, axis = _dev(_freqs(rotary // 2), torch.float64), _dev(rng.integers(0, 2, rotary // 2), torch.uint8)
    ins = _split(_qkv(tokens, heads, dim, dtype, 5), heads, dim)
    outs = [torch.empty(tokens, h, dim, dtype=BF16, device=G.DEV) for h in heads]
    G.note("rope, a token among many, %s" % dtype)
    nv.nvfp4_rope(list(zip(ins, outs)), positions, freqs, axis, adjacent, 1.5)
    for t in (0, 1, 1249, tokens - 1):
        one = [torch.empty(1, h, dim, dtype=BF16, device=G.DEV) for h in heads]
        nv.nvfp4_rope(list(zip([x[t:t + 1] for x in ins], one)), positions[:, t:t + 1].contiguous(), freqs, axis, adjacent, 1.5)
        for a, b in zip(one, outs):
            assert torch.equal(a[0], b[t])


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens", [5, 3001])
def test_in_place(tokens, dtype, adjacent):
    """The same bits as out of place, and nothing beside the sets changes."""
    heads, dim = (6, 2), 128
    positions = _dev(np.arange(tokens), torch.int32)
    freqs = _dev(_freqs(32), torch.float64)
    qkv = _qkv(tokens, heads, dim, dtype, 3, more=2)
    before = qkv.clone()
    outs = [torch.empty(tokens, h, dim, dtype=dtype, device=G.DEV) for h in heads]
    G.note("rope in place, %d tokens, %s" % (tokens, dtype))
    nv.nvfp4_rope(list(zip(_split(qkv, heads, dim), outs)), positions, freqs, adjacent=adjacent)
    nv.nvfp4_rope([(x, x) for x in _split(qkv, heads, dim)], positions, freqs, adjacent=adjacent)
    for x, out in zip(_split(qkv, heads, dim), outs):
        assert torch.equal(x, out)
    assert torch.equal(qkv[:, 8 * dim:], before[:, 8 * dim:])


def test_far_positions_and_large_frequencies():
    """Positions to the ends of 32 bits; whole turns leave nothing but the fraction."""
    positions = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 9, 7]])
    tokens, freqs = positions.shape[1], np.array([1.0, 0.37, 1e-3, 2 * np.pi / 3])
    x = _qkv(tokens, (3,), 8, F32, 9, more=0).unflatten(1, (3, 8))
    out = torch.empty_like(x)
    G.note("rope of far positions")
    nv.nvfp4_rope([(x, out)], _dev(positions[0], torch.int32), _dev(freqs, torch.float64))
    _check(out, x, positions, freqs, None, False, 1.0, "far")


def test_exact_quarter_turns():
    """Angles next to whole quarter turns, where sine and cosine change places."""
    step = np.pi / 2
    positions = np.arange(-9, 10)[None]
    for freq in (step, step * (1 + 1e-9), step / 2, step / 2 * (1 - 1e-12)):
        freqs = np.full(4, freq)
        x = _qkv(19, (1,), 8, F32, 5, more=0).unflatten(1, (1, 8))
        out = torch.empty_like(x)
        nv.nvfp4_rope([(x, out)], _dev(positions, torch.int32), _dev(freqs, torch.float64), adjacent=True)
        _check(out, x, positions, freqs, None, True, 1.0, "quarters of %r" % freq)


def test_axes_that_are_not_there_and_special_values():
    """A pair of no axis turns by 0; an infinity or a NaN reaches its own pair alone."""
    tokens, freqs = 4, _freqs(8)
    axis = np.array([0, 1, 2, 255, 1, 0, 7, 1])
    positions = np.array([[5, 6, 7, 8], [50, 60, 70, 80]])
    x = _qkv(tokens, (2,), 24, F32, 6, more=0).unflatten(1, (2, 24))
    x[1, 0, 3], x[2, 1, 9], x[3, 0, 20] = float("inf"), float("nan"), float("-inf")
    out = torch.empty_like(x)
    G.note("rope: axes that are not there, infinities")
    nv.nvfp4_rope([(x, out)], _dev(positions, torch.int32), _dev(freqs, torch.float64), _dev(axis, torch.uint8),
                  factor=0.5)
    _check(out, x, positions, freqs, axis, False, 0.5, "special")


def test_turning_back():
    """Negative positions undo a rotation, to the roundings of both."""
    x = _qkv(200, (4,), 64, F32, 8, more=0).unflatten(1, (4, 64))
    pos, freqs = torch.randint(0, 1 << 20, (200,), device=G.DEV, dtype=torch.int32), _dev(_freqs(32), torch.float64)
    y, back = torch.empty_like(x), torch.empty_like(x)
    nv.nvfp4_rope([(x, y)], pos, freqs)
    nv.nvfp4_rope([(y, back)], -pos, freqs)
    size = x.unflatten(-1, (2, 32)).abs().sum(2)
    # each element of y is off by 2^-21 of its pair, which the way back at most doubles
    assert ((back - x).abs() <= 4 * 2.0 ** -21 * torch.cat((size, size), -1)).all()


def test_no_tokens():
    x = torch.empty(0, 4, 64, device=G.DEV)
    nv.nvfp4_rope([(x, x)], torch.empty(0, dtype=torch.int32, device=G.DEV), _dev(_freqs(32), torch.float64))


def test_graph_replays_follow_the_positions():
    tokens, heads, dim = 3, (4, 2), 128
    qkv = _qkv(tokens, heads, dim, F32, 11)
    pos = torch.zeros(2, tokens, dtype=torch.int32, device=G.DEV)
    freqs, axis = _freqs(64), np.arange(64) % 2
    f, ax = _dev(freqs, torch.float64), _dev(axis, torch.uint8)
    ins = _split(qkv, heads, dim)
    outs = [torch.empty(tokens, h, dim, dtype=BF16, device=G.DEV) for h in heads]
    G.note("rope in a graph")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        nv.nvfp4_rope(list(zip(ins, outs)), pos, f, ax)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_rope(list(zip(ins, outs)), pos, f, ax)
        pos.add_(1)
    for i in range(4):
        at = np.array([[i * 100, 5, 6], [7, i * 1000, 9]])
        pos.copy_(_dev(at, torch.int32))
        qkv.copy_(_qkv(tokens, heads, dim, F32, 20 + i))
        graph.replay()
        torch.cuda.synchronize()
        for x, out in zip(ins, outs):
            _check(out, x, at, freqs, axis, False, 1.0, "replay %d" % i)
        assert torch.equal(pos.cpu(), torch.from_numpy(at).int() + 1)


def test_another_stream():
    """Work of another stream: the call waits for what that stream holds, by its order."""
    x = _qkv(2000, (8,), 128, F32, 12, more=0).unflatten(1, (8, 128))
    pos, f = _dev(np.arange(2000), torch.int32), _dev(_freqs(64), torch.float64)
    want = torch.empty_like(x)
    nv.nvfp4_rope([(x, want)], pos, f)
    out, late = torch.empty_like(x), torch.zeros_like(x)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        late.copy_(x)
        nv.nvfp4_rope([(late, out)], pos, f)
    nv_out = torch.empty_like(x)
    nv.nvfp4_rope([(late, nv_out)], pos, f, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(nv_out, want)
