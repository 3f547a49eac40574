"""Rotary positions, gathered weights, eviction and log probabilities together, as the
attention layer and a program around it use them: each part of each step against its
fp64 oracle on the layer's own operands, and captured steps against eager ones."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from block_scaled_bit_nvfp4_amd.attention_layer import AttentionLayer, chain_mask
from oracle import evict as oev
from oracle import kv as okv
from tests import _gpu as G
from tests import _kv as K
from tests import test_gpu_attention_layer as L
from tests import test_gpu_kv_weights as W
from tests import test_gpu_logprobs as P
from tests import test_gpu_rope as R

pytestmark = pytest.mark.gpu
Q_HEADS, HEADS, DIM, HIDDEN, PAGE = L.Q_HEADS, L.HEADS, L.DIM, L.HIDDEN, L.PAGE


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


def _layer(pages, pairs=DIM // 2, k_format=nv.NVFP4_KV_MXFP8, v_format=nv.NVFP4_KV_MXFP8, **kw):
    gen = torch.Generator(G.DEV).manual_seed(5)
    w = [torch.randn(r, c, generator=gen, device=G.DEV) * 0.1
         for r, c in (((Q_HEADS + 2 * HEADS) * DIM, HIDDEN), (HIDDEN, Q_HEADS * DIM))]
    return AttentionLayer(*w, Q_HEADS, HEADS, DIM, 160, pages, PAGE, k_format, v_format,
                          freqs=torch.from_numpy(R._freqs(pairs)).to(G.DEV), **kw)


@pytest.mark.parametrize("k_format,v_format,pairs,adjacent,axes,window", [
    (8, 8, DIM // 2, False, 1, 0), (4, 8, DIM // 4, True, 3, 0), (8, 4, DIM // 2, False, 2, 37)])
def test_steps_and_evictions_against_the_oracles(k_format, v_format, pairs, adjacent, axes, window):
    """Chunks, decode steps and a drafted tree with evictions between them."""
    pages, budget, first, recent, factor = 24, 40, 3, 8, 1.125
    axis = np.arange(pairs) % axes
    layer = _layer(pages, pairs, k_format, v_format, adjacent=adjacent, rope_factor=factor,
                   axis=None if axes == 1 else torch.from_numpy(axis.astype(np.uint8)).to(G.DEV))
    freqs, rng = R._freqs(pairs), np.random.default_rng(pairs + axes)
    table = rng.permutation(pages).astype(np.int32).reshape(2, -1)
    keys = okv.Keys(k_format, pages, PAGE, HEADS, DIM, fill=0xFF)
    values = okv.Values(v_format, pages, PAGE, HEADS, DIM, fill=0xFF)
    for plane in layer.cache.planes:
        plane.fill_(0xFF)
    past, seen = np.zeros(2, np.int64), np.zeros(2, np.int64)      # held, and taken in all
    weights = None
    for step, (new, tree, cut) in enumerate([((90, 30), False, False), ((1, 1), False, True), ((1, 1), False, False),
                                             ((5, 9), True, True), ((50, 1), False, True), ((1, 1), False, False)]):
        tree = tree and not window
        offsets, _ = K.lengths(new, past)
        batch, n = K.batch_gpu(table, offsets, past), sum(new)
        if weights is None:
            weights = layer.alloc_weights(batch)
        x = L._inputs(n, step)
        positions = np.concatenate([np.arange(m) + at for m, at in zip(new, seen)])[None] * (1 + np.arange(axes))[:, None]
        mask = torch.cat([chain_mask(m, G.DEV) for m in new]) if tree else None
        what = "step %d: %s after %s" % (step, new, past.tolist())
        G.note("attention layer with positions, " + what)
        before, decay = weights.double().cpu().numpy(), 1.0 if step % 2 else 0.875
        layer.step(x, batch, window=window, tree=mask, weights=weights, decay=decay,
                   positions=torch.from_numpy(positions.astype(np.int32)).to(G.DEV))
        q = layer.q[:n].view(n, Q_HEADS, DIM)
        made = G.gemv_gpu(*layer.wqkv, x).view(n, -1, DIM)
        held = layer.qkv[:n].view(n, -1, DIM)
        k, v = held[:, Q_HEADS:Q_HEADS + HEADS], held[:, Q_HEADS + HEADS:]
        turned = (positions, freqs, axis, adjacent, factor, what)
        R._check(q, made[:, :Q_HEADS], *turned)
        R._check(k, made[:, Q_HEADS:Q_HEADS + HEADS], *turned)
        assert torch.equal(v, made[:, Q_HEADS + HEADS:])

        okv.append(keys, table, offsets, past, k.double().cpu().numpy())
        okv.append(values, table, offsets, past, v.double().cpu().numpy())
        q64, lse = q.double().cpu().numpy(), layer.lse[:n]
        ref = okv.attention(keys, values, table, offsets, past, q64, layer.scale, window)
        K.check(layer.o[:n].view(n, Q_HEADS, DIM), lse, ref, DIM, what)
        want, bound = oev.gather(keys, table, offsets, past, q64, layer.scale, lse.double().cpu().numpy(), before, decay, window)
        got = weights.double().cpu().numpy()
        tol = W.UNIT * bound + 2.0 ** -126 * n * Q_HEADS
        assert (np.abs(got - want) <= tol).all(), what
        # a row's probabilities add up to one over the keys it sees
        total = np.array([(got[s] - decay * np.where(np.arange(got.shape[2]) < past[s], before[s], 0))[:, :past[s] + new[s]].sum()
                          for s in range(2)])
        assert np.allclose(total, np.array(new) * Q_HEADS, rtol=1e-3)

        past, seen = past + np.asarray(new), seen + np.asarray(new)
        if cut:
            batch = K.batch_gpu(table, np.zeros(3, np.int32), past, tokens=0, max_new=0)
            kept = torch.full((2, HEADS, budget), -7, dtype=torch.int32, device=G.DEV)
            layer.evict(batch, weights, budget, kept, first=first, recent=recent)
            out = got.copy()
            ref_kept, left = oev.evict(keys, values, table, past, got, out, budget, first, recent)
            assert np.array_equal(kept.cpu().numpy(), ref_kept) and np.array_equal(batch.arrays[2].cpu().numpy(), left)
            assert np.array_equal(weights.double().cpu().numpy(), out)
            past = left
        for plane, side in zip(layer.cache.planes, (keys.codes, keys.scales, values.codes, values.scales)):
            assert np.array_equal(plane.cpu().numpy(), side.reshape(-1)), what


def test_generation_captured_equals_eager():
    """A program's whole step: the token's row, the layer, the head's product, the next
    tokens' log probabilities, and the cut to a budget that the steps grow past; captured
    and replayed, with other work between the replays."""
    vocab, start, budget, top, seqs = 1000, 44, 48, 4, 2
    table = np.arange(2 * 6, dtype=np.int32).reshape(seqs, -1)
    gen = torch.Generator(G.DEV).manual_seed(3)
    rows = torch.randn(vocab, HIDDEN, generator=gen, device=G.DEV).bfloat16()
    head = torch.randn(vocab, HIDDEN, generator=gen, device=G.DEV) * 0.1
    results = []
    for captured in (False, True):
        layer = _layer(12)
        wq, ws, tscale, r, c = layer._weights(head)
        def i32(a):
            return torch.from_numpy(np.asarray(a, np.int32)).to(G.DEV)
        arrays, past = i32(table), torch.zeros(seqs, dtype=torch.int32, device=G.DEV)
        prompt = nv.KvBatch(arrays, i32([0, start, 2 * start]), past, 2 * start, start, start)
        decode = nv.KvBatch(arrays, i32([0, 1, 2]), past, seqs, 1, 6 * PAGE)
        weights = layer.alloc_weights(decode)
        at = torch.full((seqs,), start, dtype=torch.int32, device=G.DEV)
        kept = torch.empty(seqs, HEADS, budget, dtype=torch.int32, device=G.DEV)
        x, logits = rows[[1, 2]].clone(), torch.empty(seqs, vocab, device=G.DEV)
        given = torch.zeros(seqs, 1, dtype=torch.int32, device=G.DEV)
        out = {"logp": torch.empty(seqs, 1, device=G.DEV), "lse": torch.empty(seqs, device=G.DEV),
               "entropy": torch.empty(seqs, device=G.DEV), "top_logp": torch.empty(seqs, top, device=G.DEV),
               "top_index": torch.empty(seqs, top, dtype=torch.int32, device=G.DEV)}
        workspace = torch.empty(nv.nvfp4_logprobs_workspace_bytes(seqs, vocab, top), dtype=torch.uint8, device=G.DEV)
        hidden = torch.empty(seqs, HIDDEN, dtype=torch.bfloat16, device=G.DEV)

        def step():
            hidden.copy_(layer.step(x, decode, positions=at, weights=weights))
            nv.nvfp4_gemv(wq, ws, tscale, r, c, hidden, seqs, logits)
            nv.nvfp4_logprobs(logits, tokens=given, workspace=workspace, **out)
            x.copy_(rows[out["top_index"][:, 0].long()])
            past.add_(1)
            at.add_(1)
            layer.evict(decode, weights, budget, kept, first=2, recent=6)

        def begin():
            past.zero_()
            weights.zero_()
            layer.step(rows[:2 * start], prompt, weights=weights,
                       positions=torch.arange(start, dtype=torch.int32, device=G.DEV).repeat(2))
            past.fill_(start)
            at.fill_(start)
            x.copy_(rows[[1, 2]])

        layer.reserve(decode)
        layer.reserve(prompt)
        G.note("generation, %s" % ("captured" if captured else "eager"))
        begin()
        graph = torch.cuda.CUDAGraph()
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            with torch.cuda.graph(graph):
                step()
            begin()
        got = []
        for i in range(9):
            given.fill_(7 * i)
            graph.replay() if captured else step()
            P._check(out, logits, given, top, 1.0, "step %d" % i)
            assert torch.equal(out["top_index"][:, 0], G.gemv_argmax_gpu(wq, ws, tscale, r, c, hidden)[1])
            got += [t.clone() for t in (logits, weights, kept, past, *out.values())]
            if i % 2:
                torch.cuda.synchronize()
                L._inputs(3, 9).sum()
        assert past.tolist() == [budget] * seqs and at.tolist() == [start + 9] * seqs
        assert not torch.equal(kept[0, 0].cpu(), torch.arange(budget, dtype=torch.int32))
        results.append([t.cpu() for t in got])
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_the_layer_without_frequencies_is_as_it_was():
    """Steps that gather weights give the results of steps that do not, and a layer without
    frequencies leaves its queries and keys as they are."""
    from tests.test_gpu_attention_layer import _layer as plain
    table = np.arange(12, dtype=np.int32).reshape(1, -1)
    results = []
    for gathers in (False, True):
        layer = plain()
        for seed, (n, past) in enumerate(((50, 0), (1, 50), (6, 51))):
            batch = K.batch_gpu(table, np.array([0, n]), np.array([past]))
            weights = layer.alloc_weights(batch) if gathers else None
            G.note("attention layer, weights %s" % gathers)
            y = layer.step(L._inputs(n, seed), batch, weights=weights).clone()
            results.append((y, layer.q[:n].clone(), layer.qkv[:n].clone()))
            assert torch.equal(layer.q[:n].view(-1), layer.qkv[:n, :Q_HEADS * DIM].bfloat16().reshape(-1))
    for a, b in zip(results[:3], results[3:]):
        assert all(torch.equal(*t) for t in zip(a, b))
