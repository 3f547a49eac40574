"""Two layers of one model that share a batch, both cut to a budget."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from tests import _gpu as G
from tests import test_gpu_attention_layer as L
from tests import test_gpu_attention_layer_evict as E

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_two_layers_of_one_batch(captured):
    """The first layer's cut leaves the lengths to the second one's: caches, weights and the
    next step are those of layers with a batch of their own each."""
    start, budget, seqs, pages = (70, 45), 50, 2, 12
    results = []
    for shared in (False, True):
        layers = [E._layer(pages) for _ in range(2)]
        for layer in layers:
            for plane in layer.cache.planes:
                plane.zero_()

        def i32(a):
            return torch.from_numpy(np.asarray(a, np.int32)).to(G.DEV)

        table = i32(np.arange(pages).reshape(seqs, -1))
        pasts = [torch.zeros(seqs, dtype=torch.int32, device=G.DEV) for _ in layers]
        if shared:
            pasts[1] = pasts[0]
        prompts = [nv.KvBatch(table, i32([0, start[0], sum(start)]), p, sum(start), max(start), max(start)) for p in pasts]
        decodes = [nv.KvBatch(table, i32([0, 1, 2]), p, seqs, 1, pages // seqs * L.PAGE) for p in pasts]
        weights = [layer.alloc_weights(b) for layer, b in zip(layers, decodes)]
        kept = [torch.full((seqs, L.HEADS, budget), -7, dtype=torch.int32, device=G.DEV) for _ in layers]
        left = torch.empty(seqs, dtype=torch.int32, device=G.DEV)
        at = i32(np.concatenate([np.arange(n) for n in start]))
        for i, (layer, b, w) in enumerate(zip(layers, prompts, weights)):
            layer.reserve(b)
            layer.reserve(decodes[i])
            layer.step(L._inputs(sum(start), i), b, positions=at, weights=w)
        for p in pasts:
            p.copy_(i32(start))

        def cut():
            layers[0].evict(decodes[0], weights[0], budget, kept[0], first=2, recent=6, left=left if shared else None)
            layers[1].evict(decodes[1], weights[1], budget, kept[1], first=2, recent=6)

        G.note("eviction of two layers, shared %s, captured %s" % (shared, captured))
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                cut()
            graph.replay()
        else:
            cut()
        assert all(p.tolist() == [budget, start[1]] for p in pasts)
        if shared:
            assert left.tolist() == [budget, start[1]]
        x, got = L._inputs(seqs, 7), []
        for layer, b, w, k in zip(layers, decodes, weights, kept):
            y = layer.step(x, b, positions=i32(start), weights=w)
            got += [y.clone(), w, k, *layer.cache.planes]
        assert not torch.equal(kept[0][0], kept[1][0])
        results.append([t.cpu() for t in got])
    for a, b in zip(*results):
        assert torch.equal(a, b)
