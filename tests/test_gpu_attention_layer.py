"""The attention layer built on the products, the cache and its attention: each
step's attention against the fp64 oracle on the layer's own queries, keys and
values, the products bit for bit, and a captured decode step against eager ones."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import kv as okv
from tests import _gpu as G
from tests import _kv as K

pytestmark = pytest.mark.gpu

HIDDEN, Q_HEADS, HEADS, DIM, PAGE, PAGES = 256, 8, 2, 64, 16, 12


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


def _layer(k_format=nv.NVFP4_KV_MXFP8, v_format=nv.NVFP4_KV_MXFP8):
    from block_scaled_bit_nvfp4_amd.attention_layer import AttentionLayer
    gen = torch.Generator(G.DEV).manual_seed(5)
    w = [torch.randn(r, c, generator=gen, device=G.DEV) * 0.06
         for r, c in (((Q_HEADS + 2 * HEADS) * DIM, HIDDEN), (HIDDEN, Q_HEADS * DIM))]
    return AttentionLayer(*w, Q_HEADS, HEADS, DIM, 96, PAGES, PAGE, k_format, v_format)


def _inputs(n, seed):
    gen = torch.Generator(G.DEV).manual_seed(seed)
    return torch.randn(n, HIDDEN, generator=gen, device=G.DEV).bfloat16()


@pytest.mark.parametrize("k_format,v_format", [(nv.NVFP4_KV_MXFP8, nv.NVFP4_KV_MXFP8),
                                               (nv.NVFP4_KV_MXFP4, nv.NVFP4_KV_MXFP8)])
def test_steps_against_the_oracle(k_format, v_format):
    from block_scaled_bit_nvfp4_amd.attention_layer import chain_mask
    layer = _layer(k_format, v_format)
    table = np.arange(PAGES, dtype=np.int32)[::-1].reshape(2, PAGES // 2).copy()
    keys = okv.Keys(k_format, PAGES, PAGE, HEADS, DIM, fill=0xFF)
    values = okv.Values(v_format, PAGES, PAGE, HEADS, DIM, fill=0xFF)
    past = np.zeros(2, np.int64)
    for seed, (new, tree) in enumerate([((70, 3), False), ((1, 1), False), ((5, 5), True)]):
        offsets, _ = K.lengths(new, past)
        batch, n = K.batch_gpu(table, offsets, past), sum(new)
        x = _inputs(n, seed)
        mask = torch.cat([chain_mask(m, G.DEV) for m in new]) if tree else None
        G.note("attention layer: %s after %s" % (new, past.tolist()))
        y = layer.step(x, batch, tree=mask).clone()
        qkv = G.gemv_gpu(*layer.wqkv, x)
        assert torch.equal(qkv, layer.qkv[:n])
        heads = qkv.view(n, -1, DIM).cpu().numpy().astype(np.float64)
        okv.append(keys, table, offsets, past, heads[:, Q_HEADS:Q_HEADS + HEADS])
        okv.append(values, table, offsets, past, heads[:, Q_HEADS + HEADS:])
        # a chain of drafted tokens sees what a causal mask shows
        ref = okv.attention(keys, values, table, offsets, past, K.bf16(heads[:, :Q_HEADS]), layer.scale)
        o = layer.o[:n].view(n, Q_HEADS, DIM)
        K.check(o, torch.from_numpy(ref[1]), ref, DIM, "step %d" % seed)
        assert torch.equal(y, G.gemv_gpu(*layer.wo, o.reshape(n, -1)))
        past += np.asarray(new)


def test_captured_decode_equals_eager():
    table = np.arange(PAGES, dtype=np.int32).reshape(1, PAGES)
    outs = []
    for captured in (False, True):
        layer = _layer()
        past = torch.zeros(1, dtype=torch.int32, device=G.DEV)
        arrays = [torch.from_numpy(a).to(G.DEV) for a in (table, np.array([0, 40], np.int32), np.array([0, 1], np.int32))]
        layer.step(_inputs(40, 1), nv.KvBatch(arrays[0], arrays[1], past, 40, 40, 40))
        past.fill_(40)
        token, batch = _inputs(1, 2), nv.KvBatch(arrays[0], arrays[2], past, 1, 1, PAGES * PAGE)

        def step():
            y = layer.step(token, batch)
            token.copy_(y)
            past.add_(1)

        layer.reserve(batch)
        G.note("decode steps, %s" % ("captured" if captured else "eager"))
        if captured:
            graph = torch.cuda.CUDAGraph()
            keep = token.clone()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            with torch.cuda.graph(graph):
                step()
            token.copy_(keep)
            past.fill_(40)
        got = []
        for i in range(6):
            graph.replay() if captured else step()
            got.append(layer.y[:1].clone())
            if i % 2:
                torch.cuda.synchronize()
                _inputs(3, 9).sum()              # work of the program's own between the replays
        assert int(past) == 46
        outs.append(torch.cat(got).cpu())
    assert torch.equal(*outs)
    assert outs[0].isfinite().all() and (outs[0][0] != outs[0][5]).any()


def test_refusals():
    layer = _layer()
    table = np.arange(PAGES, dtype=np.int32).reshape(1, PAGES)
    batch = K.batch_gpu(table, np.array([0, 97], np.int32), np.array([0], np.int32))
    with pytest.raises(ValueError):
        layer.step(_inputs(97, 0), batch)        # more than max_tokens
    with pytest.raises(ValueError):
        layer.step(_inputs(5, 0), batch)
    none = K.batch_gpu(table, np.array([0, 0], np.int32), np.array([0], np.int32))
    assert layer.step(_inputs(0, 0), none).shape == (0, HIDDEN)
