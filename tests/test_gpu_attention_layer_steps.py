"""The attention layer as a server runs it: captured decode steps beside larger
steps, against the same steps taken eagerly."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from block_scaled_bit_nvfp4_amd.attention_layer import AttentionLayer
from oracle import kv as okv
from tests import _gpu as G
from tests import _kv as K
from tests import test_gpu_attention_layer as L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    nv.load()
    yield
    torch.cuda.synchronize()


def test_captured_decode_survives_larger_steps():
    """Steps that need a larger workspace than the captured one's, between its
    replays: the replays equal eager steps, and what the program allocated
    meanwhile keeps its contents."""
    table = np.arange(L.PAGES, dtype=np.int32).reshape(2, -1)
    arrays = [torch.from_numpy(a).to(G.DEV) for a in (table, np.array([0, 40, 40], np.int32), np.array([0, 1, 1], np.int32),
                                                      np.array([0, 0, 60], np.int32))]
    outs = []
    for captured in (False, True):
        layer = L._layer()
        past, zero = torch.zeros(2, dtype=torch.int32, device=G.DEV), torch.zeros(2, dtype=torch.int32, device=G.DEV)
        layer.step(L._inputs(40, 1), nv.KvBatch(arrays[0], arrays[1], past, 40, 40, 40))
        past[:1].fill_(40)
        # the bounds shape the launches: a decode step and a chunk of the other sequence, both in splits
        token, decode = L._inputs(1, 2), nv.KvBatch(arrays[0], arrays[2], past, 1, 1, 4000)
        large = nv.KvBatch(arrays[0], arrays[3], zero, 60, 60, 100000)
        sizes = [nv.nvfp4_kv_attention_workspace_bytes(layer.cache, b, L.Q_HEADS) for b in (decode, large)]
        assert 0 < 2 * sizes[0] < sizes[1]
        layer.reserve(decode)
        G.note("decode steps beside chunks, %s" % ("captured" if captured else "eager"))
        graph = torch.cuda.CUDAGraph()
        if captured:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                layer.step(token, decode)
            torch.cuda.current_stream().wait_stream(side)
            with torch.cuda.graph(graph):
                layer.step(token, decode)
        got, bystanders = [], []
        for i in range(5):
            token.copy_(L._inputs(1, 10 + i))
            past[:1].fill_(40 + i)
            graph.replay() if captured else layer.step(token, decode)
            got.append(layer.y[:1].clone())
            got.append(layer.step(L._inputs(60, 20 + i), large).clone())
            # blocks of the size that the first workspace had
            bystanders += [torch.full((sizes[0],), 0x55, dtype=torch.uint8, device=G.DEV) for _ in range(4)]
            torch.cuda.synchronize()
        for b in bystanders:
            assert (b == 0x55).all()
        outs.append(torch.cat(got).cpu())
    assert torch.equal(*outs) and outs[0].isfinite().all()


@pytest.mark.parametrize("std", [1e4, 0.06, 0.01, 0.002, 1e-5])
def test_weights_of_any_size_are_held(std):
    """Each weight within the E2M1 code's half step of its block: a block's unit is its
    largest magnitude over 6, rounded to E4M3 (at most 2^-4 of it, while the scales are
    normal numbers), and the widest gap between codes is two units.  A scale for each
    matrix keeps the block scales in E4M3's range whatever the weights' size."""
    G.note("attention layer, weights of %g" % std)
    gen = torch.Generator(G.DEV).manual_seed(7)
    weights = [torch.randn(r, c, generator=gen, device=G.DEV) * s
               for r, c, s in (((L.Q_HEADS + 2 * L.HEADS) * L.DIM, L.HIDDEN, std), (L.HIDDEN, L.Q_HEADS * L.DIM, 0.1 * std))]
    layer = AttentionLayer(*weights, L.Q_HEADS, L.HEADS, L.DIM, 8, L.PAGES, L.PAGE)
    for w, planes in zip(weights, (layer.wqkv, layer.wo)):
        held = torch.empty_like(w)
        nv.nvfp4_dequant(*planes, out_f32=held)
        largest = w.double().abs().unflatten(1, (-1, 16)).amax(-1, keepdim=True)
        off = (w.double() - held.double()).abs().unflatten(1, (-1, 16))
        bad = int((off > (1 + 2.0 ** -4) / 6 * largest * (1 + 2.0 ** -20)).sum())
        assert bad == 0, "%d of %d weights are off" % (bad, off.numel())


def test_weights_without_a_scale():
    """Zeros stay zeros, weights at the bottom of float32's range are no error, and
    what is not finite is refused."""
    G.note("attention layer, weights without a scale")
    shape = (L.Q_HEADS + 2 * L.HEADS) * L.DIM, L.HIDDEN
    wo = torch.zeros(L.HIDDEN, L.Q_HEADS * L.DIM, device=G.DEV)
    batch = K.batch_gpu(np.arange(L.PAGES).reshape(1, -1), np.array([0, 3]), np.array([0]))
    for w in (torch.zeros(shape, device=G.DEV), torch.full(shape, 2.0 ** -149, device=G.DEV)):
        layer = AttentionLayer(w, wo, L.Q_HEADS, L.HEADS, L.DIM, 8, L.PAGES, L.PAGE)
        assert (layer.step(L._inputs(3, 1), batch) == 0).all()
    for bad in (float("inf"), float("nan")):
        w = torch.zeros(shape, device=G.DEV)
        w[3, 5] = bad
        with pytest.raises(ValueError):
            AttentionLayer(w, wo, L.Q_HEADS, L.HEADS, L.DIM, 8, L.PAGES, L.PAGE)


def test_a_steps_attention_against_the_oracle():
    """The layer's attention outputs, and the log-sum-exp of the same call on its own
    queries and cache, against the fp64 oracle."""
    layer = L._layer()
    table = np.arange(L.PAGES, dtype=np.int32)[::-1].reshape(2, -1).copy()
    keys, values = (kind(8, L.PAGES, L.PAGE, L.HEADS, L.DIM, fill=0xFF) for kind in (okv.Keys, okv.Values))
    past = np.zeros(2, np.int64)
    for seed, new in enumerate([(70, 3), (1, 1), (9, 30)]):
        offsets, _ = K.lengths(new, past)
        batch, n = K.batch_gpu(table, offsets, past), sum(new)
        G.note("attention layer: %s after %s, log-sum-exp" % (new, past.tolist()))
        layer.step(L._inputs(n, seed), batch)
        heads = layer.qkv[:n].view(n, -1, L.DIM).double().cpu().numpy()
        okv.append(keys, table, offsets, past, heads[:, L.Q_HEADS:L.Q_HEADS + L.HEADS])
        okv.append(values, table, offsets, past, heads[:, L.Q_HEADS + L.HEADS:])
        q = layer.q[:n].view(n, L.Q_HEADS, L.DIM)
        assert np.array_equal(q.double().cpu().numpy(), K.bf16(heads[:, :L.Q_HEADS]))
        out, lse = K.attend(layer.cache, batch, q, layer.scale, L.Q_HEADS)
        assert torch.equal(out, layer.o[:n].view_as(out))
        ref = okv.attention(keys, values, table, offsets, past, q.double().cpu().numpy(), layer.scale)
        K.check(out, lse, ref, L.DIM, "step %d" % seed)
        past += np.asarray(new)
