"""The attention layer as a server runs it: captured decode steps beside larger
steps, against the same steps taken eagerly."""
import numpy as np
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from tests import _gpu as G
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
