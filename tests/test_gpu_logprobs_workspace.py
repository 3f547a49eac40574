"""One workspace of the log probabilities, sized for the largest batch, in every smaller one."""
import pytest
import torch

import block_scaled_bit_nvfp4_amd as nv
from tests import _gpu as G
from tests import test_gpu_logprobs as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most,vocab,top", [(128, 32003, 20), (27, 151936, 20), (600, 9001, 5)])
def test_smaller_batches(most, vocab, top):
    """Rows on both sides of the change of chunks; nothing behind the workspace is written."""
    need = nv.nvfp4_logprobs_workspace_bytes(most, vocab, top)
    held = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device=G.DEV)
    short = 511 // -(-vocab // 8192)                     # the most rows in short chunks
    for n in (most, short + 1, short, 1):
        logits, likely = P._logits(n, vocab, n, torch.float32)
        G.note("logprobs of %d x %d in the workspace of %d" % (n, vocab, most))
        out = P._run(logits, likely[:, :1].int().contiguous(), top, workspace=held[:need])
        P._check(out, logits, likely[:, :1], top, 1.0, "%d rows" % n)
        assert (held[need:] == 0xA5).all()
