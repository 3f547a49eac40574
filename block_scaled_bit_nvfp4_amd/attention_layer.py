"""The attention half of a decoder layer on the library's low-bit products and its
quantised, paged key/value cache, as a program uses them:

    qkv = Wqkv x              nvfp4_gemv, float32
    q, k turned by position   nvfp4_rope, where the layer has frequencies
    cache <- k, v             nvfp4_kv_append, from the product's own rows
    o = attention(q, cache)   nvfp4_kv_attention
    weights <- p(q, cache)    nvfp4_kv_weights, where the step is given weights
    y = Wo o                  nvfp4_gemv

One AttentionLayer serves prefill chunks, decode steps, batches of both, and the
verify of a tree of drafted tokens.  A decode step has no host-side state but the
batch's bounds, so it can be captured in a graph that advances the sequences by
itself.  A cache that is to stay within a budget is cut by `evict`, which keeps the
keys that the gathered weights name (nvfp4_kv_evict); tokens keep the positions that
they were turned by.  Normalisation is not part of it.

    python -m block_scaled_bit_nvfp4_amd.attention_layer

runs one: a prompt in two chunks, decode steps replayed from a graph, and a verify
of seven drafted tokens, decode steps that gather their weights and the eviction
of half of the cache, and prints what each took.
"""
from __future__ import annotations

import math

import torch

import block_scaled_bit_nvfp4_amd as nv


class AttentionLayer:
    """Weights [rows, cols] float32 on the GPU, quantised to NVFP4 here: wqkv
    [(q_heads + 2 * heads) * head_dim, hidden] (queries, keys, values), wo [hidden,
    q_heads * head_dim].  max_tokens: the most tokens of a step.  freqs, axis, adjacent
    and rope_factor: how q and k are turned, as nvfp4_rope takes them; not at all
    without freqs."""

    def __init__(self, wqkv, wo, q_heads, heads, head_dim, max_tokens, pages, page_tokens=64,
                 k_format=nv.NVFP4_KV_MXFP8, v_format=nv.NVFP4_KV_MXFP8, freqs=None, axis=None, adjacent=False,
                 rope_factor=1.0):
        self.q_heads, self.heads, self.head_dim = q_heads, heads, head_dim
        self.hidden = wo.shape[0]
        rows = (q_heads + 2 * heads) * head_dim
        if tuple(wqkv.shape) != (rows, self.hidden) or wo.shape[1] != q_heads * head_dim:
            raise ValueError("wqkv %s, wo %s: expected %s and %s" % (
                tuple(wqkv.shape), tuple(wo.shape), (rows, self.hidden), (self.hidden, q_heads * head_dim)))
        self.max_tokens, self.device = max_tokens, wqkv.device
        self.wqkv, self.wo = self._weights(wqkv), self._weights(wo)
        self.cache = nv.alloc_kv_cache(pages, page_tokens, heads, head_dim, k_format, v_format, self.device)
        self.scale = head_dim ** -0.5
        self.freqs, self.axis, self.adjacent, self.rope_factor = freqs, axis, adjacent, rope_factor

        def buffer(width, dtype):
            return torch.empty(max_tokens, width, dtype=dtype, device=self.device)

        self.qkv = buffer(rows, torch.float32)
        self.q, self.o = buffer(q_heads * head_dim, torch.bfloat16), buffer(q_heads * head_dim, torch.bfloat16)
        self.y, self.lse = buffer(self.hidden, torch.float32), buffer(q_heads, torch.float32)
        self.workspace = torch.empty(0, dtype=torch.uint8, device=self.device)
        self.retired = []            # outgrown workspaces, see reserve

    def _weights(self, w):
        """Planes and tensor scale of a matrix: the scale puts the largest block's at
        E4M3's largest, 448, so that the others' are normal numbers down to 2^-14 of it."""
        R, K = w.shape
        largest = float(w.abs().amax())
        if not math.isfinite(largest):
            raise ValueError("weights must be finite")
        tscale = max(largest / (6 * 448), 2.0 ** -126) if largest else 1.0
        codes = torch.empty(R, K // 2, dtype=torch.uint8, device=self.device)
        scales = torch.empty(R, K // 16, dtype=torch.uint8, device=self.device)
        nv.nvfp4_quantize(w.contiguous(), R, K, tscale, codes, scales)
        wq, ws = nv.alloc_repacked(R, K, self.device)
        nv.nvfp4_repack(codes, scales, R, K, wq, ws)
        return wq, ws, tscale, R, K

    def reserve(self, batch):
        """Room for the split attention of `batch`; before a capture, for its batch.  A
        captured step keeps writing to the workspace that it was captured with, so one
        that is outgrown stays the layer's own; each is at least twice the one
        before, so that all of them together take less than twice the last."""
        need = nv.nvfp4_kv_attention_workspace_bytes(self.cache, batch, self.q_heads)
        have = self.workspace.numel()
        if need > have:
            if have:
                self.retired.append(self.workspace)
            self.workspace = torch.empty(max(need, 2 * have), dtype=torch.uint8, device=self.device)

    def alloc_weights(self, batch):
        """Weights of 0 for the sequences of `batch`: of every key its page table can name."""
        seqs, width = batch.arrays[0].shape
        return torch.zeros(seqs, self.heads, width * self.cache.page_tokens, device=self.device)

    def step(self, x, batch, window=0, tree=None, positions=None, weights=None, decay=1.0):
        """x bfloat16 [tokens, hidden], the batch's new tokens in its order; the
        result float32 [tokens, hidden], overwritten by the next step.  positions int32
        [tokens] or [axes, tokens]: the tokens' own, for a layer that turns q and k (after
        an eviction they are no longer their places in the cache).  weights: of
        alloc_weights, to which the step adds the attention that each key receives; a cache
        that is to be cut is given them in every step, since only such a step starts its
        new keys at 0."""
        n = batch.tokens
        if n > self.max_tokens or tuple(x.shape) != (n, self.hidden):
            raise ValueError("x has shape %s, expected (%d, %d) with at most %d tokens" % (
                tuple(x.shape), n, self.hidden, self.max_tokens))
        if (positions is None) != (self.freqs is None):
            raise ValueError("positions come with a layer that has freqs, and only with one")
        if n == 0:
            return self.y[:0]
        self.reserve(batch)
        qkv, wide = self.qkv[:n], self.q_heads * self.head_dim
        nv.nvfp4_gemv(*self.wqkv, x, n, qkv)
        q, o = self.q[:n].view(n, self.q_heads, self.head_dim), self.o[:n].view(n, self.q_heads, self.head_dim)
        heads = qkv.view(n, -1, self.head_dim)
        k = heads[:, self.q_heads:self.q_heads + self.heads]
        if self.freqs is None:
            q.copy_(heads[:, :self.q_heads])
        else:
            nv.nvfp4_rope([(heads[:, :self.q_heads], q), (k, k)], positions, self.freqs, self.axis, self.adjacent,
                          self.rope_factor)
        nv.nvfp4_kv_append(self.cache, batch, k, heads[:, self.q_heads + self.heads:])
        lse = None if weights is None else self.lse[:n]
        nv.nvfp4_kv_attention(self.cache, batch, q, self.scale, o, lse=lse, window=window, tree=tree,
                              workspace=self.workspace)
        if weights is not None:
            nv.nvfp4_kv_weights(self.cache, batch, q, self.scale, lse, weights, decay=decay, window=window, tree=tree)
        nv.nvfp4_gemv(*self.wo, o.view(n, wide), n, self.y[:n])
        return self.y[:n]

    def evict(self, batch, weights, budget, kept, first=0, recent=0, left=None):
        """Cut the batch's sequences that hold more than `budget` tokens (`past`, without
        the step's new ones) down to it: of each head the first `first`, the last `recent`
        and the keys of the largest weights stay.  kept int32 [seqs, heads, budget] gets
        their places before the cut; weights move with them.  left int32 [seqs] gets the
        tokens held now; without it past itself does.  Where layers share a batch, all but the
        last to be cut are given a `left`: a layer that finds the budget in past cuts
        nothing, and would take its first tokens for all that it holds."""
        nv.nvfp4_kv_evict(self.cache, batch, weights, budget, kept, batch.arrays[2] if left is None else left,
                          first=first, recent=recent)


def chain_mask(n, device):
    """A tree mask of n tokens in a chain: token i sees tokens 0 .. i."""
    bits = [(1 << (i + 1)) - 1 for i in range(n)]
    return torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device=device)


def main(hidden=5120, q_heads=40, heads=8, head_dim=128, prompt=4096, steps=64, device="cuda"):
    import time

    torch.manual_seed(0)
    page, chunk = 64, prompt // 2
    room = prompt + steps + 64
    pages = -(-room // page)
    layer = AttentionLayer(torch.randn((q_heads + 2 * heads) * head_dim, hidden, device=device) * 0.02,
                           torch.randn(hidden, q_heads * head_dim, device=device) * 0.02,
                           q_heads, heads, head_dim, chunk, pages, page,
                           freqs=10000.0 ** -(torch.arange(head_dim // 2, dtype=torch.float64, device=device) * 2 / head_dim))
    place = torch.arange(room, dtype=torch.int32, device=device)
    table = torch.randperm(pages, device=device).to(torch.int32).view(1, pages)
    past = torch.zeros(1, dtype=torch.int32, device=device)

    def batch(n, context):
        return nv.KvBatch(table, torch.tensor([0, n], dtype=torch.int32, device=device), past, n, n, context)

    def timed(what, f, times=1):
        f()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for _ in range(times):
            f()
        torch.cuda.synchronize()
        print("%-44s %9.1f us" % (what, (time.perf_counter() - t0) / times * 1e6), flush=True)

    x = torch.randn(chunk, hidden, device=device).bfloat16()
    for at in (0, chunk):                        # the prompt, in two chunks
        past.fill_(at)
        b = batch(chunk, at + chunk)
        timed("prefill of %d tokens after %d" % (chunk, at),
              lambda: layer.step(x, b, positions=place[at:at + chunk]))
    past.fill_(prompt)

    # Decode: one token a step; the graph moves `past` and the position on by itself.
    token, b, at = x[:1].clone(), batch(1, room), past.clone()
    layer.reserve(b)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.step(token, b, positions=at)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(token, b, positions=at)
        token.copy_(y)                           # a stand-in for the rest of the layers
        past.add_(1)
        at.add_(1)
    timed("decode step after %d tokens (graph)" % prompt, graph.replay, steps - 1)

    # Verify: seven drafted tokens and the one before them, as a tree of one chain.
    n = 8
    b, tree = batch(n, room), chain_mask(n, device)
    timed("verify of %d tokens (tree)" % n,
          lambda: layer.step(x[:n], b, tree=tree, positions=place[prompt + steps:prompt + steps + n]), 20)

    # A budget: steps that gather what the keys receive, and the cut to half of the cache.
    b = batch(1, room)
    weights, kept = layer.alloc_weights(b), torch.empty(1, heads, prompt // 2, dtype=torch.int32, device=device)
    timed("decode step that gathers weights", lambda: layer.step(token, b, positions=at, weights=weights), 20)

    def cut():
        past.fill_(prompt)
        layer.evict(b, weights, prompt // 2, kept, first=4, recent=64)

    timed("eviction of %d tokens of %d" % (prompt - prompt // 2, prompt), cut, 20)
    timed("decode step after it", lambda: layer.step(token, b, positions=at, weights=weights), 20)


if __name__ == "__main__":
    main()
