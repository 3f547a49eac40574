"""The attention half of a decoder layer on the library's low-bit products and its
quantised, paged key/value cache, as a program uses them:

    qkv = Wqkv x              nvfp4_gemv, float32
    cache <- k, v             nvfp4_kv_append, from the product's own rows
    o = attention(q, cache)   nvfp4_kv_attention
    y = Wo o                  nvfp4_gemv

One AttentionLayer serves prefill chunks, decode steps, batches of both, and the
verify of a tree of drafted tokens.  A decode step has no host-side state but the
batch's bounds, so it can be captured in a graph that advances the sequences by
itself.  Normalisation and the rotation of q and k by position are not part of it.

    python -m block_scaled_bit_nvfp4_amd.attention_layer

runs one: a prompt in two chunks, decode steps replayed from a graph, and a verify
of seven drafted tokens, and prints what each took.
"""
from __future__ import annotations

import math

import torch

import block_scaled_bit_nvfp4_amd as nv


class AttentionLayer:
    """Weights [rows, cols] float32 on the GPU, quantised to NVFP4 here: wqkv
    [(q_heads + 2 * heads) * head_dim, hidden] (queries, keys, values), wo [hidden,
    q_heads * head_dim].  max_tokens: the most tokens of a step."""

    def __init__(self, wqkv, wo, q_heads, heads, head_dim, max_tokens, pages, page_tokens=64,
                 k_format=nv.NVFP4_KV_MXFP8, v_format=nv.NVFP4_KV_MXFP8):
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

        def buffer(width, dtype):
            return torch.empty(max_tokens, width, dtype=dtype, device=self.device)

        self.qkv = buffer(rows, torch.float32)
        self.q, self.o = buffer(q_heads * head_dim, torch.bfloat16), buffer(q_heads * head_dim, torch.bfloat16)
        self.y = buffer(self.hidden, torch.float32)
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

    def step(self, x, batch, window=0, tree=None):
        """x bfloat16 [tokens, hidden], the batch's new tokens in its order; the
        result float32 [tokens, hidden], overwritten by the next step."""
        n = batch.tokens
        if n > self.max_tokens or tuple(x.shape) != (n, self.hidden):
            raise ValueError("x has shape %s, expected (%d, %d) with at most %d tokens" % (
                tuple(x.shape), n, self.hidden, self.max_tokens))
        if n == 0:
            return self.y[:0]
        self.reserve(batch)
        qkv, wide = self.qkv[:n], self.q_heads * self.head_dim
        nv.nvfp4_gemv(*self.wqkv, x, n, qkv)
        q, o = self.q[:n].view(n, self.q_heads, self.head_dim), self.o[:n].view(n, self.q_heads, self.head_dim)
        heads = qkv.view(n, -1, self.head_dim)
        q.copy_(heads[:, :self.q_heads])
        nv.nvfp4_kv_append(self.cache, batch, heads[:, self.q_heads:self.q_heads + self.heads],
                           heads[:, self.q_heads + self.heads:])
        nv.nvfp4_kv_attention(self.cache, batch, q, self.scale, o, window=window, tree=tree,
                              workspace=self.workspace)
        nv.nvfp4_gemv(*self.wo, o.view(n, wide), n, self.y[:n])
        return self.y[:n]


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
                           q_heads, heads, head_dim, chunk, pages, page)
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
        timed("prefill of %d tokens after %d" % (chunk, at), lambda: layer.step(x, b))
    past.fill_(prompt)

    # Decode: one token a step; the graph moves `past` on by itself.
    token, b = x[:1].clone(), batch(1, room)
    layer.reserve(b)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer.step(token, b)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer.step(token, b)
        token.copy_(y)                           # a stand-in for the rest of the layers
        past.add_(1)
    timed("decode step after %d tokens (graph)" % prompt, graph.replay, steps - 1)

    # Verify: seven drafted tokens and the one before them, as a tree of one chain.
    n = 8
    b, tree = batch(n, room), chain_mask(n, device)
    timed("verify of %d tokens (tree)" % n, lambda: layer.step(x[:n], b, tree=tree), 20)


if __name__ == "__main__":
    main()
