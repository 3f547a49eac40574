"""Helpers for the key/value cache tests: the same seeded case as numpy planes
for the oracle and as GPU tensors for the library."""
from __future__ import annotations

import numpy as np
import torch

import block_scaled_bit_nvfp4_amd as nv
from oracle import kv as okv

DEV = "cuda:0"
shape = "exact"              # of a batch's host numbers, see test_gpu_kv_attention.py


def lengths(new, past):
    return (np.concatenate(([0], np.cumsum(new))).astype(np.int32), np.asarray(past, np.int32))


def page_table(rng, new, past, page, spare=2, width=None):
    """A table of randomly ordered pages, one set per sequence, -1 past the end."""
    need = [-(-(n + p) // page) for n, p in zip(new, past)]
    width = max(need + [1]) if width is None else width
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(need), width), -1, np.int32)
    at = 0
    for s, k in enumerate(need):
        table[s, :k] = order[at:at + k]
        at += k
    return table, pages


def bf16(x):
    """The bf16 values nearest to x, float64."""
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def to_gpu(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).to(DEV)


def cache_gpu(keys, values, page):
    planes = [torch.from_numpy(a.reshape(-1)).to(DEV) for a in (keys.codes, keys.scales, values.codes, values.scales)]
    return nv.KvCache(*planes, keys.fmt, values.fmt, page, keys.heads, keys.dim)


def batch_gpu(table, offsets, past, tokens=None, max_new=None, max_context=None):
    new = np.diff(offsets)
    return nv.KvBatch(*[torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV) for a in (table, offsets, past)],
                      int(offsets[-1]) if tokens is None else tokens,
                      int(new.max()) if max_new is None else max_new,
                      int((new + past).max()) if max_context is None else max_context)


def filled(rng, new, past, heads, dim, k_fmt, v_fmt, page, big_channels=True):
    """Oracle planes holding random keys and values of every sequence's past and
    new tokens; what no token owns is NaN codes and NaN scales."""
    table, pages = page_table(rng, new, past, page)
    keys = okv.Keys(k_fmt, pages, page, heads, dim, fill=0xFF)
    values = okv.Values(v_fmt, pages, page, heads, dim, fill=0xFF)
    total = np.asarray(new) + np.asarray(past)
    offsets, zero = np.concatenate(([0], np.cumsum(total))), np.zeros(len(new), int)
    k = rng.standard_normal((total.sum(), heads, dim))
    if big_channels:
        k[..., rng.random(dim) < 0.05] *= 6
    okv.append(keys, table, offsets, zero, k)
    okv.append(values, table, offsets, zero, rng.standard_normal((total.sum(), heads, dim)))
    return table, keys, values


def attend(cache, batch, q, scale, q_heads, **kw):
    """One nvfp4_kv_attention into NaN-filled outputs and workspace."""
    out = torch.full_like(q, float("nan"))
    lse = torch.full((q.shape[0], q_heads), float("nan"), device=DEV)
    need = nv.nvfp4_kv_attention_workspace_bytes(cache, batch, q_heads)
    workspace = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV) if need else None
    nv.nvfp4_kv_attention(cache, batch, q, scale, out, lse=lse, workspace=workspace, **kw)
    return out, lse


def check(out, lse, ref, dim, what):
    """Each output within: bf16 rounding of the result (half a unit of 8 significant
    bits: at most 2^-8 of it); bf16 rounding of each weight (2^-8 of
    sum p |v|); the weights' own errors, exp2 to 2^-20 and the
    scores' fp32 sums of `dim` products, 2 dim 2^-24 sum |q k| on every key; the
    log-sum-exp by the same scores' error and 2^-20 of itself."""
    o_ref, lse_ref, spread, zmax = ref
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    dz = 2 * dim * 2.0 ** -24 * zmax + 2.0 ** -20
    tol = 1.01 * 2.0 ** -8 * np.abs(o_ref) + (1.01 * 2.0 ** -8 + 2 * dz[..., None]) * spread + 1e-30
    same = (np.isnan(o_ref) & np.isnan(o)) | (np.abs(o - o_ref) <= tol)
    assert same.all(), "%s: %d of %d outputs off, first at %s: %r for %r" % (
        what, (~same).sum(), same.size, np.argwhere(~same)[0], o[~same][0], o_ref[~same][0])
    ltol = dz + 2.0 ** -20 * np.abs(np.where(np.isfinite(lse_ref), lse_ref, 0))
    with np.errstate(invalid="ignore"):
        off = np.abs(l - lse_ref)
    lsame = (lse_ref == l) | (np.isnan(lse_ref) & np.isnan(l)) | (off <= ltol)
    assert lsame.all(), "%s: %d of %d log-sum-exps off, first %r for %r" % (
        what, (~lsame).sum(), lsame.size, l[~lsame][0], lse_ref[~lsame][0])
