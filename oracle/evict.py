"""fp64 oracle of the gathered attention weights and of eviction by them, in plain numpy
loops.  Written from the definitions in ``include/nvfp4.h`` alone."""
from __future__ import annotations

import numpy as np

from oracle import kv as okv


def allowed(n, past, i, window, word):
    """Which of the past + n positions new token i sees."""
    j, pos = np.arange(past + n), past + i
    ok = j <= pos
    if word is not None:
        bit = j - past
        ok = (j < past) | ((bit >= 0) & (bit < 64) & ((int(word) >> np.clip(bit, 0, 63).astype(object)) & 1).astype(bool))
    return ok & (j > pos - window) if window else ok


def gather(keys, table, offsets, past, q, scale, lse, old, decay, window=0, tree=None):
    """-> (weights as `old` with the gathered ones, and a bound of their error in units of
    2^-24, laid out as old).

    The bound, for each weight p = exp(z - lse): scores are sums of D products in fp32 (2 D
    units of sum |q k| scale), the exponent's multiply-add rounds once and its constants
    are off by a unit (3 |z - lse| / ln 2 with exp2's argument), exp2 and the row's factor
    are off by 2 units each, and the sums take a step for each 32 rows and 16 more; the
    decayed weight and the last sum round once each."""
    heads, dim = keys.heads, keys.dim
    group = q.shape[1] // heads
    out, bound = old.copy(), np.zeros_like(old)
    for s in range(len(past)):
        n = offsets[s + 1] - offsets[s]
        if n == 0:
            continue
        k, some = okv.held(keys, table, s, past[s] + n)
        for h in range(heads):
            good = some & np.isfinite(k[:, h]).all(-1)
            total, err = np.zeros(past[s] + n), np.zeros(past[s] + n)
            for i in range(n):
                t = offsets[s] + i
                ok = allowed(n, past[s], i, window, None if tree is None else tree[t]) & good
                for g in range(group):
                    r = h * group + g
                    if not np.isfinite(lse[t, r]):
                        continue
                    z = scale * (k[ok, h] @ q[t, r])
                    p = np.exp(z - lse[t, r])
                    size = scale * (np.abs(k[ok, h]) @ np.abs(q[t, r]))
                    total[ok] += p
                    err[ok] += p * (2 * dim * size + 3 * np.abs(z - lse[t, r]) / np.log(2) + 8)
            steps = n * group / 32 + 16
            end = min(past[s] + n, table.shape[1] * keys.page_tokens)      # positions past the table have no place
            total, err = total[:end], err[:end]
            before = np.where(np.arange(end) < past[s], old[s, h, :end], 0.0)
            before = decay * before if decay else np.zeros_like(before)
            out[s, h, :end] = before + total
            bound[s, h, :end] = err + steps * total + 2 * np.abs(before) + 2 * total
    return out, bound


def choose(weights, length, budget, first, recent):
    """The kept positions of one head, ascending."""
    if length <= budget:
        return np.arange(length)
    inner = np.arange(first, length - recent)
    w = weights[inner]
    order = sorted(range(len(inner)), key=lambda i: (np.isnan(w[i]), -w[i] if not np.isnan(w[i]) else 0, i))
    stay = np.sort(inner[order[:budget - first - recent]])
    return np.concatenate((np.arange(first), stay, np.arange(length - recent, length))).astype(int)


def evict(keys, values, table, past, weights, weights_out, budget, first, recent):
    """Moves the planes' bytes and weights_out in place; -> (kept, left)."""
    heads, page = keys.heads, keys.page_tokens
    kept = np.full((len(past), heads, budget), -1, np.int64)
    left = np.array(past, np.int64)
    for s, length in enumerate(past):
        pages = [okv.page_of(table, len(keys.codes), page, s, p) for p in range(max(length, 0))]
        if -1 in pages:
            continue
        cut = length > budget
        for h in range(heads):
            stay = choose(weights[s, h], length, budget, first, recent)
            kept[s, h, :len(stay)] = stay
            weights_out[s, h, :len(stay)] = weights[s, h, stay]
            if not cut:
                continue
            for side in (keys, values):
                raw = [(side.codes[pages[p], h, p % page // 16][side._code_bytes(p % 16)].copy(),
                        side.scales[pages[p], h, p % page // 16][side._scale_bytes(p % 16)].copy()) for p in stay]
                for i, (codes, scales) in enumerate(raw):
                    side.codes[pages[i], h, i % page // 16][side._code_bytes(i % 16)] = codes
                    side.scales[pages[i], h, i % page // 16][side._scale_bytes(i % 16)] = scales
        if cut:
            left[s] = budget
    return kept, left
