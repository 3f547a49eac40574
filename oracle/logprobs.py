"""fp64 oracle of the log probabilities, written from the definition in
``include/nvfp4.h`` alone."""
from __future__ import annotations

import numpy as np


def logprobs(logits, tokens, top, scale=1.0):
    """logits [n, vocab], tokens [n, given] -> dict of logp, lse, entropy, top_index,
    top_logp, and for error bounds `square`, sum p (z - max z)^2 of each row."""
    x = np.asarray(logits, np.float64)
    n, vocab = x.shape
    out = {"logp": np.full(tokens.shape, np.nan), "lse": np.empty(n), "entropy": np.empty(n), "square": np.zeros(n),
           "top_index": np.empty((n, top), np.int64), "top_logp": np.empty((n, top))}
    for r in range(n):
        z = x[r] * scale
        best = sorted(range(vocab), key=lambda i: (np.isnan(x[r, i]), -x[r, i], i))[:top] if vocab <= 4096 else _best(x[r], top)
        if np.isnan(z).any() or np.isposinf(z).any():
            lse = entropy = np.nan
            logp = np.full(vocab, np.nan)
        elif np.isneginf(z).all():
            lse, entropy, logp = -np.inf, 0.0, np.full(vocab, -np.inf)
        else:
            m = z.max()
            e = np.exp(z - m)
            lse = m + np.log(e.sum())
            logp = (z - m) - np.log(e.sum())     # z - lse would lose both where m is huge
            p, some = e / e.sum(), e > 0
            entropy = -(p[some] * logp[some]).sum()
            out["square"][r] = (p[some] * (z[some] - m) ** 2).sum()
        out["lse"][r], out["entropy"][r], out["top_index"][r], out["top_logp"][r] = lse, entropy, best, logp[best]
        for i, t in enumerate(tokens[r]):
            if 0 <= t < vocab:
                out["logp"][r, i] = logp[t]
    return out


def _best(x, top):
    """The same order for long rows, by a stable sort of the values, NaN last."""
    return np.argsort(np.where(np.isnan(x), np.inf, -x) + 0.0, kind="stable")[:top] if not np.isnan(x).any() else \
        np.lexsort((np.arange(len(x)), np.where(np.isnan(x), 0, -x) + 0.0, np.isnan(x)))[:top]
