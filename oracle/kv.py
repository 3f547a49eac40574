"""fp64 oracle of the paged key/value cache: quantisation of the new tokens, the
cache's bytes, and attention over it, in plain numpy loops over sequences and
heads.  Written from the definitions in ``include/nvfp4.h`` alone."""
from __future__ import annotations

import numpy as np

MXFP4, MXFP8 = 4, 8


def code_values(fmt: int) -> np.ndarray:
    """The value of every code of a format, float64 (E4M3: 0x7F and 0xFF NaN)."""
    if fmt == MXFP4:
        mag = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    else:
        c = np.arange(128)
        e, m = c >> 3, c & 7
        mag = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
        mag[127] = np.nan
    return np.concatenate((mag, -mag))


def quantise(x: np.ndarray, fmt: int):
    """x [..., D] -> (codes uint8 [..., D], scale bytes uint8 [..., D / 32])."""
    x = np.asarray(x, np.float64)
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    bad = ~np.isfinite(b).all(-1)
    safe = np.where(bad[..., None], 0.0, b)
    amax = np.abs(safe).max(-1)
    part, ex = np.frexp(amax)                       # amax = part * 2^ex
    if fmt == MXFP4:
        E = ex - 1 - 2
    else:
        E = np.where(part * 2 <= 1.75, ex - 1 - 8, ex - 8)
    E = np.where(amax == 0, -127, np.clip(E, -127, 127))
    y = np.ldexp(np.abs(safe), -E[..., None])
    mags = code_values(fmt)[:8 if fmt == MXFP4 else 127]
    y = np.minimum(y, mags[-1])
    hi = np.clip(np.searchsorted(mags, y), 0, len(mags) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = mags[hi] - y, y - mags[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    code |= np.where(np.signbit(safe), 8 if fmt == MXFP4 else 128, 0).astype(np.uint8)
    code[bad] = 0
    return code.reshape(x.shape), np.where(bad, 255, E + 127).astype(np.uint8)


def dequantise(codes: np.ndarray, scales: np.ndarray, fmt: int) -> np.ndarray:
    v = code_values(fmt)[codes]
    unit = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(unit, 32, -1)


class Side:
    """One side's planes of a pool, as bytes, and the place of every token's."""

    def __init__(self, fmt, pages, page_tokens, heads, dim, fill=0):
        self.fmt, self.page_tokens, self.heads, self.dim = fmt, page_tokens, heads, dim
        units = page_tokens // 16
        self.codes = np.full((pages, heads, units, 16 * dim * fmt // 8), fill, np.uint8)
        self.scales = np.full((pages, heads, units, 16 * dim // 32), fill, np.uint8)

    def _code_bytes(self, r):
        """Offsets in the unit of token r's code bytes."""
        raise NotImplementedError

    def _scale_bytes(self, r):
        raise NotImplementedError

    def _row_bytes(self, codes):
        return codes if self.fmt == MXFP8 else codes[..., 0::2] | (codes[..., 1::2] << 4)

    def put(self, page, pos, codes, scales):
        """Store one token [heads, D] at place pos of a page."""
        u, r = divmod(pos, 16)
        self.codes[page, :, u, self._code_bytes(r)] = self._row_bytes(codes).T
        self.scales[page, :, u, self._scale_bytes(r)] = scales.T

    def get(self, page, pos):
        u, r = divmod(pos, 16)
        raw = self.codes[page, :, u, self._code_bytes(r)].T
        if self.fmt == MXFP4:
            raw = np.stack((raw & 15, raw >> 4), -1).reshape(self.heads, self.dim)
        return dequantise(raw, self.scales[page, :, u, self._scale_bytes(r)].T, self.fmt)


class Keys(Side):
    def _code_bytes(self, r):
        row = self.dim * self.fmt // 8
        piece = 8 if row == 32 else 16
        b = np.arange(row)
        return (b // piece) * (16 * piece) + r * piece + b % piece

    def _scale_bytes(self, r):
        return r * (self.dim // 32) + np.arange(self.dim // 32)


class Values(Side):
    def _code_bytes(self, r):
        part = self.dim * self.fmt // 8 // 16        # bytes of a token in one of 16 rows
        per = min(4, 16 // part)                     # tokens of a slot
        quad, t = divmod(r, 4)
        slot, t = divmod(t, per)
        b = np.arange(16 * part)
        row, k = b // part, b % part
        return (((slot * 4 + quad) * 16 + row) * per + t) * part + k

    def _scale_bytes(self, r):
        quad, t = divmod(r, 4)
        return (quad * (self.dim // 32) + np.arange(self.dim // 32)) * 4 + t


def page_of(table, pages, page_tokens, s, pos):
    k = pos // page_tokens
    if k >= table.shape[1]:
        return -1
    p = int(table[s, k])
    return p if 0 <= p < pages else -1


def append(side, table, offsets, past, x):
    """Quantise the new tokens x [tokens, heads, D] into a side's planes."""
    codes, scales = quantise(x, side.fmt)
    for s in range(len(past)):
        for i in range(offsets[s + 1] - offsets[s]):
            pos = past[s] + i
            p = page_of(table, len(side.codes), side.page_tokens, s, pos)
            if p >= 0:
                side.put(p, pos % side.page_tokens, codes[offsets[s] + i], scales[offsets[s] + i])


def held(side, table, s, count):
    """float64 [count, heads, D] of a sequence's first positions and which of
    them have a page (zeros where none)."""
    out = np.zeros((count, side.heads, side.dim))
    some = np.zeros(count, bool)
    for pos in range(count):
        p = page_of(table, len(side.codes), side.page_tokens, s, pos)
        if p >= 0:
            out[pos], some[pos] = side.get(p, pos % side.page_tokens), True
    return out, some


def attention(keys, values, table, offsets, past, q, scale, window=0, tree=None):
    """q float64 [tokens, q_heads, D] -> (out, lse, spread, zmax): the attention, its
    log-sum-exp, and for error bounds sum_j p_j |v_j| (laid out as out) and the
    largest scale * sum_d |q_d k_d| of a row's allowed keys."""
    tokens, q_heads, dim = q.shape
    group = q_heads // keys.heads
    out, spread = np.zeros_like(q), np.zeros_like(q)
    lse, zmax = np.full((tokens, q_heads), -np.inf), np.zeros((tokens, q_heads))
    for s in range(len(past)):
        n = offsets[s + 1] - offsets[s]
        if n == 0:
            continue
        k, some = held(keys, table, s, past[s] + n)
        v, _ = held(values, table, s, past[s] + n)
        for i in range(n):
            t, pos = offsets[s] + i, past[s] + i
            j = np.arange(past[s] + n)
            ok = j <= pos
            if tree is not None:
                ok = (j < past[s]) | ((j - past[s] >= 0) & (j - past[s] < 64) &
                                      ((int(tree[t]) >> np.clip(j - past[s], 0, 63).astype(object)) & 1).astype(bool))
            if window:
                ok &= j > pos - window
            ok &= some
            if not ok.any():
                continue
            for h in range(q_heads):
                kk, vv = k[ok, h // group], v[ok, h // group]
                z = scale * (kk @ q[t, h])
                m = z.max()
                e = np.exp(z - m)
                out[t, h] = (e @ vv) / e.sum()
                spread[t, h] = (e @ np.abs(vv)) / e.sum()
                lse[t, h] = m + np.log(e.sum())
                zmax[t, h] = scale * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, spread, zmax
