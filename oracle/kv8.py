"""The 8-bit K/V cache of grouped heads (oracle side), in fp64.

A sequence is held as one array of rows per head: codes (their values as
float64), and one scale per block of rows.  Scales are powers of two, so every
value code * scale is exact in float64.

Parity: codes, scales, kept rows and moved weights are exact; attention, its log
normaliser and the accumulated weights are fp64 values for a tolerance.
"""
from __future__ import annotations

import math

import numpy as np

from . import formats

E4M3, INT8 = 0, 1
QMAX = {E4M3: 448.0, INT8: 127.0}


def scale_of(amax: float, fmt: int) -> float:
    """The smallest power of two s >= 2^-126 with amax <= qmax * s; 0 for 0."""
    if amax == 0.0:
        return 0.0
    s = 2.0 ** -126
    while amax > QMAX[fmt] * s:
        s *= 2.0
    return s


def nearest(y, fmt: int):
    """The format's nearest value, ties to even, saturating at +-qmax."""
    y = np.clip(np.asarray(y, np.float64), -QMAX[fmt], QMAX[fmt])
    if fmt == INT8:
        return np.rint(y)
    mag = formats.e4m3_magnitude(formats._nearest_code(np.abs(y), formats._E4M3_FINITE))
    return np.copysign(mag, y)


def decode(codes, fmt: int):
    """Stored bytes -> values of the codes."""
    codes = np.asarray(codes, np.uint8)
    return codes.view(np.int8).astype(np.float64) if fmt == INT8 else formats.e4m3_decode(codes)


class Seq:
    """One head's rows of one side (K or V): code values [n, D], scales [blocks]."""

    def __init__(self, block: int, fmt: int, dim: int):
        self.block, self.fmt = block, fmt
        self.codes = np.zeros((0, dim))
        self.scales = np.zeros(0)

    def values(self):
        return self.codes * np.repeat(self.scales, self.block)[: len(self.codes), None]

    def append(self, x, start: int | None = None):
        """Rows x (any finite or non-finite fp64 values) at `start` (default: the end)."""
        x = np.asarray(x, np.float64)
        if start is not None:
            self.codes = self.codes[:start]
        n, blk = len(self.codes), self.block
        nblocks = -(-(n + len(x)) // blk)
        self.scales = np.concatenate([self.scales[: -(-n // blk)],
                                      np.zeros(max(0, nblocks - -(-n // blk)))])
        self.codes = np.concatenate([self.codes, np.zeros_like(x)])
        for b in range(n // blk, nblocks):
            lo, hi = max(n, b * blk), min(n + len(x), (b + 1) * blk)
            if lo >= hi:
                continue
            new = x[lo - n: hi - n]
            fin = np.abs(new[np.isfinite(new)])
            s0 = self.scales[b] if lo > b * blk else 0.0
            s1 = max(s0, scale_of(float(fin.max()) if fin.size else 0.0, self.fmt))
            if s1 > s0 > 0.0:
                self.codes[b * blk: lo] = nearest(self.codes[b * blk: lo] * (s0 / s1), self.fmt)
            if s1 > 0.0:
                y = np.where(np.isnan(new), 0.0, new) / s1
                self.codes[lo:hi] = nearest(y, self.fmt)
            self.scales[b] = s1

    def keep(self, rows):
        """The rows that stay (ascending), in blocks of their own."""
        rows = np.asarray(rows)
        vals = self.values()[rows]
        out = Seq(self.block, self.fmt, self.codes.shape[1])
        out.append(vals)
        for b in range(len(out.scales)):
            sl = slice(b * self.block, min(len(rows), (b + 1) * self.block))
            if np.array_equal(rows[sl], np.arange(sl.start, sl.stop)):
                out.scales[b] = self.scales[b]
                out.codes[sl] = self.codes[sl]
        return out


def visible(n: int, ql: int, i: int) -> int:
    """How many of n rows query i of the last ql sees."""
    return max(0, min(n, n - ql + i + 1))


def attention(q, k, v, scale: float):
    """q [ql, G, D] over rows k, v [n, D]: (o, lse, A, L) with the sums
    A = sum p |v| and the largest L = scale * sum |q| |k| that error bounds use."""
    ql, G, D = q.shape
    n = len(k)
    o, a = np.zeros((ql, G, v.shape[1])), np.zeros((ql, G, v.shape[1]))
    lse, big = np.full((ql, G), -np.inf), np.zeros((ql, G))
    for i in range(ql):
        m = visible(n, ql, i)
        if m == 0:
            continue
        x = scale * (q[i] @ k[:m].T)
        top = x.max(1, keepdims=True)
        e = np.exp(x - top)
        z = e.sum(1, keepdims=True)
        lse[i] = (top + np.log(z))[:, 0]
        o[i], a[i] = (e / z) @ v[:m], (e / z) @ np.abs(v[:m])
        big[i] = (scale * (np.abs(q[i]) @ np.abs(k[:m]).T)).max(1)
    return o, lse, a, big


def mass(q, lse, k, scale: float):
    """Weight of each of the rows k [n, D] from the queries q [ql, G, D]."""
    ql, n = len(q), len(k)
    w = np.zeros(n)
    for i in range(ql):
        m = visible(n, ql, i)
        fin = np.isfinite(lse[i])
        if m and fin.any():
            w[:m] += np.exp(scale * (q[i][fin] @ k[:m].T) - lse[i][fin][:, None]).sum(0)
    return w


def evict(weight, n: int, keep: int, sink: int, recent: int):
    """Positions that stay, ascending."""
    if n <= keep:
        return np.arange(n)
    w = np.asarray(weight[:n], np.float64).copy()
    w[np.isnan(w)] = math.inf
    nan_first = np.isnan(np.asarray(weight[:n], np.float64))
    mid = np.arange(sink, n - recent)
    # largest first, NaN above everything, equal ones by position
    order = sorted(mid, key=lambda j: (not nan_first[j], -w[j], j))
    take = order[: keep - sink - recent]
    return np.array(sorted(set(range(sink)) | set(range(n - recent, n)) | set(take)), dtype=np.int64)
