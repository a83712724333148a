"""Helpers of the tests of rotated, scored and drafted tokens over the 8-bit cache."""
import numpy as np
import torch

import fp4_kv_cache_rope_gb300 as K
from oracle import kv8 as O

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def ints(x, device="cuda"):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=device)


def tables(positions, R, theta=10000.0):
    """cos and sin [positions, R / 2], fp32 (numpy)."""
    a = np.arange(positions, dtype=np.float64)[:, None] * theta ** (-2.0 * np.arange(R // 2) / R)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


def rope(positions, R, first=0, style=O.HALVES, device="cuda"):
    c, s = tables(positions, R)
    return K.Rope(torch.from_numpy(c), torch.from_numpy(s), first=first, style=style, device=device), c, s


def rotated(x, pos, c, s, first, style):
    """Rows x [B, T, heads, D] of any type at pos [B][T]: fp32 on the host."""
    y = np.stack([O.rotate(x[b].float().numpy(), pos[b], c, s, first, style) for b in range(len(x))])
    return torch.from_numpy(y)


def tree(rng, B, T, chain=0.35):
    """Parents [B][T]: the token before, or any earlier one, or none."""
    return [[-1 if i == 0 else i - 1 if rng.random() < chain else int(rng.integers(-1, i))
             for i in range(T)] for _ in range(B)]


def scored_want(pair, q, b, h, G, ql, scale, dtype, cap=0.0, window=0, sink=0, slopes=None, prefix=0,
                k=None, v=None, parent=None):
    """The oracle's (o, lse, tol, ltol) for the first ql queries of sequence b and the heads
    of K/V head h; with parent, drafted tokens whose rows are k, v [T, D]."""
    n = pair.len[b]
    kc, vc = (pair.seq[b, h, s].values() for s in "kv")
    j = np.arange(n)
    if parent is None:
        p = n - ql + np.arange(ql)
        see = O.sees(p, j, n, window, sink, prefix)
    else:
        paths = [O.path_to(parent, i) for i in range(ql)]
        p = n + np.array([len(x) - 1 for x in paths], dtype=np.int64)
        see = O.sees(p, j, n, window, sink)
        on = np.zeros((ql, ql), bool)
        for i, x in enumerate(paths):
            for a in x:
                on[i, a] = not window or p[a] > p[i] - window or p[a] < sink
        see = np.concatenate([see, on], 1)
        j = np.concatenate([j, p])
        kc, vc = np.concatenate([kc, k[:ql]]), np.concatenate([vc, v[:ql]])
    qq = q[b, :ql, h * G:(h + 1) * G].double().numpy()
    sl = None if slopes is None else slopes[h * G:(h + 1) * G]
    return O.attend(qq, kc, vc, scale, see, p[:, None] - j, cap, sl, HALF[dtype])


def check_attention(got, lse, want, where=""):
    """out [T, G, D] and lse [T, G] on the host within the oracle's bounds."""
    o, l, tol, ltol = want
    x, y = got.double().numpy(), lse.double().numpy()
    assert np.isfinite(x).all(), where
    none = np.isinf(l)
    assert (x[none] == 0).all() and (y[none] == -np.inf).all(), where
    bad = np.abs(x - o) > tol
    assert not bad.any(), (where, int(bad.sum()), float((np.abs(x - o) / tol).max()))
    with np.errstate(invalid="ignore"):
        off = np.abs(y - l)[~none] > ltol[~none]
    assert not off.any(), (where, "lse", float(np.abs(y - l)[~none].max()))
