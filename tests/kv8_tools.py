"""Helpers of the 8-bit K/V cache's tests: a device cache beside its oracle."""
import numpy as np
import torch

import fp4_kv_cache_rope_gb300 as K
from oracle import kv8 as O

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


class Pair:
    """A Cache8 whose unheld rows hold garbage (NaN codes for E4M3), with one
    oracle sequence per (sequence, head, side)."""

    def __init__(self, B, Hkv, D, max_len, block, page, fmt, seed=0, mass=True, device="cuda"):
        rng = np.random.default_rng(seed)
        self.B, self.Hkv, self.D, self.block, self.fmt, self.rng = B, Hkv, D, block, fmt, rng
        table, pages = None, 0
        if page:
            per_seq = -(-max_len // page)
            pages = B * per_seq + 2
            table = torch.from_numpy(rng.permutation(pages)[: B * per_seq].reshape(B, per_seq)
                                     .astype(np.int32))
        else:
            max_len = -(-max_len // block) * block
        self.c = K.Cache8(B, Hkv, D, max_len, block=block, page_size=page, page_table=table,
                          num_pages=pages, fmt=fmt, mass=mass, device=device)
        self.c.k_codes.fill_(0x7F)
        self.c.v_codes.fill_(0x7F)
        self.c.k_scales.fill_(float("nan"))
        self.c.v_scales.fill_(float("inf"))
        if mass:
            self.c.mass.fill_(float("nan"))
        self.table = table
        self.seq = {(b, h, s): O.Seq(block, fmt, D) for b in range(B) for h in range(Hkv)
                    for s in "kv"}
        self.len = [0] * B

    def rows(self, T, heads, dtype, size=1.0):
        """Random rows [B, T, heads, D] of uneven channels and tokens, on the host."""
        r = self.rng
        x = r.standard_normal((self.B, T, heads, self.D)) * np.exp(
            0.7 * r.standard_normal((1, 1, heads, self.D))) * np.exp(
            0.5 * r.standard_normal((self.B, T, heads, 1))) * size
        return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])

    def append(self, k, v, ws, lens=None, start=None, on_gpu=None):
        dev = self.c.device
        ints = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
        kk, vv = on_gpu if on_gpu is not None else (k.to(dev), v.to(dev))
        K.kv8_append(self.c, kk, vv, ws, new_len=ints(lens), start=ints(start))
        for b in range(self.B):
            t = k.shape[1] if lens is None else lens[b]
            s = self.len[b] if start is None else start[b]
            for h in range(self.Hkv):
                for side, x in (("k", k), ("v", v)):
                    self.seq[b, h, side].append(x[b, :t, h].double().numpy(), s)
            self.len[b] = s + t

    def at(self, name, b, h):
        """Rows (or scales) of one sequence and head in position order, on the host."""
        x = getattr(self.c, name)
        pages = [b] if self.table is None else self.table[b].tolist()
        return torch.cat([x[p, h] for p in pages]).cpu().numpy()

    def check(self):
        """Everything held equals the oracle's; nothing else was written."""
        assert self.c.seq_len.tolist() == self.len
        for (b, h, side), s in self.seq.items():
            n, nb = self.len[b], -(-self.len[b] // self.block)
            codes = self.at(side + "_codes", b, h)
            assert np.array_equal(O.decode(codes[:n], self.fmt), s.codes[:n]), (b, h, side)
            assert np.array_equal(self.at(side + "_scales", b, h)[:nb].astype(np.float64),
                                  s.scales[:nb]), (b, h, side)

    def untouched_behind(self, ends):
        for (b, h, side) in self.seq:
            assert (self.at(side + "_codes", b, h)[ends[b]:] == 0x7F).all(), (b, h, side)
        if self.table is not None:
            used = set(self.table.flatten().tolist())
            for p in set(range(self.c.num_pages)) - used:
                assert (self.c.k_codes[p] == 0x7F).all() and (self.c.v_codes[p] == 0x7F).all()

    def set_mass(self, w):
        """mass of every held row, w[b][h] arrays."""
        for b in range(self.B):
            for h in range(self.Hkv):
                x = torch.from_numpy(np.asarray(w[b][h], np.float32)).to(self.c.device)
                if self.table is None:
                    self.c.mass[b, h, : len(x)] = x
                else:
                    ps = self.c.page_size
                    for i in range(0, len(x), ps):
                        part = x[i:i + ps]
                        self.c.mass[int(self.table[b, i // ps]), h, : len(part)] = part


def attention_bounds(q, p, b, h, G, ql, scale, out_half):
    """The oracle's attention of sequence b, K/V head h and element-wise bounds.

    A logit is a sum of D exact products in fp32: off by at most
    ds = D 2^-23 L, L = scale sum |q k| (two roundings' worth per addition,
    for an accumulator that truncates), plus its multiplication by the logit
    factor, 2 2^-24 L.  A weight is exp of it: relative error 2 ds (its own
    logit's and the maximum's) + 2^-20 (exp2, its argument's rounding), and is
    rounded to f16 once, 2^-11.  The output is off by that times A = sum p |v|,
    by the fp32 additions of n terms and of the normaliser's, 2 n 2^-23 A, and
    by its own rounding: half a step, which is out_half of it and, for f16 below
    2^-14, where the steps are 2^-24 throughout, 2^-25.  Weights far below the largest lose bits: a weight
    is held in steps of 2^-31 of the running maximum's (f16's smallest step 2^-24
    over the factor 2^7), an error of half that times max |v| each; and a code times its block's share of the largest scale is held
    in steps of 2^-24 of that scale, at most max |v| / 63: 2^-25 / 63 < 2^-30 of it.
    """
    n = p.len[b]
    k, v = (p.seq[b, h, s].values() for s in "kv")
    o, lse, a, big = O.attention(q, k, v, scale)
    ds = (p.D + 2) * 2.0 ** -23 * big
    rel = 2 * ds + 2.0 ** -20 + 2.0 ** -11 + 2 * n * 2.0 ** -23
    vmax = np.abs(v).max() if n else 0.0
    tol = a * rel[..., None] + (n * 2.0 ** -32 + 2.0 ** -30) * vmax
    tol = tol + out_half * (np.abs(o) + tol) + (2.0 ** -25 if out_half == 2.0 ** -11 else 1e-30)
    ltol = ds + 2.0 ** -20 + n * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))
    return o, lse, tol, ltol
