"""Run by test_gpu_kv8_scored_timeout.py: calls on the library that the command line
names, with waits that run out."""
import ctypes
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
load = ctypes.CDLL
ctypes.CDLL = lambda name, *a, **k: load(
    sys.argv[1] if name and os.path.basename(str(name)) == "libcsa2.so" else name, *a, **k)

import numpy as np  # noqa: E402
import torch  # noqa: E402

import fp4_kv_cache_rope_gb300 as K  # noqa: E402
from kv8_more_tools import ints, tree  # noqa: E402
from kv8_tools import Pair  # noqa: E402

assert os.path.samefile(K._lib._name, sys.argv[1])


def run(T, G, D, lens):
    Hkv = 2
    H = Hkv * G
    p = Pair(2, Hkv, D, max(lens), 64, 64, K.KV8_E4M3, seed=45, mass=False)
    ws = p.c.tree_workspace(T, H)
    p.append(*(p.rows(max(lens), Hkv, "bf16") for _ in "kv"), ws, lens=lens)
    q, k, v = p.rows(T, H, "bf16", 0.7).cuda(), p.rows(T, Hkv, "bf16").cuda(), p.rows(T, Hkv, "bf16").cuda()
    par = ints(tree(p.rng, 2, T))
    q_len = ints([T, T - 1])
    slopes = torch.full((H,), 0.1, device="cuda")
    forms = [K.Scores(window=300), K.Scores(cap=20.0), K.Scores(slopes=slopes), K.Scores(cap=20.0, slopes=slopes)]

    def attend(form, drafted):
        o, ls = torch.full_like(q, 7.0), torch.full((2, T, H), 7.0, device="cuda")
        if drafted:
            K.kv8_attn_tree(p.c, q, k, v, par, o, ws, lse=ls, q_len=q_len, scores=form)
        else:
            K.kv8_attn_scored(p.c, q, o, ws, form, lse=ls, q_len=q_len)
        torch.cuda.synchronize()
        return o, ls

    n = 0
    for form in forms:
        for drafted in (False, True):
            out, lse = attend(form, drafted)
            assert K.get_status(ws) == 0
            try:
                K.set_wait_limit(1)
                a, b = attend(form, drafted)
            finally:
                K.set_wait_limit(0)
            assert K.get_status(ws) == K.DEV_TIMEOUT
            K.reset_status(ws)
            assert (a[1, T - 1:] == 7.0).all() and (b[1, T - 1:] == 7.0).all()
            again, lse2 = attend(form, drafted)
            assert torch.equal(again, out) and torch.equal(lse2, lse)
            assert K.get_status(ws) == 0
            n += 1
    return n


print(sum(run(*c) for c in ((200, 4, 128, [2000, 900]), (130, 2, 64, [5000, 131]))), "calls reported")
