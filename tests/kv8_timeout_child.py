"""Run by test_gpu_kv8_timeout.py: the calls of the binding on the library that
the command line names, with waits that run out."""
import ctypes
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "tests")]
load = ctypes.CDLL
ctypes.CDLL = lambda name, *a, **k: load(
    sys.argv[1] if name and os.path.basename(str(name)) == "libcsa2.so" else name, *a, **k)

import torch  # noqa: E402

import fp4_kv_cache_rope_gb300 as K  # noqa: E402
from kv8_tools import Pair  # noqa: E402

assert os.path.samefile(K._lib._name, sys.argv[1])


def run(T, G, D, lens):
    Hkv = 2
    p = Pair(2, Hkv, D, max(lens), 64, 64, K.KV8_E4M3, seed=45)
    ws = p.c.workspace(T, Hkv * G)
    p.append(*(p.rows(max(lens), Hkv, "bf16") for _ in "kv"), ws, lens=lens)
    q = p.rows(T, Hkv * G, "bf16", 0.7).cuda()
    q_len = torch.tensor([T, min(T, lens[1]) - 1], dtype=torch.int32, device="cuda")
    p.c.mass.fill_(0.5)
    held = torch.zeros_like(p.c.mass, dtype=torch.bool)
    for b in range(2):
        for i, page in enumerate(p.table[b].tolist()):
            held[page, :, : max(0, min(64, lens[b] - 64 * i))] = True

    def attend():
        o, ls = torch.full_like(q, 7.0), torch.full((2, T, Hkv * G), 7.0, device="cuda")
        K.kv8_attn(p.c, q, o, ws, lse=ls, q_len=q_len)
        torch.cuda.synchronize()
        return o, ls

    out, lse = attend()

    def weigh():
        K.kv8_mass(p.c, q, lse, ws, q_len=q_len, decay=0.0)
        torch.cuda.synchronize()
        return p.c.mass.clone(), None

    want = weigh()[0]
    assert K.get_status(ws) == 0
    for call in (attend, weigh):
        try:
            K.set_wait_limit(1)
            a, b = call()
        finally:
            K.set_wait_limit(0)
        assert K.get_status(ws) == K.DEV_TIMEOUT
        K.reset_status(ws)
        if call is weigh:
            assert (a[~held] == 0.5).all()
            continue
        for s in range(2):
            assert (a[s, int(q_len[s]):] == 7.0).all() and (b[s, int(q_len[s]):] == 7.0).all()
    again, lse2 = attend()
    assert torch.equal(again, out) and torch.equal(lse2, lse) and torch.equal(weigh()[0], want)
    assert K.get_status(ws) == 0
    return 2


print(sum(run(*c) for c in ((600, 4, 128, [2000, 900]), (130, 2, 64, [5000, 131]),
                            (90, 8, 128, [640, 90]))), "calls reported")
