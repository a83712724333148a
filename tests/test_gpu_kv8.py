"""GPU parity of the 8-bit K/V cache's operators with the fp64 oracle: stored
bytes, kept rows and moved weights exactly; attention, its log normaliser and
the accumulated weights within bounds derived in kv8_tools.attention_bounds."""
import math
import os
import re

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp4_kv_cache_rope_gb300 as K  # noqa: E402
from oracle import kv8 as O  # noqa: E402
from kv8_tools import DT, Pair, attention_bounds  # noqa: E402

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


# --------------------------------------------------------------------- append
@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
@pytest.mark.parametrize("Hkv,D,block,page,dtype", [
    (2, 128, 64, 64, "bf16"), (1, 64, 16, 16, "f16"), (3, 128, 16, 48, "f32"),
    (8, 64, 128, 0, "bf16"), (20, 128, 32, 128, "f32"), (4, 64, 64, 0, "f32")])
def test_append(fmt, Hkv, D, block, page, dtype):
    p = Pair(3, Hkv, D, 400, block, page, fmt, seed=11)
    ws = p.c.workspace(1, Hkv)
    # a prompt, tokens one by one into half-filled blocks (some raise the scale),
    # nothing, a few, a ragged chunk over several blocks
    for step, (T, lens) in enumerate([(70, [70, 1, 33]), (1, None), (1, [0, 1, 1]), (3, None),
                                      (0, None), (8, [8, 5, 0]), (9, None), (150, [0, 150, 97])]):
        k, v = (p.rows(T, Hkv, dtype, 2.0 ** (step % 3)) for _ in "kv")
        p.append(k, v, ws, lens)
        p.check()
        p.untouched_behind(p.len)
    for b in range(3):
        for h in range(Hkv):
            m = p.at("mass", b, h)
            assert (m[: p.len[b]] == 0).all() and np.isnan(m[p.len[b]:]).all()
    assert K.get_status(ws) == 0


def test_append_strided_slices_of_a_fused_projection():
    p = Pair(2, 2, 64, 128, 32, 32, O.E4M3, seed=3, mass=False)
    ws = p.c.workspace(1, 2)
    for T in (40, 2):
        fused = p.rows(T, 8, "bf16").cuda()
        k, v = fused[:, :, 4:6], fused[:, :, 6:]
        p.append(k.cpu(), v.cpu(), ws, on_gpu=(k, v))
        p.check()
    # heads in front of tokens, and one row for all tokens (stride 0)
    x = p.rows(2, 9, "f16").cuda().transpose(1, 2)
    y = p.rows(1, 2, "f16").cuda().expand(2, 9, 2, 64)
    p.append(x.cpu(), y.cpu(), ws, on_gpu=(x, y))
    p.check()


@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
def test_append_at_a_start_drops_what_was_behind(fmt):
    p = Pair(2, 2, 64, 200, 32, 0, fmt, seed=5)
    ws = p.c.workspace(1, 2)
    p.append(p.rows(100, 2, "f32"), p.rows(100, 2, "f32"), ws)
    for T, start in [(3, [97, 50]), (40, [64, 10]), (0, [70, 3]), (5, [70, 0]), (60, [0, 5])]:
        p.append(p.rows(T, 2, "f32", 4.0), p.rows(T, 2, "f32", 0.1), ws, start=start)
        p.check()


@pytest.mark.parametrize("T", [3, 90])
def test_append_with_seq_len_as_start(T):
    p = Pair(3, 5, 64, 400, 16, 16, O.E4M3, seed=8)
    ws = p.c.workspace(1, 5)
    for step in range(3):
        k, v = p.rows(T, 5, "f16"), p.rows(T, 5, "f16")
        K.kv8_append(p.c, k.cuda(), v.cuda(), ws, start=p.c.seq_len)
        for b in range(3):
            for h in range(5):
                for s, x in (("k", k), ("v", v)):
                    p.seq[b, h, s].append(x[b, :, h].double().numpy())
            p.len[b] += T
        p.check()


@pytest.mark.parametrize("T", [2, 60])
def test_append_values_at_the_edges(T):
    for fmt in (O.E4M3, O.INT8):
        p = Pair(1, 1, 64, 256, 16, 16, fmt, seed=6)
        ws = p.c.workspace(1, 1)
        k = torch.zeros(1, T, 1, 64)
        v = p.rows(T, 1, "f32") * 2.0 ** -120
        k[0, 1, 0, :8] = torch.tensor([O.QMAX[fmt], -3.0, 0.5, 2.0 ** -149, 2.0 ** -126, 1e-20, -0.0, 1.0])
        p.append(k, v, ws)
        p.append(torch.zeros(1, T, 1, 64), torch.full((1, T, 1, 64), 3.0e38), ws)
        p.check()
        assert K.get_status(ws) == 0
        k = p.rows(T, 1, "f32")
        k[0, 0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 2.0])
        v = torch.full((1, T, 1, 64), math.inf)
        p.append(k, v, ws)
        p.check()
        assert K.get_status(ws) == K.DEV_NONFINITE


@pytest.mark.parametrize("T", [4, 50])
def test_append_past_the_end_and_bad_pages(T):
    p = Pair(2, 2, 64, 64, 16, 16, O.E4M3, seed=7)
    ws = p.c.workspace(1, 2)
    p.append(p.rows(62, 2, "bf16"), p.rows(62, 2, "bf16"), ws, lens=[62, 10])
    k, v = p.rows(T, 2, "bf16"), p.rows(T, 2, "bf16")
    K.kv8_append(p.c, k.cuda(), v.cuda(), ws)
    for h in range(2):
        for s, x in (("k", k), ("v", v)):
            p.seq[0, h, s].append(x[0, :2, h].double().numpy())
            p.seq[1, h, s].append(x[1, :T, h].double().numpy())
    p.len = [64, 10 + T]
    p.check()
    assert K.get_status(ws) == K.DEV_OVERFLOW
    K.reset_status(ws)
    for start in (-1, 65):
        K.kv8_append(p.c, k.cuda(), v.cuda(), ws,
                     start=torch.tensor([start, 10], dtype=torch.int32, device="cuda"))
        assert K.get_status(ws) == K.DEV_OVERFLOW
        K.reset_status(ws)
        assert p.c.seq_len.tolist() == [0 if start < 0 else 64, 10 + T]
    p.len[0] = 0
    for h in range(2):
        for s in "kv":
            p.seq[0, h, s].append(np.zeros((0, 64)), 0)
    p.c.page_table[1, 0] = p.c.num_pages
    before = p.c.k_codes.clone()
    K.kv8_append(p.c, k.cuda(), v.cuda(), ws, start=torch.zeros(2, dtype=torch.int32, device="cuda"),
                 new_len=torch.tensor([0, 3], dtype=torch.int32, device="cuda"))
    assert K.get_status(ws) == K.DEV_BAD_PAGE
    assert torch.equal(before, p.c.k_codes)


# ------------------------------------------------------------------ attention
def filled(B, Hkv, D, lens, block, page, fmt, seed, cap=None):
    cap = cap or max(max(lens), 1) + 5
    p = Pair(B, Hkv, D, cap, block, page, fmt, seed=seed)
    ws = p.c.workspace(1, Hkv)
    T = max(max(lens), 1)
    p.append(p.rows(T, Hkv, "f32"), p.rows(T, Hkv, "f32"), ws, lens=lens)
    assert K.get_status(ws) == 0
    return p


def run_attention(p, q, G, q_lens=None, scale=0.0, out=None):
    """kv8_attn against the oracle; q [B, T, H, D] on the host."""
    B, T, H, D = q.shape
    ws = p.c.workspace(T, H)
    ws[256:] = 0xFF          # an earlier call's leavings: NaN
    qd = q.cuda() if q.device.type == "cpu" else q
    out = torch.full((B, T, H, D), 7.0, dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((B, T, H), 7.0, device="cuda")
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device="cuda")
    K.kv8_attn(p.c, qd, out, ws, lse=lse, q_len=ql, softmax_scale=scale)
    assert K.get_status(ws) == 0
    o, ls = out.cpu().double().numpy(), lse.cpu().double().numpy()
    sc = scale if scale > 0 else 1.0 / math.sqrt(D)
    qn = q.cpu().double().numpy()
    half = HALF["bf16" if q.dtype == torch.bfloat16 else "f16"]
    for b in range(B):
        n_q = T if q_lens is None else q_lens[b]
        assert (o[b, n_q:] == 7.0).all() and (ls[b, n_q:] == 7.0).all()
        for h in range(p.Hkv):
            hs = slice(h * G, (h + 1) * G)
            ro, rl, tol, ltol = attention_bounds(qn[b, :n_q, hs], p, b, h, G, n_q, sc, half)
            err = np.abs(o[b, :n_q, hs] - ro)
            at = np.unravel_index(np.argmax(err / tol), err.shape) if err.size else None
            assert (err <= tol).all(), (b, h, at, err[at], tol[at], ro[at])
            fin = np.isfinite(rl)
            assert np.array_equal(fin, np.isfinite(ls[b, :n_q, hs]))
            assert (ls[b, :n_q, hs][~fin] == -np.inf).all()
            assert (np.abs(ls[b, :n_q, hs][fin] - rl[fin]) <= ltol[fin]).all()
    return qd, lse


SHAPES = [
    # B, Hkv, G, D, lens, T, q_lens, block, page, dtype
    (1, 1, 1, 64, [1], 1, None, 16, 16, "bf16"),
    (2, 2, 7, 128, [1000, 129], 1, None, 64, 64, "bf16"),
    (3, 2, 8, 128, [0, 127, 4000], 1, None, 64, 64, "f16"),
    (5, 1, 3, 64, [31, 32, 33, 300, 2], 1, [1, 0, 1, 1, 1], 32, 96, "bf16"),
    (2, 4, 4, 64, [513, 700], 5, None, 128, 0, "f16"),
    (2, 2, 16, 128, [600, 90], 2, [2, 1], 16, 16, "bf16"),
    (2, 1, 5, 128, [3, 40], 9, None, 16, 32, "f16"),       # the first queries see nothing
    (40, 2, 2, 64, [1 + 37 * i % 290 for i in range(40)], 1, None, 16, 48, "bf16"),
    (1, 2, 4, 128, [300], 300, None, 32, 64, "bf16"),
    (2, 2, 3, 64, [500, 131], 131, [100, 131], 16, 16, "f16"),
    (1, 1, 1, 128, [257], 257, None, 128, 0, "bf16"),
    (1, 8, 20, 64, [200], 70, None, 64, 64, "f16"),
    (1, 2, 1, 64, [640], 520, None, 32, 32, "bf16"),
    (1, 2, 13, 128, [5000], 5, None, 64, 64, "bf16"),          # 65 rows: key splits
    (2, 1, 16, 64, [3001, 40], 9, [9, 3], 128, 256, "f16"),    # 144 rows, splits with nothing
    (3, 2, 8, 128, [0, 1, 700], 33, [33, 20, 0], 16, 48, "bf16"),
    (2, 1, 2, 128, [1100, 130], 129, None, 64, 0, "f16"),
]


@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention_and_mass(i, fmt):
    B, Hkv, G, D, lens, T, q_lens, block, page, dtype = SHAPES[i]
    p = filled(B, Hkv, D, lens, block, page, fmt, seed=100 + i)
    q = p.rows(T, Hkv * G, dtype, 0.7)
    qd, lse = run_attention(p, q, G, q_lens)
    check_mass(p, q, qd, lse, G, q_lens)


def check_mass(p, q, qd, lse, G, q_lens):
    B, T, H, D = q.shape
    ws = p.c.workspace(T, H)
    ql = None if q_lens is None else torch.tensor(q_lens, dtype=torch.int32, device="cuda")
    sc = 1.0 / math.sqrt(D)
    qn, ln = q.double().numpy(), lse.cpu().double().numpy()
    w = {}
    for b in range(B):
        n_q = T if q_lens is None else q_lens[b]
        for h in range(p.Hkv):
            hs = slice(h * G, (h + 1) * G)
            k = p.seq[b, h, "k"].values()
            w[b, h] = O.mass(qn[b, :n_q, hs], ln[b, :n_q, hs], k, sc)
            # a weight's relative error: its logit's (see attention_bounds) and
            # exp2's, whose argument is rounded once more; lse is the given one,
            # times log2 e in fp32; then fp32 additions of T G weights
            big = sc * (np.abs(qn[b, :n_q, hs]).reshape(-1, D) @ np.abs(k).T).max() if n_q and len(k) else 0.0
            fin = np.isfinite(ln[b, :n_q, hs])
            top = np.abs(ln[b, :n_q, hs][fin]).max() if fin.any() else 0.0
            w[b, h, "rel"] = (D + 4) * 2.0 ** -23 * big + 2.0 ** -22 * top + 2.0 ** -20 + (
                n_q * G + 2) * 2.0 ** -23
    for decay, f in ((0.0, 1.0), (1.0, 2.0), (0.25, 1.5)):
        K.kv8_mass(p.c, qd, lse, ws, q_len=ql, decay=decay)
        assert K.get_status(ws) == 0
        for b in range(B):
            for h in range(p.Hkv):
                m, n = p.at("mass", b, h), p.len[b]
                assert np.isnan(m[n:]).all()
                assert (np.abs(m[:n] - f * w[b, h]) <= f * w[b, h] * w[b, h, "rel"] + 1e-36).all()


@pytest.mark.parametrize("T,D,fmt", [(435, 128, O.E4M3), (333, 64, O.INT8), (90, 128, O.INT8), (30, 128, O.E4M3)])
def test_weights_of_many_query_tiles_sum_to_one_per_query_and_repeat(T, D, fmt):
    B, Hkv, G, n = 7, 4, 13, 577
    p = filled(B, Hkv, D, [n] * B, 32, 32, fmt, seed=41)
    q = p.rows(T, Hkv * G, "f16", 0.7).cuda()
    ws = p.c.workspace(T, Hkv * G)
    out = torch.empty_like(q)
    lse = torch.empty(B, T, Hkv * G, device="cuda")
    K.kv8_attn(p.c, q, out, ws, lse=lse)
    first = None
    for _ in range(12):
        K.kv8_mass(p.c, q, lse, ws, decay=0.0)
        first = p.c.mass.clone() if first is None else first
        assert torch.equal(p.c.mass.view(torch.int32), first.view(torch.int32))
    assert K.get_status(ws) == 0
    # a weight is off by its logit's error (D + 4 roundings of at most 2^-23 of the
    # sum of its products' magnitudes, at most |q| |k|), here and in lse, by lse's
    # own roundings, and by the additions: T G of them
    big = 0.0
    for b in range(B):
        for h in range(Hkv):
            k = p.seq[b, h, "k"].values()
            big = max(big, (q[b, :, h * G:(h + 1) * G].double().norm(dim=-1).max().item()
                            * np.linalg.norm(k, axis=-1).max() / math.sqrt(D)))
    rel = 2 * ((D + 4) * 2.0 ** -23 * big + 2.0 ** -22 * lse.abs().max().item() + 2.0 ** -20) + (
        T * G + n) * 2.0 ** -23
    for b in range(B):
        for h in range(Hkv):
            assert abs(p.at("mass", b, h)[:n].astype(np.float64).sum() / (T * G) - 1) <= rel


@pytest.mark.parametrize("T,G,D,fmt", [(11, 3, 128, O.E4M3), (16, 4, 64, O.INT8), (5, 13, 64, O.E4M3)])
def test_weights_of_33_to_65_query_rows_in_a_large_cache(T, G, D, fmt):
    # (large by its capacity: 612 tiles of 128 rows)
    p = filled(3, 4, D, [300, 170, 9], 16, 0, fmt, seed=44, cap=6500)
    q = p.rows(T, 4 * G, "f16", 0.7)
    qd, lse = run_attention(p, q, G, [T, T // 2, 3])
    check_mass(p, q, qd, lse, G, [T, T // 2, 3])


@pytest.mark.parametrize("T", [3, 50])
def test_queries_whose_lse_is_infinite_add_nothing(T):
    p = filled(2, 2, 64, [300, 170], 16, 0, O.E4M3, seed=43)
    q = p.rows(T, 4, "bf16", 0.7)
    qd, lse = run_attention(p, q, 2)
    bad = lse.clone()
    bad[0, 0, 1], bad[1, T - 1, 2], bad[0, T // 2] = float("inf"), float("-inf"), float("inf")
    check_mass(p, q, qd, bad, 2, None)


@pytest.mark.parametrize("T", [1, 140])
def test_attention_of_extreme_rows(T):
    """Large and tiny queries, V blocks whose scales lie far apart, zero rows,
    one key that outweighs all others."""
    p = Pair(1, 1, 64, 700, 16, 16, O.E4M3, seed=21)
    ws = p.c.workspace(1, 1)
    k, v = p.rows(650, 1, "f32"), p.rows(650, 1, "f32")
    v *= torch.exp2(torch.arange(650) // 16 % 21 - 10.0)[None, :, None, None]
    v[:, 64:96] = 0
    k[:, 128:160] = 0
    k[:, 333] *= 40
    p.append(k, v, ws)
    q = p.rows(T, 6, "bf16")
    q[:, :, 0] = 0
    q[:, :, 1] *= 4.0
    q[:, :, 2] *= 2.0 ** -100
    q[:, :, 3] *= 2.0 ** -9
    run_attention(p, q, 6)
    run_attention(p, q, 6, scale=3.0)
    # queries beyond f16's range: the logits stay apart, the heaviest key takes all
    big = torch.zeros(1, T, 6, 64, dtype=torch.bfloat16)
    big[..., 0] = 2.0 ** 40
    out = torch.empty(1, T, 6, 64, dtype=torch.bfloat16, device="cuda")
    K.kv8_attn(p.c, big.cuda(), out, p.c.workspace(T, 6))
    kk, vv = p.seq[0, 0, "k"].values(), p.seq[0, 0, "v"].values()
    for t in (0, T - 1):
        n = O.visible(650, T, t)
        best = vv[:n][kk[:n, 0] == kk[:n, 0].max()].mean(0)
        got = out[0, t].cpu().double().numpy()
        assert (np.abs(got - best) <= 2.0 ** -7 * np.abs(best) + 2.0 ** -9 * np.abs(best).max()).all()


@pytest.mark.parametrize("T", [1, 150])
def test_attention_keeps_bad_rows_to_themselves(T):
    """A NaN query spoils its own row alone; garbage behind the length, none."""
    p = filled(1, 2, 128, [400], 64, 64, O.E4M3, seed=31)
    q = p.rows(T, 8, "bf16")
    ws = p.c.workspace(T, 8)
    a, b = (torch.empty(1, T, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in "ab")
    K.kv8_attn(p.c, q.cuda(), a, ws)
    q[0, 0, 3, 5] = math.nan
    q[0, T // 2, 6, 1] = math.inf
    K.kv8_attn(p.c, q.cuda(), b, ws)
    same = torch.ones(1, T, 8, dtype=torch.bool, device="cuda")
    same[0, 0, 3] = False
    same[0, T // 2, 6] = False
    assert torch.isfinite(a).all() and torch.equal(a[same], b[same])
    assert torch.isnan(b[0, 0, 3]).all()


@pytest.mark.parametrize("T", [1, 100])
def test_attention_leaves_out_rows_of_bad_pages(T):
    p = filled(2, 2, 64, [200, 210], 16, 16, O.INT8, seed=41)
    q = p.rows(T, 8, "f16")
    ws = p.c.workspace(T, 8)
    bad = p.c.page_table.clone()
    for b, i, to in ((0, 3, -1), (1, 0, p.c.num_pages), (1, 12, 2 ** 30)):
        p.c.page_table[b, i] = to
    out = torch.empty(2, T, 8, 64, dtype=torch.float16, device="cuda")
    lse = torch.empty(2, T, 8, device="cuda")
    K.kv8_attn(p.c, q.cuda(), out, ws, lse=lse)
    assert K.get_status(ws) == K.DEV_BAD_PAGE
    K.reset_status(ws)
    p.c.mass.fill_(-1.0)
    K.kv8_mass(p.c, q.cuda(), lse, ws, decay=0.0)
    assert K.get_status(ws) == K.DEV_BAD_PAGE
    p.c.page_table.copy_(bad)
    for b in range(2):
        gone = {0: [3], 1: [0, 12]}[b]
        n = p.len[b]
        hid = np.isin(np.arange(n) // 16, gone)
        for h in range(2):
            k, v = p.seq[b, h, "k"].values(), p.seq[b, h, "v"].values()
            x = q[b, :, 4 * h: 4 * h + 4].double().numpy() @ k.T / 8.0
            i = np.arange(T)[:, None, None]
            x = np.where((np.arange(n) > n - T + i) | hid, -np.inf, x)
            e = np.exp(x - x.max(-1, keepdims=True))
            o = (e / e.sum(-1, keepdims=True)) @ v
            got = out[b, :, 4 * h: 4 * h + 4].cpu().double().numpy()
            assert np.abs(got - o).max() <= 2.0 ** -9 * np.abs(v).max()
            m = p.at("mass", b, h)[:n]
            assert (m[hid] == -1.0).all() and (m[~hid] >= 0).all()


def test_attention_strided_tensors_and_streams():
    p = filled(2, 2, 64, [300, 170], 32, 64, O.E4M3, seed=51)
    for T in (1, 90):
        fused = p.rows(T, 12, "bf16").cuda()
        q = fused[:, :, 2:10]
        store = torch.full((2, 8, T, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        run_attention(p, q, 4, out=store.transpose(1, 2))
        a = store.transpose(1, 2).clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        b = torch.empty_like(a)
        ws = p.c.workspace(T, 8)
        K.kv8_attn(p.c, q, b, ws, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(a, b)
        K.kv8_attn(p.c, q, b.zero_(), ws)              # and the same bits again
        assert torch.equal(a, b)


def test_a_short_wait_limit_ends_in_a_status_or_the_right_result():
    """With a limit of 1 ns every on-chip wait gives up that is not over when the
    hardware's own suspension of it ends.  A call then reports it, or, where none
    did, its result is the right one; the next calls are right either way."""
    p = filled(2, 2, 128, [2000, 900], 64, 64, O.E4M3, seed=55)
    q = p.rows(600, 8, "bf16", 0.7)
    qd, lse = run_attention(p, q, 4)
    ws = p.c.workspace(600, 8)
    out, again = torch.empty_like(qd), torch.empty_like(qd)
    K.kv8_attn(p.c, qd, out, ws)
    K.kv8_mass(p.c, qd, lse, ws, decay=0.0)
    mass = p.c.mass.clone()
    for call, got, want in ((lambda: K.kv8_attn(p.c, qd, again, ws), again, out),
                            (lambda: K.kv8_mass(p.c, qd, lse, ws, decay=0.0), p.c.mass, mass)):
        try:
            K.set_wait_limit(1)
            call()
            torch.cuda.synchronize()
        finally:
            K.set_wait_limit(0)
        status = K.get_status(ws)
        assert status in (0, K.DEV_TIMEOUT)
        assert status or torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
        K.reset_status(ws)
    qd, lse = run_attention(p, q, 4)
    check_mass(p, q, qd, lse, 4, None)


@pytest.mark.parametrize("T", [1, 6, 90])
def test_captured_and_replayed(T):
    """A graph of all operators, captured before any of them ran on these shapes,
    replayed on new inputs in the same buffers, two graphs on one workspace."""
    G, Hkv, D = 3, 3, 64
    for fmt in (O.E4M3, O.INT8):
        a, b = (Pair(2, Hkv, D, 512, 32, 32, fmt, seed=56 + i) for i in range(2))
        ws = a.c.workspace(T, G * Hkv)
        runs = []
        for p in (a, b):
            x = {n: torch.zeros(2, T, h, D, dtype=torch.float16, device="cuda")
                 for n, h in (("k", Hkv), ("v", Hkv), ("q", G * Hkv), ("o", G * Hkv))}
            x["lse"] = torch.zeros(2, T, G * Hkv, device="cuda")
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                K.kv8_append(p.c, x["k"], x["v"], ws)
                K.kv8_attn(p.c, x["q"], x["o"], ws, lse=x["lse"])
                K.kv8_mass(p.c, x["q"], x["lse"], ws, decay=0.0)
            runs.append((p, g, x))
        for _ in range(3):
            ins = []
            for p, g, x in runs:
                new = {n: p.rows(T, x[n].shape[2], "f16", 0.7) for n in "kvq"}
                for n in "kvq":
                    x[n].copy_(new[n])
                ins.append(new)
                g.replay()
            torch.cuda.synchronize()
            for (p, g, x), new in zip(runs, ins):
                for bb in range(2):
                    for h in range(Hkv):
                        for s in "kv":
                            p.seq[bb, h, s].append(new[s][bb, :, h].double().numpy())
                    p.len[bb] += T
                p.check()
                for bb in range(2):
                    for h in range(Hkv):
                        hs = slice(h * G, (h + 1) * G)
                        ro, rl, tol, _ = attention_bounds(new["q"][bb, :, hs].double().numpy(), p, bb,
                                                          h, G, T, 1 / math.sqrt(D), HALF["f16"])
                        assert (np.abs(x["o"][bb, :, hs].cpu().double().numpy() - ro) <= tol).all()
                        m = p.at("mass", bb, h)[: p.len[bb]]
                        assert abs(m.sum() - T * G) < 1e-4 * T * G
        assert K.get_status(ws) == 0


def test_output_over_the_queries():
    """out may be q: rows are read before they are written."""
    p = filled(2, 2, 64, [3000, 700], 64, 64, O.E4M3, seed=57)
    for T in (1, 7, 40, 200):
        q = p.rows(T, 8, "bf16").cuda()
        ws = p.c.workspace(T, 8)
        out = torch.empty_like(q)
        K.kv8_attn(p.c, q, out, ws)
        K.kv8_attn(p.c, q, q, ws)
        assert torch.equal(q, out)


def test_a_page_shared_by_two_sequences():
    p = filled(2, 1, 64, [80, 80], 16, 16, O.E4M3, seed=61)
    p.c.page_table[1, :3] = p.c.page_table[0, :3]
    for s in "kv":
        a, b = p.seq[0, 0, s], p.seq[1, 0, s]
        b.codes[:48], b.scales[:3] = a.codes[:48], a.scales[:3]
    p.table = p.c.page_table.cpu()
    run_attention(p, p.rows(1, 4, "f16"), 4)


# ------------------------------------------------------------------- eviction
def weights(p, kind):
    r = p.rng
    w = []
    for b in range(p.B):
        w.append([])
        for h in range(p.Hkv):
            x = np.exp(2 * r.standard_normal(p.len[b])).astype(np.float32)
            if kind == "ties":
                x = np.floor(x).astype(np.float32)
            if kind == "equal":
                x[:] = 0.0
            if kind == "odd" and len(x) > 8:
                x[r.integers(0, len(x), 3)] = np.nan
                x[r.integers(0, len(x), 3)] = np.inf
                x[r.integers(0, len(x), 3)] = -0.0
                x[r.integers(0, len(x), 3)] = -1.0
            w[-1].append(x)
    return w


@pytest.mark.parametrize("into", ["place", "cache", "pool"])
@pytest.mark.parametrize("i,fmt", [(i, f) for i in range(10) for f in (O.E4M3, O.INT8)])
def test_evict(i, fmt, into):
    B, Hkv, D, lens, block, page, keep, sink, recent, kind = [
        (2, 2, 64, [300, 50], 16, 16, 100, 4, 20, "plain"),
        (3, 1, 128, [1500, 101, 100], 64, 64, 100, 0, 0, "ties"),
        (1, 3, 64, [257], 32, 96, 256, 1, 255, "plain"),
        (2, 2, 128, [900, 4100], 128, 0, 777, 0, 777, "plain"),
        (2, 1, 64, [400, 0], 16, 48, 1, 0, 0, "odd"),
        (2, 2, 128, [400, 399], 16, 16, 130, 130, 0, "ties"),
        (1, 2, 64, [2300], 32, 64, 1999, 3, 10, "odd"),
        (2, 2, 64, [600, 555], 64, 0, 200, 4, 32, "equal"),
        (2, 1, 64, [9000, 8999], 64, 64, 3000, 7, 100, "ties"),      # spread over eight CTAs
        (1, 1, 64, [140000], 128, 128, 20001, 0, 1, "ties")][i]      # keys beyond the registers
    p = filled(B, Hkv, D, lens, block, page, fmt, seed=200 + i, cap=max(lens) + 7)
    # a few tokens one by one: blocks whose scale is larger than their rows need
    ws = p.c.workspace(1, Hkv)
    w = weights(p, kind)
    p.set_mass(w)
    kept = torch.full((B, Hkv, keep), -9, dtype=torch.int32, device="cuda")
    src_codes = p.c.k_codes.clone()
    if into == "place":
        d = p
        K.kv8_evict(p.c, keep, sink, recent, kept, ws)
    else:
        d = Pair(B, Hkv, D, keep + 3, block, page, fmt, seed=300 + i)
        if into == "pool" and page:
            # both caches over one pool of pages, tables of different pages
            n = p.c.num_pages + d.c.num_pages
            big = {k: torch.cat([getattr(p.c, k), getattr(d.c, k)]) for k in
                   ("k_codes", "v_codes", "k_scales", "v_scales", "mass")}
            seqs = (p.c.seq_len, d.c.seq_len)
            tabs = (p.table, d.table + p.c.num_pages)
            for x, s, t in zip((p, d), seqs, tabs):
                x.table = t
                x.c = K.Cache8(B, Hkv, D, x.c.max_len, block=block, page_size=page, page_table=t,
                               num_pages=n, fmt=fmt, tensors=big | {"seq_len": s})
            src_codes = p.c.k_codes.clone()
        K.kv8_evict(p.c, keep, sink, recent, kept, ws, dst=d.c)
        assert p.c.seq_len.tolist() == p.len
        own = torch.unique(p.table).long() if page else torch.arange(B)
        assert torch.equal(src_codes[own.cuda()], p.c.k_codes[own.cuda()])
    assert K.get_status(ws) == 0
    d_seq, lens2 = {}, []
    for b in range(B):
        lens2.append(min(p.len[b], keep))
        for h in range(Hkv):
            rows = O.evict(w[b][h], p.len[b], keep, sink, recent)
            assert kept[b, h, : len(rows)].tolist() == rows.tolist()
            assert (kept[b, h, len(rows):] == -1).all()
            for s in "kv":
                d_seq[b, h, s] = p.seq[b, h, s].keep(rows)
            m = d.at("mass", b, h)[: len(rows)]
            assert np.array_equal(m, w[b][h][rows], equal_nan=True)
    d.seq, d.len = d_seq, lens2
    d.check()
    if into == "cache":
        d.untouched_behind(lens2)


@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
def test_evict_of_rows_far_below_their_block(fmt):
    """The rows that stay hold the smallest codes only: their blocks' new scales
    are up to 2^17 below the old ones; and blocks of zeros."""
    for small in (2.0 ** -6, 2.0 ** -16, 2.0 ** -17, 1.5 * 2.0 ** -18, 0.0):
        p = Pair(1, 2, 64, 64, 32, 32, fmt, seed=72)
        ws = p.c.workspace(1, 2)
        k, v = (torch.sign(p.rows(64, 2, "f32")) * 448.0 for _ in "kv")
        k[:, 1::2] *= small
        v[:, 1::2] *= small
        p.append(k, v, ws)
        p.set_mass([[np.tile([0.0, 1.0], 32)] * 2])
        kept = torch.empty(1, 2, 32, dtype=torch.int32, device="cuda")
        K.kv8_evict(p.c, 32, 0, 0, kept, ws)
        for h in range(2):
            for s in "kv":
                p.seq[0, h, s] = p.seq[0, h, s].keep(np.arange(1, 64, 2))
        p.len = [32]
        p.check()


def test_evict_of_a_sequence_with_a_bad_page():
    p = filled(1, 1, 64, [100], 16, 16, O.E4M3, seed=71)
    ws = p.c.workspace(1, 1)
    p.set_mass([[np.arange(100.0)]])
    p.c.page_table[0, 4] = -5
    kept = torch.empty(1, 1, 50, dtype=torch.int32, device="cuda")
    K.kv8_evict(p.c, 50, 20, 10, kept, ws)
    # rows 64..79, on the bad page, rank below all others
    assert kept[0, 0].tolist() == [*range(20), *range(54, 64), *range(80, 100)]
    assert K.get_status(ws) == K.DEV_BAD_PAGE
    assert p.c.seq_len.tolist() == [50]
    assert np.array_equal(O.decode(p.at("k_codes", 0, 0)[:16], O.E4M3), p.seq[0, 0, "k"].codes[:16])


# ------------------------------------------------------------- all of them
@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop(fmt, graph):
    """A prompt, its weights, eviction, then tokens: append, attend, accumulate,
    evict at the budget, as one program; captured once and replayed."""
    B, Hkv, G, D, keep = 2, 2, 4, 64, 96
    H = Hkv * G
    p = Pair(B, Hkv, D, 256, 16, 16, fmt, seed=81)
    ws = p.c.workspace(140, H)
    lens = [140, 75]
    p.append(p.rows(140, Hkv, "bf16"), p.rows(140, Hkv, "bf16"), ws, lens=lens)
    q = p.rows(140, H, "bf16", 0.7)
    qd, lse = run_attention(p, q, G, lens)
    K.kv8_mass(p.c, qd, lse, ws, q_len=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    kept = torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda")

    def evicted():
        """What the oracle keeps by the device's own weights."""
        for b in range(B):
            rows = {h: O.evict(before[b, h], p.len[b], keep, 4, 16) for h in range(Hkv)}
            for h in range(Hkv):
                assert kept[b, h, : len(rows[h])].tolist() == rows[h].tolist()
                for s in "kv":
                    p.seq[b, h, s] = p.seq[b, h, s].keep(rows[h])
            p.len[b] = min(p.len[b], keep)
        p.check()

    before = {(b, h): p.at("mass", b, h) for b in range(B) for h in range(Hkv)}
    K.kv8_evict(p.c, keep, 4, 16, kept, ws)
    evicted()

    kt, vt = (torch.zeros(B, 1, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    qt, ot = (torch.zeros(B, 1, H, D, dtype=torch.bfloat16, device="cuda") for _ in "qo")
    ls = torch.zeros(B, 1, H, device="cuda")
    copy = torch.empty_like(p.c.mass)

    def step():
        K.kv8_append(p.c, kt, vt, ws)
        K.kv8_attn(p.c, qt, ot, ws, lse=ls)
        K.kv8_mass(p.c, qt, ls, ws, decay=0.9)
        copy.copy_(p.c.mass)
        K.kv8_evict(p.c, keep, 4, 16, kept, ws)

    g = None
    if graph:
        keep_state = [t.clone() for t in (p.c.k_codes, p.c.v_codes, p.c.k_scales, p.c.v_scales,
                                          p.c.mass, p.c.seq_len)]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        for t, x in zip((p.c.k_codes, p.c.v_codes, p.c.k_scales, p.c.v_scales, p.c.mass,
                         p.c.seq_len), keep_state):
            t.copy_(x)
    for i in range(30):
        k, v, q = p.rows(1, Hkv, "bf16"), p.rows(1, Hkv, "bf16"), p.rows(1, H, "bf16", 0.7)
        kt.copy_(k), vt.copy_(v), qt.copy_(q)
        if g is not None:
            g.replay()
        else:
            step()
        torch.cuda.synchronize()
        for b in range(B):
            for h in range(Hkv):
                for s, x in (("k", k), ("v", v)):
                    p.seq[b, h, s].append(x[b, :1, h].double().numpy())
            p.len[b] += 1
        o, l2 = ot.cpu().double().numpy(), ls.cpu().double().numpy()
        for b in range(B):
            for h in range(Hkv):
                hs = slice(h * G, (h + 1) * G)
                ro, rl, tol, ltol = attention_bounds(q[b, :, hs].double().numpy(), p, b, h, G, 1,
                                                     1 / math.sqrt(D), HALF["bf16"])
                assert (np.abs(o[b, :, hs] - ro) <= tol).all()
                assert (np.abs(l2[b, :, hs] - rl) <= ltol).all()
        real, p.c.mass = p.c.mass, copy
        before = {(b, h): p.at("mass", b, h) for b in range(B) for h in range(Hkv)}
        p.c.mass = real
        evicted()
    assert K.get_status(ws) == 0


def test_readme_example():
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")).read()
    blocks = re.findall(r"```py\n(.*?)```", text, re.S)
    assert len(blocks) == 1
    env = {}
    exec(compile(blocks[0], "README.md", "exec"), env)
    B, Hkv, G, keep = env["B"], env["Hkv"], env["H"] // env["Hkv"], env["keep"]
    cache, kept = env["cache"], env["kept"].cpu()
    assert cache.seq_len.tolist() == [keep + 1] * B
    assert (kept.diff(dim=-1) > 0).all()
    assert torch.equal(kept[..., :4], torch.arange(4, dtype=torch.int32).expand(B, Hkv, 4))
    assert torch.equal(kept[..., -64:], torch.arange(1436, 1500, dtype=torch.int32).expand(B, Hkv, 64))
    # the token's weights sum to one a query; behind them 0.99 of what stayed
    m = cache.mass[:, :, : keep + 1].double()
    assert torch.isfinite(m).all() and (m.sum(-1) <= 0.99 * env["prompt"] * G + G + 0.1).all()
    assert (m.sum(-1) > G).all() and torch.isfinite(env["out"]).all() and torch.isfinite(env["out1"]).all()
