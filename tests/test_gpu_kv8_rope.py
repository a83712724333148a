"""GPU parity of the rotation, of the append with it and of the append of chosen rows:
every byte equals the oracle's, and what is not the calls' to write stays."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp4_kv_cache_rope_gb300 as K  # noqa: E402
from oracle import kv8 as O  # noqa: E402
from kv8_tools import DT, Pair  # noqa: E402
from kv8_more_tools import ints, rope, rotated, tree  # noqa: E402


def same(got, want):
    """Equal element for element, NaN where NaN."""
    got, want = got.cpu().double(), want.double()
    return torch.equal(got.nan_to_num(nan=12345.0), want.nan_to_num(nan=12345.0))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("Hkv,G,D,R,first,style", [
    (2, 7, 128, 128, 0, O.HALVES), (1, 1, 64, 64, 0, O.PAIRS), (8, 8, 128, 64, 64, O.PAIRS),
    (4, 2, 64, 16, 8, O.HALVES), (3, 5, 128, 96, 16, O.HALVES), (1, 3, 64, 48, 0, O.PAIRS)])
def test_rope(dtype, Hkv, G, D, R, first, style):
    B, T, H = 3, 9, Hkv * G
    p = Pair(B, Hkv, D, 64, 16, 16, O.E4M3, seed=3)
    ws = p.c.workspace(1, Hkv)
    p.c.seq_len.copy_(ints([0, 33, 64]))
    r, c, s = rope(70, R, first, style)
    q, k = p.rows(T, H, dtype), p.rows(T, Hkv, dtype)
    lens = [9, 5, 0]
    parent = tree(p.rng, B, T)
    depth = [[len(O.path_to(parent[b], i)) - 1 for i in range(T)] for b in range(B)]
    pos = p.rng.integers(0, 70, (B, T)).tolist()
    for how, at in [("row", [[n + i for i in range(T)] for n in (0, 33, 64)]), ("pos", pos),
                    ("tree", [[n + d for d in x] for n, x in zip((0, 33, 64), depth)])]:
        args = {"pos": ints(pos)} if how == "pos" else {"parent": ints(parent)} if how == "tree" else {}
        # a row past the table (64 + 6 on) stays as it is
        want = [rotated(x, at, c, s, first, style).to(DT[dtype]) for x in (q, k)]
        for lens2 in (None, lens):
            qo, ko = (torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda") for x in (q, k))
            K.kv8_rope(p.c, q.cuda(), qo, r, ws, k=k.cuda(), k_out=ko, q_len=ints(lens2), **args)
            for got, w in ((qo, want[0]), (ko, want[1])):
                for b in range(B):
                    n = T if lens2 is None else lens2[b]
                    assert same(got[b, :n], w[b, :n]), (how, b)
                    assert (got[b, n:] == 7.0).all()
        # in place, and without keys
        x = q.cuda()
        K.kv8_rope(p.c, x, x, r, ws, **args)
        assert same(x, want[0]), how
        bad = any(y >= 70 for z in at for y in z)
        assert K.get_status(ws) == (K.DEV_BAD_INDEX if bad else 0), how
        K.reset_status(ws)


def test_rope_of_slices_of_a_fused_projection_in_place():
    p = Pair(2, 2, 64, 64, 16, 0, O.INT8, seed=4)
    ws = p.c.workspace(1, 2)
    r, c, s = rope(40, 32)
    fused = p.rows(11, 10, "bf16")
    x = fused.cuda()
    K.kv8_rope(p.c, x[:, :, :6], x[:, :, :6], r, ws, k=x[:, :, 6:8], k_out=x[:, :, 6:8])
    at = [list(range(11))] * 2
    want = fused.clone()
    want[:, :, :8] = rotated(fused[:, :, :8], at, c, s, 0, O.HALVES).to(torch.bfloat16)
    assert same(x, want)
    # heads in front of tokens, one row for all sequences
    y = p.rows(6, 11, "f16")[:1].expand(2, 6, 11, 64).transpose(1, 2)
    out = torch.empty(2, 6, 11, 64, dtype=torch.float16, device="cuda").transpose(1, 2)
    K.kv8_rope(p.c, y.cuda(), out, r, ws)
    assert same(out, rotated(y, at, c, s, 0, O.HALVES).half())


def test_parents_that_are_no_earlier_tokens():
    p = Pair(1, 1, 64, 64, 16, 0, O.E4M3, seed=4)
    ws = p.c.workspace(1, 1)
    p.c.seq_len.fill_(10)
    r, c, s = rope(40, 64)
    parent = [[-1, 0, 2, 100, 1, -7, 2 ** 31 - 1]]
    at = [[10 + len(O.path_to(parent[0], i)) - 1 for i in range(7)]]
    q = p.rows(7, 2, "f32")
    out = torch.empty(1, 7, 2, 64, device="cuda")
    K.kv8_rope(p.c, q.cuda(), out, r, ws, parent=ints(parent))
    assert same(out, rotated(q, at, c, s, 0, O.HALVES))
    assert K.get_status(ws) == K.DEV_BAD_TREE


# ------------------------------------------------------------- append with rotation
@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
@pytest.mark.parametrize("Hkv,G,D,block,page,dtype,R,first,style", [
    (2, 3, 128, 64, 64, "bf16", 128, 0, O.HALVES), (1, 1, 64, 16, 16, "f16", 64, 0, O.PAIRS),
    (3, 2, 128, 16, 48, "f32", 64, 32, O.HALVES), (8, 8, 64, 128, 0, "bf16", 32, 0, O.PAIRS),
    (20, 1, 128, 32, 128, "f32", 16, 112, O.PAIRS), (4, 4, 128, 128, 128, "f16", 96, 0, O.HALVES),
    (2, 2, 64, 64, 0, "f32", 64, 0, O.HALVES)])
def test_append_rope(fmt, Hkv, G, D, block, page, dtype, R, first, style):
    B, H = 3, Hkv * G
    p = Pair(B, Hkv, D, 400, block, page, fmt, seed=11)
    ws = p.c.workspace(1, Hkv)
    r, c, s = rope(500, R, first, style)
    ever = [0] * B
    for step, (T, lens, how) in enumerate([
            (70, [70, 1, 33], ""), (1, None, ""), (1, [0, 1, 1], "pos"), (3, None, "start"), (0, None, ""),
            (8, [8, 5, 0], "start"), (9, None, "pos"), (150, [0, 150, 97], "own"), (20, None, "start")]):
        k, v = (p.rows(T, Hkv, dtype, 2.0 ** (step % 3)) for _ in "kv")
        q = p.rows(T, H, dtype)
        start, args = None, {}
        if how == "start":
            start = [max(0, n - 2 * b) for b, n in enumerate(p.len)]
            args["start"] = ints(start)
        elif how == "own":
            args["start"] = p.c.seq_len
        first_at = p.len if start is None else start
        at = [[n + i for i in range(T)] for n in first_at]
        if how == "pos":
            at = p.rng.integers(0, 500, (B, T)).tolist()
            args["pos"] = ints(at)
        qo = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        K.kv8_append_rope(p.c, k.cuda(), v.cuda(), r, ws, q=q.cuda(), q_out=qo, new_len=ints(lens), **args)
        kr = rotated(k, at, c, s, first, style) if T else k
        for b in range(B):
            t = T if lens is None else lens[b]
            for h in range(Hkv):
                p.seq[b, h, "k"].append(kr[b, :t, h].double().numpy(), first_at[b])
                p.seq[b, h, "v"].append(v[b, :t, h].double().numpy(), first_at[b])
            if T:
                want = rotated(q[b:b + 1], at[b:b + 1], c, s, first, style).to(DT[dtype])
                assert same(qo[b, :t], want[0, :t])
                assert (qo[b, t:] == 7.0).all()
        p.len = [n + (T if lens is None else lens[b]) for b, n in enumerate(first_at)]
        p.check()
        ever = [max(n, m) for n, m in zip(p.len, ever)]
        p.untouched_behind(ever)
    for b in range(B):
        for h in range(Hkv):
            assert (p.at("mass", b, h)[: p.len[b]] == 0).all()
    assert K.get_status(ws) == 0


@pytest.mark.parametrize("T", [1, 8, 60])
def test_append_rope_alone_and_in_place(T):
    """Without queries, and with queries rotated in place in the fused projection."""
    p, p2 = (Pair(2, 2, 128, 128, 32, 32, O.E4M3, seed=3, mass=False) for _ in "ab")
    ws = p.c.workspace(1, 2)
    r, c, s = rope(128, 128)
    fused = p.rows(T, 10, "bf16")
    at = [list(range(T))] * 2
    kr = rotated(fused[:, :, 6:8], at, c, s, 0, O.HALVES)
    for x, with_q in ((p, False), (p2, True)):
        f = fused.cuda()
        args = {"q": f[:, :, :6], "q_out": f[:, :, :6]} if with_q else {}
        K.kv8_append_rope(x.c, f[:, :, 6:8], f[:, :, 8:], r, ws, **args)
        for b in range(2):
            for h in range(2):
                x.seq[b, h, "k"].append(kr[b, :, h].double().numpy())
                x.seq[b, h, "v"].append(fused[b, :, 8 + h].double().numpy())
        x.len = [T, T]
        x.check()
        want = fused.clone()
        if with_q:
            want[:, :, :6] = rotated(fused[:, :, :6], at, c, s, 0, O.HALVES).to(torch.bfloat16)
        assert same(f, want)


@pytest.mark.parametrize("T", [2, 60])
def test_append_rope_values_at_the_edges(T):
    for fmt in (O.E4M3, O.INT8):
        p = Pair(1, 1, 64, 256, 16, 16, fmt, seed=6)
        ws = p.c.workspace(1, 1)
        r, c, s = rope(256, 64)
        for step in range(3):
            k, v = p.rows(T, 1, "f32"), p.rows(T, 1, "f32")
            if step == 0:       # tiny and huge values, which rotate into subnormal and infinite ones
                k[0, 1, 0, :4] = torch.tensor([2.0 ** -149, -2.0 ** -126, 1e-38, 0.0])
                k[0, 1, 0, 4:] = 0.0
            elif step == 1:
                k[0, 0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 2.0])
            else:
                k[0, T - 1] = 3.4e38
            at = [[p.len[0] + i for i in range(T)]]
            K.kv8_append_rope(p.c, k.cuda(), v.cuda(), r, ws)
            kr = rotated(k, at, c, s, 0, O.HALVES)
            assert torch.isfinite(kr).all() == (step == 0)
            p.seq[0, 0, "k"].append(kr[0, :, 0].double().numpy())
            p.seq[0, 0, "v"].append(v[0, :, 0].double().numpy())
            p.len[0] += T
            p.check()
            assert K.get_status(ws) == (0 if step == 0 else K.DEV_NONFINITE)
            K.reset_status(ws)


@pytest.mark.parametrize("T", [4, 50])
def test_append_rope_past_the_end_of_cache_and_table(T):
    p = Pair(2, 2, 64, 64, 16, 16, O.E4M3, seed=7)
    ws = p.c.workspace(1, 2)
    r, c, s = rope(63, 64)          # the table ends before the cache
    p.append(p.rows(62, 2, "bf16"), p.rows(62, 2, "bf16"), ws, lens=[62, 10])
    k, v, q = p.rows(T, 2, "bf16"), p.rows(T, 2, "bf16"), p.rows(T, 4, "bf16")
    out = torch.zeros(2, T, 4, 64, dtype=torch.bfloat16, device="cuda")
    K.kv8_append_rope(p.c, k.cuda(), v.cuda(), r, ws, q=q.cuda(), q_out=out)
    at = [[n + i for i in range(T)] for n in p.len]
    kr = rotated(k, at, c, s, 0, O.HALVES)
    for h in range(2):
        for side, x in (("k", kr), ("v", v)):
            p.seq[0, h, side].append(x[0, :2, h].double().numpy())
            p.seq[1, h, side].append(x[1, :T, h].double().numpy())
    p.len = [64, 10 + T]
    p.check()
    assert same(out, rotated(q, at, c, s, 0, O.HALVES).to(torch.bfloat16))
    assert K.get_status(ws) == K.DEV_OVERFLOW | K.DEV_BAD_INDEX


@pytest.mark.parametrize("T", [3, 40])
def test_append_rope_bad_pages_and_starts(T):
    p = Pair(2, 2, 64, 64, 16, 16, O.E4M3, seed=7)
    ws = p.c.workspace(1, 2)
    r, c, s = rope(64, 64)
    p.c.page_table[0, 0] = 10 ** 6
    p.table[0, 0] = p.c.num_pages - 1
    k, v = p.rows(T, 2, "bf16"), p.rows(T, 2, "bf16")
    q = p.rows(T, 2, "bf16")
    out = torch.zeros_like(q, device="cuda")
    K.kv8_append_rope(p.c, k.cuda(), v.cuda(), r, ws, q=q.cuda(), q_out=out, start=ints([0, -3]))
    assert K.get_status(ws) == K.DEV_BAD_PAGE | K.DEV_OVERFLOW | K.DEV_BAD_INDEX
    # a start before the cache appends nothing; its queries at positions from 0 on are turned
    assert p.c.seq_len.tolist() == [T, 0]
    at = [list(range(T)), [i - 3 for i in range(T)]]
    assert same(out, rotated(q, at, c, s, 0, O.HALVES).to(torch.bfloat16))


# --------------------------------------------------------------- append of a path
@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
@pytest.mark.parametrize("Hkv,D,block,page,dtype", [
    (2, 128, 64, 64, "bf16"), (1, 64, 16, 16, "f16"), (3, 128, 16, 48, "f32"),
    (8, 64, 128, 0, "bf16"), (20, 128, 32, 128, "f32"), (4, 128, 128, 0, "f16")])
def test_append_path(fmt, Hkv, D, block, page, dtype):
    p = Pair(3, Hkv, D, 400, block, page, fmt, seed=12)
    ws = p.c.workspace(1, Hkv)
    for step, (T, M, lens, start) in enumerate([
            (60, 7, [7, 1, 0], None), (60, 60, None, None), (5, 9, [2, 9, 5], None), (1, 1, None, None),
            (200, 150, [150, 0, 93], None), (9, 0, None, None), (9, 3, None, [10, 0, 40]),
            (30, 30, None, [5, 0, 43])]):
        k, v = (p.rows(T, Hkv, dtype, 2.0 ** (step % 3)) for _ in "kv")
        path = p.rng.integers(0, T, (3, M))
        fused = torch.cat([k, v], 2).cuda()      # strided
        K.kv8_append_path(p.c, fused[:, :, :Hkv], fused[:, :, Hkv:], ints(path.tolist()).view(3, M), ws,
                          new_len=ints(lens), start=ints(start))
        at = p.len if start is None else start
        for b in range(3):
            m = path[b][: M if lens is None else lens[b]]
            for h in range(Hkv):
                for side, x in (("k", k), ("v", v)):
                    p.seq[b, h, side].append(x[b, m, h].double().numpy(), at[b])
        p.len = [n + (M if lens is None else lens[b]) for b, n in enumerate(at)]
        p.check()
    assert K.get_status(ws) == 0


@pytest.mark.parametrize("M", [4, 40])
def test_append_path_of_rows_that_are_not_there(M):
    p = Pair(2, 2, 64, 128, 16, 16, O.E4M3, seed=13)
    ws = p.c.workspace(1, 2)
    k, v = p.rows(6, 2, "f16"), p.rows(6, 2, "f16")
    path = [[i % 6 for i in range(M)] for _ in range(2)]
    path[0][1], path[0][3], path[1][0], path[1][2] = 6, -1, 2 ** 31 - 1, -2 ** 31
    K.kv8_append_path(p.c, k.cuda(), v.cuda(), ints(path), ws)
    for b in range(2):
        rows = [i if 0 <= i < 6 else None for i in path[b]]
        for h in range(2):
            for side, x in (("k", k), ("v", v)):
                p.seq[b, h, side].append(np.stack([np.zeros(64) if i is None else x[b, i, h].double().numpy()
                                                   for i in rows]))
    p.len = [M, M]
    p.check()
    assert K.get_status(ws) == K.DEV_BAD_INDEX
