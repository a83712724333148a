"""GPU parity of the attention with changed scores and of drafted tokens' attention
with the fp64 oracle, within the bounds that oracle.kv8.attend derives."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp4_kv_cache_rope_gb300 as K  # noqa: E402
from oracle import kv8 as O  # noqa: E402
from kv8_tools import Pair  # noqa: E402
from kv8_more_tools import check_attention, ints, scored_want, tree  # noqa: E402


def filled(B, Hkv, D, lens, block, page, fmt, dtype="bf16", seed=1, max_len=None):
    p = Pair(B, Hkv, D, max_len or max(max(lens), 1), block, page, fmt, seed=seed, mass=False)
    ws = p.c.workspace(1, Hkv)
    if max(lens):
        p.append(*(p.rows(max(lens), Hkv, dtype) for _ in "kv"), ws, lens=lens)
    return p


def slopes_of(H):
    return (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32)


def run_scored(p, G, T, dtype, scale=0.0, q_len=None, size=0.7, cap=0.0, window=0, sink=0, slopes=None,
               prefix=None, q=None):
    H = p.Hkv * G
    q = p.rows(T, H, dtype, size) if q is None else q
    ws = p.c.workspace(T, H)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((p.B, T, H), 7.0, device="cuda")
    sc = K.Scores(cap, window, sink, None if slopes is None else torch.from_numpy(slopes).cuda(),
                  ints(prefix))
    K.kv8_attn_scored(p.c, q.cuda(), out, ws, sc, lse=lse, q_len=ints(q_len), softmax_scale=scale)
    assert K.get_status(ws) == 0
    out, lse = out.cpu(), lse.cpu()
    for b in range(p.B):
        ql = T if q_len is None else q_len[b]
        assert (out[b, ql:] == 7.0).all() and (lse[b, ql:] == 7.0).all()
        for h in range(p.Hkv):
            want = scored_want(p, q, b, h, G, ql, scale or p.D ** -0.5, dtype, cap, window, sink, slopes,
                               prefix[b] if prefix else 0)
            hs = slice(h * G, h * G + G)
            check_attention(out[b, :ql, hs], lse[b, :ql, hs], want, (b, h))
    return q, out, lse


# (capacity, lengths, T, G): few rows in one launch, few rows split and joined, many rows,
# many rows whose cached rows are split
SHAPES = [(None, [300, 1, 77], 1, 3), (4096, [3000, 130, 2999], 2, 8), (4096, [2500, 0, 31], 5, 5),
          (None, [700, 90, 333], 40, 4), (9000, [9000, 400, 5000], 70, 2)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"T{s[2]}G{s[3]}")
@pytest.mark.parametrize("what", ["cap", "window", "sink", "slopes", "prefix", "all", "none"])
@pytest.mark.parametrize("D,fmt,dtype,block,page", [(128, O.E4M3, "bf16", 64, 64), (64, O.INT8, "f16", 16, 48)])
def test_scored(shape, what, D, fmt, dtype, block, page):
    cap_rows, lens, T, G = shape
    p = filled(3, 2, D, lens, block, page, fmt, seed=21, max_len=cap_rows)
    args = {}
    if what in ("cap", "all"):
        args["cap"], args["size"] = 5.0, 3.0
    if what in ("window", "sink", "all"):
        args["window"] = 129
    if what in ("sink", "all"):
        args["sink"] = 37
    if what in ("slopes", "all"):
        args["slopes"] = slopes_of(2 * G)
    if what in ("prefix", "all"):
        args["prefix"] = [260, 5, 0]
    q_len = None if what == "cap" else [T, max(0, T - 1), min(T, 3)]
    run_scored(p, G, T, dtype, q_len=q_len, **args)


@pytest.mark.parametrize("T,G", [(1, 4), (3, 7), (33, 3), (90, 4)])
@pytest.mark.parametrize("window,sink", [(1, 0), (1, 1), (2, 300), (128, 0), (128, 128), (500, 1000),
                                         (100000, 4), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_windows_at_the_edges(T, G, window, sink):
    """Windows of one row, on tile borders, beyond the rows; more queries than rows."""
    lens = [513, 20, 256, 0]
    p = filled(4, 1, 64, lens, 32, 0, O.E4M3, seed=22, max_len=4096 if T == 3 else None)
    run_scored(p, G, T, "f16", window=window, sink=sink)


@pytest.mark.parametrize("T,G", [(1, 8), (40, 3)])
def test_caps_and_scales_at_the_edges(T, G):
    p = filled(2, 2, 128, [400, 130], 64, 64, O.E4M3, seed=23)
    for cap, scale, size in [(2.0 ** -10, 0.0, 1.0), (30.0, 2.0, 4.0), (2.0 ** 20, 0.0, 1.0), (50.0, 1e-3, 1.0)]:
        run_scored(p, G, T, "bf16", cap=cap, scale=scale, size=size)


@pytest.mark.parametrize("T,G", [(1, 4), (50, 4)])
def test_steep_slopes_and_prefixes_beyond_the_rows(T, G):
    p = filled(3, 1, 64, [300, 40, 129], 16, 16, O.INT8, seed=24)
    for slopes in (np.array([0.0, 1000.0, 0.5, -0.01], np.float32), np.array([1e-20, 30.0, -1e-3, 0.0], np.float32)):
        run_scored(p, G, T, "bf16", slopes=slopes)
        run_scored(p, G, T, "bf16", slopes=slopes, prefix=[1000, -5, 64], q_len=[T, T, 0])
    # queries in front of the first row see the prefix alone
    run_scored(p, G, 60, "f16", prefix=[0, 13, 200], q_len=[60, 60, 60])


@pytest.mark.parametrize("T,G,max_len", [(1, 8, 512), (1, 8, 4096), (3, 8, 4096), (33, 8, 512), (10, 8, 9000)])
@pytest.mark.parametrize("D,fmt,dtype", [(128, K.KV8_E4M3, "bf16"), (64, K.KV8_INT8, "f16")])
def test_without_scores_it_is_the_plain_attention(T, G, max_len, D, fmt, dtype):
    p = filled(3, 2, D, [400, 1, 333], 64, 64, fmt, seed=25, max_len=max_len)
    H = 2 * G
    q = p.rows(T, H, dtype).cuda()
    ws = p.c.workspace(T, H)
    a, b = torch.empty_like(q), torch.empty_like(q)
    la, lb = (torch.empty(3, T, H, device="cuda") for _ in "ab")
    K.kv8_attn(p.c, q, a, ws, lse=la)
    K.kv8_attn_scored(p.c, q, b, ws, K.Scores(), lse=lb)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("T,G", [(1, 4), (4, 8), (60, 4)])
def test_queries_that_hold_no_numbers(T, G):
    """A NaN in one query spoils that query alone; garbage behind the rows and on unread
    pages counts nowhere (the caches here hold it)."""
    p = filled(2, 1, 64, [200, 150], 16, 16, O.E4M3, seed=26)
    q = p.rows(T, G, "bf16", 2.0)
    run_scored(p, G, T, "bf16", cap=10.0, window=90, sink=3, slopes=slopes_of(G), q=q)
    q2 = q.clone()
    q2[0, 0, 1, 5] = math.nan
    q2[1, T - 1, 0, 0] = math.inf
    ws = p.c.workspace(T, G)
    out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(2, T, G, device="cuda")
    K.kv8_attn_scored(p.c, q2.cuda(), out, ws, K.Scores(10.0, 90, 3, torch.from_numpy(slopes_of(G)).cuda()),
                      lse=lse)
    spoiled = torch.zeros(2, T, G, dtype=torch.bool)
    spoiled[0, 0, 1] = spoiled[1, T - 1, 0] = True
    assert out[0, 0, 1].isnan().all() and lse[0, 0, 1].isnan()
    out, lse = out.cpu(), lse.cpu()
    for b in range(2):
        want = scored_want(p, q, b, 0, G, T, p.D ** -0.5, "bf16", 10.0, 90, 3, slopes_of(G))
        keep = ~spoiled[b]
        check_attention(out[b][keep], lse[b][keep], tuple(x[keep.numpy()] for x in want), b)


def test_bad_pages_are_left_out():
    for T, G in ((1, 4), (40, 4)):
        p = filled(1, 1, 64, [200], 16, 16, O.E4M3, seed=27)
        q = p.rows(T, G, "bf16")
        ws = p.c.workspace(T, G)
        p.c.page_table[0, 3] = -1
        out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        lse = torch.empty(1, T, G, device="cuda")
        K.kv8_attn_scored(p.c, q.cuda(), out, ws, K.Scores(cap=20.0), lse=lse)
        assert K.get_status(ws) == K.DEV_BAD_PAGE
        k, v = (p.seq[0, 0, s].values() for s in "kv")
        pos = 200 - T + np.arange(T)
        j = np.arange(200)
        see = O.sees(pos, j, 200) & ((j < 48) | (j >= 64))
        want = O.attend(q[0].double().numpy(), k, v, 0.125, see, pos[:, None] - j, 20.0, None, 2.0 ** -8)
        check_attention(out[0].cpu(), lse[0].cpu(), want)


def test_scored_many_sequences_and_units():
    """More than 32 sequences, and several pieces of work for a CTA."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 900, 70)]
    p = filled(70, 3, 64, lens, 16, 16, O.INT8, seed=28, max_len=5000)
    run_scored(p, 2, 1, "bf16", cap=15.0)
    run_scored(p, 2, 2, "f16", window=200, sink=20, slopes=slopes_of(6))


# ---------------------------------------------------------------- drafted tokens
def run_tree(p, G, T, dtype, q_len=None, size=0.7, cap=0.0, window=0, sink=0, slopes=None, parent=None,
             chain=0.35, scores=True):
    H = p.Hkv * G
    q, k, v = p.rows(T, H, dtype, size), p.rows(T, p.Hkv, dtype), p.rows(T, p.Hkv, dtype)
    parent = tree(p.rng, p.B, T, chain) if parent is None else parent
    ws = p.c.tree_workspace(T, H)
    # rows behind q_len are garbage that no path leads to
    for b in range(p.B):
        if q_len is not None:
            k[b, q_len[b]:] = math.nan
            v[b, q_len[b]:] = math.nan
            parent[b][q_len[b]:] = [0] * (T - q_len[b])
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((p.B, T, H), 7.0, device="cuda")
    sc = K.Scores(cap, window, sink, None if slopes is None else torch.from_numpy(slopes).cuda())
    K.kv8_attn_tree(p.c, q.cuda(), k.cuda(), v.cuda(), ints(parent), out, ws, lse=lse, q_len=ints(q_len),
                    scores=sc if scores else None)
    assert K.get_status(ws) == 0
    out, lse = out.cpu(), lse.cpu()
    for b in range(p.B):
        ql = T if q_len is None else q_len[b]
        assert (out[b, ql:] == 7.0).all() and (lse[b, ql:] == 7.0).all()
        for h in range(p.Hkv):
            want = scored_want(p, q, b, h, G, ql, p.D ** -0.5, dtype, cap, window, sink, slopes,
                               k=k[b, :, h].double().numpy(), v=v[b, :, h].double().numpy(),
                               parent=parent[b])
            hs = slice(h * G, h * G + G)
            check_attention(out[b, :ql, hs], lse[b, :ql, hs], want, (b, h))
    return out, lse


TREES = [(None, [300, 0, 77], 1, 3), (None, [500, 129, 1], 7, 4), (4096, [3000, 130, 2999], 4, 8),
         (4096, [2500, 0, 31], 13, 4), (None, [700, 90, 333], 60, 2), (9000, [9000, 400, 0], 33, 3),
         (None, [300, 40, 0], 256, 2)]


@pytest.mark.parametrize("shape", TREES, ids=lambda s: f"T{s[2]}G{s[3]}")
@pytest.mark.parametrize("what", ["none", "cap", "window", "sink", "slopes", "all"])
@pytest.mark.parametrize("D,fmt,dtype,block,page", [(128, O.E4M3, "bf16", 64, 64), (64, O.INT8, "f16", 16, 48)])
def test_tree(shape, what, D, fmt, dtype, block, page):
    cap_rows, lens, T, G = shape
    p = filled(3, 2, D, lens, block, page, fmt, seed=31, max_len=cap_rows)
    args = {}
    if what in ("cap", "all"):
        args["cap"], args["size"] = 5.0, 3.0
    if what in ("window", "sink", "all"):
        args["window"] = 130 if what == "all" else 3
    if what in ("sink", "all"):
        args["sink"] = 37
    if what in ("slopes", "all"):
        args["slopes"] = slopes_of(2 * G)
    q_len = None if what == "cap" else [T, max(0, T - 1), min(T, 3)]
    run_tree(p, G, T, dtype, q_len=q_len, scores=what != "none", **args)


@pytest.mark.parametrize("T,G,max_len", [(5, 3, None), (12, 3, 4096), (70, 2, None)])
def test_trees_of_many_shapes(T, G, max_len):
    """A chain, a star, windows that end inside the path, first rows inside it."""
    p = filled(2, 1, 64, [140, 3], 16, 16, O.E4M3, seed=32, max_len=max_len)
    chain = [[i - 1 for i in range(T)]] * 2
    star = [[-1] + [0] * (T - 1), [-1] * T]
    for parent in (chain, star):
        for window, sink in ((0, 0), (1, 0), (4, 0), (4, 5), (2, 1000)):
            run_tree(p, G, T, "bf16", window=window, sink=sink, parent=[list(x) for x in parent])


def test_a_chain_of_drafts_is_the_attention_over_appended_rows():
    """Drafts whose rows 8 bits hold exactly: the tree gives what append and kv8_attn give."""
    for T, G in ((4, 4), (40, 4)):
        p = filled(1, 1, 64, [128], 64, 64, K.KV8_INT8, seed=33, max_len=256)
        q = p.rows(T, G, "f16")
        k, v = (torch.from_numpy(p.rng.integers(-127, 128, (1, T, 1, 64)).astype(np.float32)).half() / 32
                for _ in "kv")
        k[0, 0, 0, 0] = v[0, 0, 0, 0] = 127 / 32
        ws = p.c.tree_workspace(T, G)
        a, b = (torch.empty(q.shape, dtype=q.dtype, device="cuda") for _ in "ab")
        la, lb = (torch.empty(1, T, G, device="cuda") for _ in "ab")
        K.kv8_attn_tree(p.c, q.cuda(), k.cuda(), v.cuda(), ints([[i - 1 for i in range(T)]]), a, ws, lse=la)
        p.append(k, v, ws)
        p.check()
        K.kv8_attn(p.c, q.cuda(), b, ws, lse=lb)
        want = scored_want(p, q, 0, 0, G, T, 0.125, "f16")
        check_attention(a[0].cpu(), la[0].cpu(), want)
        check_attention(b[0].cpu(), lb[0].cpu(), want)


@pytest.mark.parametrize("T,G,max_len", [(6, 4, None), (6, 4, 4096), (40, 4, None)])
def test_bad_parents_and_rows_off_the_path(T, G, max_len):
    p = filled(1, 1, 64, [100], 16, 16, O.E4M3, seed=34, max_len=max_len)
    q, k, v = (p.rows(T, h, "bf16") for h in (G, 1, 1))
    parent = [[-1, 0, 2, 77, 2, 3] + [-1] * (T - 6)]
    k[0, 1] = math.nan               # only token 1 sees it
    v[0, 1] = math.inf
    ws = p.c.tree_workspace(T, G)
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    lse = torch.empty(1, T, G, device="cuda")
    K.kv8_attn_tree(p.c, q.cuda(), k.cuda(), v.cuda(), ints(parent), out, ws, lse=lse)
    assert K.get_status(ws) == K.DEV_BAD_TREE
    assert out[0, 1].isnan().all() and lse[0, 1].isnan().all()
    k[0, 1] = v[0, 1] = 0.0
    want = scored_want(p, q, 0, 0, G, T, 0.125, "bf16", k=k[0, :, 0].double().numpy(),
                       v=v[0, :, 0].double().numpy(), parent=parent[0])
    keep = [i for i in range(T) if i != 1]
    check_attention(out[0, keep].cpu(), lse[0, keep].cpu(), tuple(x[keep] for x in want))


def test_trees_of_many_sequences_and_strides():
    rng = np.random.default_rng(6)
    lens = [int(x) for x in rng.integers(0, 900, 40)]
    p = filled(40, 2, 64, lens, 16, 16, O.INT8, seed=35, max_len=5000)
    run_tree(p, 2, 3, "bf16")
    run_tree(p, 3, 20, "f16", cap=15.0, window=100, sink=20, slopes=slopes_of(6))
    # all from one fused projection, the outputs over the queries
    G, T = 2, 5
    fused = p.rows(T, 8, "bf16")
    parent = tree(rng, 40, T)
    ws = p.c.tree_workspace(T, 4)
    x = fused.cuda()
    K.kv8_attn_tree(p.c, x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], ints(parent), x[:, :, :4], ws)
    y = torch.empty(40, T, 4, 64, dtype=torch.bfloat16, device="cuda")
    K.kv8_attn_tree(p.c, *(fused[:, :, a:b].contiguous().cuda() for a, b in ((0, 4), (4, 6), (6, 8))),
                    ints(parent), y, ws)
    assert torch.equal(x[:, :, :4], y) and torch.equal(x[:, :, 4:].cpu(), fused[:, :, 4:])


@pytest.mark.parametrize("T,G", [(1, 8), (5, 8), (40, 4)])
@pytest.mark.parametrize("what", ["window", "cap", "far", "slopes", "both", "tree"])
def test_scores_that_grow_along_the_rows(T, G, what):
    """Every few rows raise the running maximum, inside tiles too; a cap that few, many
    or all scores reach; and a row in front that stays the largest."""
    for case in range(3):
        p = Pair(2, 1, 64, 900, 32, 32, O.E4M3, seed=41 + case, mass=False)
        ws = p.c.workspace(1, 1)
        k, v = p.rows(900, 1, "f32"), p.rows(900, 1, "f32")
        j = torch.arange(900.0)
        size = [torch.exp(j / 170), torch.exp(2 * torch.sin(j / 9)) * (1 + j / 90), torch.ones(900)][case]
        if case == 2:
            size[3] = 60.0
        p.append(k * size.view(1, -1, 1, 1), v, ws, lens=[900, 517])
        args = {"window": dict(window=700, sink=10), "cap": dict(cap=40.0), "far": dict(cap=3.0),
                "slopes": dict(slopes=slopes_of(G)), "both": dict(cap=25.0, slopes=slopes_of(G)),
                "tree": dict()}[what]
        if what == "tree":
            run_tree(p, G, T, "bf16", size=2.0, chain=0.8)
        else:
            run_scored(p, G, T, "bf16", size=2.0, **args)


@pytest.mark.parametrize("T,G", [(1, 4), (40, 4)])
@pytest.mark.parametrize("value,scale", [(math.inf, 0.0), (-math.inf, 0.0), (3e38, 2.0 ** 20), (-3e38, 2.0 ** 20)])
def test_a_cap_makes_infinite_scores_finite(T, G, value, scale):
    """Scores that are infinite, or beyond fp32, are the cap or its negative: alike for every
    row, whose plain mean comes out."""
    p = Pair(2, 1, 64, 300, 16, 16, O.E4M3, seed=71, mass=False)
    k, v = p.rows(300, 1, "f32"), p.rows(300, 1, "f32")
    k[..., 0] = 2.0
    lens = [300, 171]
    p.append(k, v, p.c.workspace(1, 1), lens=lens)
    q = torch.zeros(2, T, G, 64, dtype=torch.bfloat16)
    q[..., 0] = value
    for drafted in (False, True):
        ws = p.c.tree_workspace(T, G)
        out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(2, T, G, device="cuda")
        sc = K.Scores(cap=30.0)
        if drafted:
            kd = torch.full((2, T, 1, 64), 2.0, dtype=torch.bfloat16, device="cuda")
            vd = torch.full_like(kd, 0.5)
            K.kv8_attn_tree(p.c, q.cuda(), kd, vd, ints([[-1] * T] * 2), out, ws, lse=lse, softmax_scale=scale,
                            scores=sc)
        else:
            K.kv8_attn_scored(p.c, q.cuda(), out, ws, sc, lse=lse, softmax_scale=scale)
        for b in range(2):
            vv = p.seq[b, 0, "v"].values()
            for t in range(T):
                n = lens[b] if drafted else lens[b] - T + t + 1
                rows = np.concatenate([vv, np.full((1, 64), 0.5)]) if drafted else vv[:n]
                mean, size = rows.mean(0), np.abs(rows).mean(0)
                # the rounding of the output, of the weights (all one power of two but for the
                # cap's own rounding) and of the sums
                tol = 2.0 ** -8 * np.abs(mean) + size * (2.0 ** -10 + len(rows) * 2.0 ** -22)
                got = out[b, t].double().cpu().numpy()
                assert (np.abs(got - mean) <= tol).all(), (drafted, b, t)
                want = math.copysign(30.0, value) + math.log(len(rows))
                assert np.abs(lse[b, t].double().cpu().numpy() - want).max() < 30 * 2.0 ** -20 + 1e-5
