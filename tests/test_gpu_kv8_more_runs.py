"""Rotated, scored and drafted tokens together, as they are used: decode steps and
drafting rounds against the oracle, captured and replayed, on streams of their own,
in storage beyond 4 GiB, and the README's example."""
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
from kv8_tools import DT, Pair  # noqa: E402
from kv8_more_tools import check_attention, ints, rope, rotated, scored_want, tree  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def slopes_of(H):
    return (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32)


@pytest.mark.parametrize("Hkv,G,D,block,page,fmt,dtype,what", [
    (2, 4, 128, 64, 64, O.E4M3, "bf16", "cap"), (1, 7, 64, 16, 48, O.INT8, "f16", "window"),
    (3, 3, 64, 128, 0, O.E4M3, "bf16", "slopes")])
def test_prompt_steps_and_drafting_rounds(Hkv, G, D, block, page, fmt, dtype, what):
    """A prompt, single tokens, and rounds of drafted trees of which a path is kept."""
    B, H, R = 3, Hkv * G, D // 2
    p = Pair(B, Hkv, D, 700, block, page, fmt, seed=51, mass=False)
    ws = p.c.tree_workspace(64, H)
    ws = torch.cat([ws, torch.zeros(max(0, p.c.workspace(300, H).numel() - ws.numel()), dtype=torch.uint8,
                                    device="cuda")])
    r, c, s = rope(800, R, D - R, O.PAIRS if G == 7 else O.HALVES)
    style = O.PAIRS if G == 7 else O.HALVES
    args = {"cap": dict(cap=12.0), "window": dict(window=70, sink=5), "slopes": dict(slopes=slopes_of(H))}[what]
    sc = K.Scores(**{k: torch.from_numpy(v).cuda() if k == "slopes" else v for k, v in args.items()})
    dt = DT[dtype]

    def check(q, out, lse, lens, **more):
        for b in range(B):
            for h in range(Hkv):
                kw = {k: (v[b][:, h].double().numpy() if k in "kv" else v[b]) for k, v in more.items()}
                want = scored_want(p, q, b, h, G, lens[b], D ** -0.5, dtype, **args, **kw)
                hs = slice(h * G, h * G + G)
                check_attention(out[b, :lens[b], hs].cpu(), lse[b, :lens[b], hs].cpu(), want, (b, h))

    for T, lens in [(300, [300, 41, 128]), (1, [1, 1, 1]), (1, [1, 0, 1])]:
        fused = p.rows(T, H + 2 * Hkv, dtype)
        x = fused.cuda()
        q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
        K.kv8_append_rope(p.c, k, v, r, ws, q=q, q_out=q, new_len=ints(lens))
        at = [[n + i for i in range(T)] for n in p.len]
        turned = rotated(fused, at, c, s, D - R, style)
        for b in range(B):
            for h in range(Hkv):
                p.seq[b, h, "k"].append(turned[b, :lens[b], H + h].double().numpy())
                p.seq[b, h, "v"].append(fused[b, :lens[b], H + Hkv + h].double().numpy())
            p.len[b] += lens[b]
        p.check()
        out, lse = torch.empty(B, T, H, D, dtype=dt, device="cuda"), torch.empty(B, T, H, device="cuda")
        K.kv8_attn_scored(p.c, q, out, ws, sc, lse=lse, q_len=ints(lens))
        check(turned[:, :, :H].to(dt), out, lse, lens)
    for T, lens in [(12, [12, 7, 0]), (64, [64, 64, 33]), (1, [1, 1, 1])]:
        fused = p.rows(T, H + 2 * Hkv, dtype)
        x = fused.cuda()
        q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
        parent = tree(p.rng, B, T)
        par = ints(parent)
        K.kv8_rope(p.c, q, q, r, ws, k=k, k_out=k, q_len=ints(lens), parent=par)
        paths = [[O.path_to(parent[b], i)[::-1] for i in range(lens[b])] for b in range(B)]
        at = [[p.len[b] + len(O.path_to(parent[b], i)) - 1 for i in range(T)] for b in range(B)]
        turned = rotated(fused, at, c, s, D - R, style).to(dt)
        out, lse = torch.empty(B, T, H, D, dtype=dt, device="cuda"), torch.empty(B, T, H, device="cuda")
        K.kv8_attn_tree(p.c, q, k, v, par, out, ws, lse=lse, q_len=ints(lens), scores=sc)
        check(turned[:, :, :H], out, lse, lens, k=turned[:, :, H:H + Hkv], v=fused[:, :, H + Hkv:], parent=parent)
        # the longest path is kept, without its last token
        kept = [max(x, key=len)[:-1] if x else [] for x in paths]
        M = max(1, max(map(len, kept)))
        path = torch.zeros(B, M, dtype=torch.int32)
        for b in range(B):
            path[b, :len(kept[b])] = torch.tensor(kept[b], dtype=torch.int32)
        K.kv8_append_path(p.c, k, v, path.cuda(), ws, new_len=ints([len(x) for x in kept]))
        for b in range(B):
            for h in range(Hkv):
                p.seq[b, h, "k"].append(turned[b, kept[b], H + h].double().numpy())
                p.seq[b, h, "v"].append(fused[b, kept[b], H + Hkv + h].double().numpy())
            p.len[b] += len(kept[b])
        p.check()
    assert K.get_status(ws) == 0


def test_steps_captured_and_replayed():
    """One graph of a step's four calls, replayed as the cache grows, gives what eager calls
    give on a cache of their own; two graphs share a workspace."""
    B, Hkv, G, D, T = 3, 2, 4, 64, 6
    H = Hkv * G
    r, _, _ = rope(600, 64)
    sc = K.Scores(cap=20.0, window=100, sink=4)
    pairs = [Pair(B, Hkv, D, 512, 16, 16, O.E4M3, seed=61, mass=False) for _ in "ab"]
    for p in pairs:
        p.append(p.rows(200, Hkv, "bf16"), p.rows(200, Hkv, "bf16"), p.c.workspace(1, Hkv), lens=[200, 3, 90])
    rng = np.random.default_rng(62)
    feed = pairs[0].rows(T, H + 2 * Hkv, "bf16").cuda()
    par, path, m = ints(tree(rng, B, T)), ints([[0, 2]] * B), ints([2, 1, 0])
    ws = pairs[0].c.tree_workspace(T, H)

    def step(c, x, o, l, o2, l2, y):
        q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
        K.kv8_rope(c, q, y[:, :, :H], r, ws, k=k, k_out=y[:, :, H:], parent=par)
        K.kv8_attn_tree(c, y[:, :, :H], y[:, :, H:], v, par, o, ws, lse=l, scores=sc)
        K.kv8_append_path(c, y[:, :, H:], v, path, ws, new_len=m)
        K.kv8_append_rope(c, k[:, :1], v[:, :1], r, ws, q=q[:, :1], q_out=y[:, :1, :H])
        K.kv8_attn_scored(c, y[:, :1, :H], o2, ws, sc, lse=l2)

    def buffers():
        f = dict(device="cuda")
        return (torch.zeros(B, T, H, D, dtype=torch.bfloat16, **f), torch.zeros(B, T, H, **f),
                torch.zeros(B, 1, H, D, dtype=torch.bfloat16, **f), torch.zeros(B, 1, H, **f),
                torch.zeros(B, T, H + Hkv, D, dtype=torch.bfloat16, **f))

    captured, eager = buffers(), buffers()
    graphs = []
    start = pairs[0].c.seq_len.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step(pairs[0].c, feed, *captured)
            graphs.append(g)
    torch.cuda.synchronize()
    assert torch.equal(pairs[0].c.seq_len, start)
    for i in range(6):
        feed.copy_(pairs[1].rows(T, H + 2 * Hkv, "bf16"))
        graphs[i % 2].replay()
        step(pairs[1].c, feed, *eager)
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b), i
        for n in ("seq_len", "k_codes", "v_codes", "k_scales", "v_scales"):
            a, b = (getattr(x.c, n) for x in pairs)
            assert torch.equal(a.nan_to_num(5.0) if a.is_floating_point() else a,
                               b.nan_to_num(5.0) if b.is_floating_point() else b), n
    assert pairs[0].c.seq_len.tolist() == [200 + 18, 3 + 12, 90 + 6]
    assert K.get_status(ws) == 0


def test_streams_and_repeats():
    """On a stream that waits for another's inputs; the same call gives the same bits."""
    B, Hkv, G, D = 4, 2, 8, 128
    p = Pair(B, Hkv, D, 4096, 64, 64, O.E4M3, seed=63, mass=False)
    p.append(p.rows(3000, Hkv, "bf16"), p.rows(3000, Hkv, "bf16"), p.c.workspace(1, Hkv), lens=[3000, 100, 2222, 1])
    for T in (1, 5, 40):
        q, k, v = (p.rows(T, h, "bf16").cuda() for h in (Hkv * G, Hkv, Hkv))
        par = ints(tree(p.rng, B, T))
        sc = K.Scores(cap=30.0, slopes=torch.from_numpy(slopes_of(Hkv * G)).cuda())
        torch.cuda.synchronize()
        res = []
        for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
            ws = p.c.tree_workspace(T, Hkv * G)
            o = [torch.zeros_like(q) for _ in "ab"]
            l = [torch.zeros(B, T, Hkv * G, device="cuda") for _ in "ab"]
            stream.wait_stream(torch.cuda.current_stream())
            K.kv8_attn_scored(p.c, q, o[0], ws, sc, lse=l[0], stream=stream)
            K.kv8_attn_tree(p.c, q, k, v, par, o[1], ws, lse=l[1], scores=sc, stream=stream.cuda_stream)
            stream.synchronize()
            res.append(o + l)
        for x in res[1:]:
            assert all(torch.equal(a, b) for a, b in zip(res[0], x))


@pytest.mark.parametrize("T,G", [(1, 4), (40, 4)])
def test_storage_beyond_4_gib(T, G):
    B, Hkv, D, block, cap, H = 40, 8, 128, 64, 131072, 8 * G
    p = Pair(B, Hkv, D, block, block, 0, O.E4M3, seed=64, mass=False)
    p.c = K.Cache8(B, Hkv, D, cap, block=block, fmt=O.E4M3)
    assert p.c.k_codes.numel() > 2 ** 32
    p.len = [0] * B
    ws = p.c.tree_workspace(max(T, 8), H)
    r, c, s = rope(500, 128)
    lens = [0] * (B - 1) + [300]
    k, v = p.rows(300, Hkv, "bf16"), p.rows(300, Hkv, "bf16")
    K.kv8_append_rope(p.c, k.cuda(), v.cuda(), r, ws, new_len=ints(lens))
    turned = rotated(k, [list(range(300))] * B, c, s, 0, O.HALVES)
    for h in range(Hkv):
        p.seq[B - 1, h, "k"].append(turned[B - 1, :, h].double().numpy())
        p.seq[B - 1, h, "v"].append(v[B - 1, :, h].double().numpy())
    p.len[-1] = 300
    K.kv8_append_path(p.c, k.cuda(), v.cuda(), ints([[7, 5]] * B), ws, new_len=ints([0] * (B - 1) + [2]))
    for h in range(Hkv):
        p.seq[B - 1, h, "k"].append(k[B - 1, [7, 5], h].double().numpy())
        p.seq[B - 1, h, "v"].append(v[B - 1, [7, 5], h].double().numpy())
    p.len[-1] = 302
    b = B - 1
    assert p.c.seq_len.tolist() == p.len
    for h in range(Hkv):
        for side in "kv":
            got = O.decode(getattr(p.c, side + "_codes")[b, h, :302].cpu().numpy(), O.E4M3)
            assert np.array_equal(got, p.seq[b, h, side].codes)
    q, k, v = (p.rows(T, h, "bf16", 0.7) for h in (H, Hkv, Hkv))
    parent = tree(p.rng, B, T)
    for drafted in (False, True):
        out, lse = torch.empty(B, T, H, D, dtype=q.dtype, device="cuda"), torch.empty(B, T, H, device="cuda")
        if drafted:
            K.kv8_attn_tree(p.c, q.cuda(), k.cuda(), v.cuda(), ints(parent), out, ws, lse=lse)
        else:
            K.kv8_attn_scored(p.c, q.cuda(), out, ws, K.Scores(cap=9.0, window=200), lse=lse)
        for h in range(Hkv):
            more = (dict(k=k[b, :, h].double().numpy(), v=v[b, :, h].double().numpy(), parent=parent[b])
                    if drafted else dict(cap=9.0, window=200))
            want = scored_want(p, q, b, h, G, T, D ** -0.5, "bf16", **more)
            hs = slice(h * G, h * G + G)
            check_attention(out[b, :, hs].cpu(), lse[b, :, hs].cpu(), want, h)
    assert K.get_status(ws) == 0


def test_the_readme_example():
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python3\n(.*?)```", text, re.S)
    assert len(blocks) == 1
    torch.manual_seed(0)
    env = {}
    exec(compile(blocks[0], "README.md", "exec"), env)
    torch.cuda.synchronize()
    n = env["cache"].seq_len.tolist()
    assert n == [env["prompt"] + 1 + len(x) for x in env["kept"]]
    assert torch.isfinite(env["out"].float()).all() and torch.isfinite(env["out_tree"].float()).all()
