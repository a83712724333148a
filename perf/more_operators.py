"""The 8-bit K/V cache's operators for rotated, scored and drafted tokens.

Five operators over the cache of grouped heads (codes in 8 bits, one power of two
as the scale of each block of rows and head):

  rope         rotate the channel pairs of query and key rows by their positions
               (in a row, given, or those of a tree of drafted tokens);
  rope_append  rotate new K rows on their way into the cache, append V beside
               them, and rotate the step's queries;
  path         append the rows of the drafted tokens on an accepted path;
  scored       attention whose scores are capped by a tanh, lowered by a slope
               times the distance, and masked by a window with first rows and by
               a prefix that every query sees;
  tree         attention of drafted tokens over the cache and over the drafted
               rows on their own path to the root.

`run` computes them in elementary torch operations in 32 bits, or, with `own`
set, through the package.  `exact` states them once more in 64 bits.
"""
import math
import random

import torch

own = False

E4M3, INT8 = "e4m3", "int8"
QMAX = {E4M3: 448.0, INT8: 127.0}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALVES, PAIRS = "halves", "pairs"


# ------------------------------------------------------------------- the cases
def _case(name, op, B, T, N, Hkv, G, D, dtype, fmt, block, page, ragged, R=0, first=0, style=HALVES,
          where="", M=0, cap=0.0, window=0, sink=0, slopes=False, prefix=0):
    return {"name": name, "op": op, "B": B, "T": T, "N": N, "Hkv": Hkv, "G": G, "D": D,
            "dtype": dtype, "fmt": fmt, "block": block, "page": page, "ragged": ragged, "R": R,
            "first": first, "style": style, "where": where, "M": M, "cap": cap, "window": window,
            "sink": sink, "slopes": slopes, "prefix": prefix}


def listed():
    return [
        # one decode step of 32 sequences: a token's queries, K and V from a fused projection
        _case("rope_append_token_b32", "rope_append", 32, 1, 2048, 8, 8, 128, "bf16", E4M3, 64, 64, True,
              R=128),
        # four prompts of different lengths, padded to the longest
        _case("rope_append_prompts_b4", "rope_append", 4, 8192, 8192, 8, 8, 128, "bf16", E4M3, 64, 64,
              True, R=128),
        # drafted tokens of a batch, at the positions of their trees, half of the channels
        _case("rope_tree_b16", "rope", 16, 60, 9001, 4, 8, 128, "bf16", E4M3, 64, 64, True, R=64,
              where="tree"),
        # queries and keys of a long prompt whose positions are not those of its rows
        _case("rope_prompt", "rope", 1, 16384, 16384, 8, 8, 128, "bf16", E4M3, 64, 0, False, R=128,
              style=PAIRS, where="pos"),
        # the accepted tokens of a batch's trees
        _case("path_b16", "path", 16, 60, 9001, 4, 8, 128, "bf16", E4M3, 64, 64, True, M=8),
        # a long accepted chain of one sequence, small pages
        _case("path_long", "path", 1, 256, 40000, 8, 4, 64, "f16", INT8, 16, 16, False, M=200),
        # a serving batch of a model that caps its scores
        _case("capped_token_b32", "scored", 32, 1, 32768, 8, 8, 128, "bf16", E4M3, 64, 64, True,
              cap=30.0),
        # long contexts of which a layer sees a window and the first rows
        _case("window_token_b8", "scored", 8, 1, 131072, 8, 4, 128, "bf16", INT8, 128, 0, False,
              window=4096, sink=4),
        # a chunk of a long prompt, capped, in a layer without a window
        _case("capped_chunk", "scored", 1, 4096, 16384, 8, 8, 128, "bf16", E4M3, 64, 64, False,
              cap=30.0),
        # prompts of odd lengths with a bias by distance and a prefix that is seen both ways
        _case("biased_prompts_b3", "scored", 3, 1501, 1501, 4, 4, 64, "f16", INT8, 32, 64, True,
              slopes=True, prefix=200),
        # a few drafted tokens, one sequence, a short context: latency alone
        _case("tree_b1", "tree", 1, 7, 1000, 2, 7, 128, "bf16", E4M3, 64, 64, False),
        # trees of 60 drafted tokens verified for a batch
        _case("tree_b16", "tree", 16, 60, 9001, 4, 8, 128, "bf16", E4M3, 64, 64, True),
    ]


def _cost(c):
    w = work(c)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def draw(rng):
    logs = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["rope_append", "rope", "path", "scored", "scored", "scored", "tree", "tree"])
        B = logs(1, 32)
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        D = rng.choice([64, 128, 128])
        block = rng.choice([16, 32, 64, 128])
        page = rng.choice([0, block, 2 * block, 128])
        N = logs(60, 131072)
        many = rng.random() < 0.5
        T = min(N, logs(32, 4096) if many else rng.choice([1, 1, 1, 2, 3, 5]))
        R = first = M = window = sink = prefix = 0
        where, cap, slopes = "", 0.0, False
        style = rng.choice([HALVES, HALVES, PAIRS])
        if op in ("rope_append", "rope"):
            R = rng.choice([16, 32, 64, 64, 128])
            if R > D:
                continue
            first = rng.choice([0, 0, D - R])
            where = rng.choice(["", "pos"] + (["tree"] if op == "rope" else []))
        if op in ("path", "tree") or where == "tree":
            T = min(N, rng.choice([1, 4, 8, 16, 31, 60, 64, 100, 200]))
        if op == "path":
            M = rng.randint(1, T)
        if op in ("scored", "tree"):
            kinds = rng.sample(["cap", "window", "slopes", "prefix"], rng.choice([1, 1, 2, 3]))
            if op == "tree":
                kinds = [k for k in kinds if k != "prefix"] if rng.random() < 0.5 else []
            cap = rng.choice([15.0, 30.0, 50.0]) if "cap" in kinds else 0.0
            if "window" in kinds:
                window, sink = logs(1, N), rng.choice([0, 0, 4, 130])
            slopes = "slopes" in kinds
            prefix = rng.randint(1, N) if "prefix" in kinds else 0
        dtype = rng.choice(["bf16", "f16"] + (["f32"] if op in ("rope_append", "path") else []))
        c = _case("", op, B, T, N, Hkv, G, D, dtype, rng.choice([E4M3, E4M3, INT8]), block, page,
                  rng.random() < 0.6, R, first, style, where, M, cap, window, sink, slopes, prefix)
        del c["name"]
        scores = B * Hkv * G * T * N if op in ("scored", "tree") else 0  # the plain form holds them whole
        if _cost(c) <= most and scores <= 1.2e9 and B * Hkv * N * D <= 1.1e9:
            return c


def _lengths(c):
    """(rows held per sequence once the call is done, its new rows, queries or drafts).
    The drafts of rope, path and tree come behind the rows that are held."""
    B, N, T = c["B"], c["N"], c["T"]
    if not c["ragged"]:
        return [N] * B, [T] * B
    n = [max(1, N - (b * N * 5) // (8 * B) - (13 * b) % 61) if b else N for b in range(B)]
    t = [min(x, T if T <= 8 else max(1, T - (b * T * 3) // (4 * B))) for b, x in enumerate(n)]
    return n, t


def _parents(c, t, seed):
    """Trees as a drafting model grows them: a token follows the one before it or any earlier one."""
    rng = random.Random(seed)
    out = [[-1] * c["T"] for _ in t]
    for b, x in enumerate(t):
        for i in range(1, x):
            out[b][i] = i - 1 if rng.random() < 0.35 else rng.randint(-1, i - 1)
    return out


def _path_to(parent, i):
    """The tokens from the root to token i."""
    path = []
    while i >= 0:
        path.append(i)
        i = parent[i]
    return path[::-1]


def _lows(c, p0, p1):
    """Rows in front of the window and behind the first ones for queries at p0 .. p1 - 1: their sum."""
    if not c["window"]:
        return 0
    return sum(max(0, p - c["window"] + 1 - c["sink"]) for p in range(p0, p1))


def work(c):
    B, Hkv, G, D, T, R = c["B"], c["Hkv"], c["G"], c["D"], c["T"], c["R"]
    n, t = _lengths(c)
    es = 4 if c["dtype"] == "f32" else 2
    new = sum(t)
    table = min(sum(t), max(t) if c["where"] else max(n)) * R * 4
    if c["op"] == "rope":
        return {"bytes": new * Hkv * (G + 1) * D * es * 2 + table + 4 * new, "flops": 3 * Hkv * (G + 1) * R * new}
    if c["op"] in ("rope_append", "path"):
        rows = min(new, B * c["M"]) if c["op"] == "path" else new
        q = 0 if c["op"] == "path" else new * Hkv * G * D * es * 2
        touched = sum(-(-x // c["block"]) for x in ([min(x, c["M"]) for x in t] if c["M"] else t))
        return {"bytes": q + 2 * Hkv * (rows * D * (es + 1) + touched * 4) + table + 8 * B,
                "flops": 4 * Hkv * rows * D + 3 * Hkv * (G + 1) * R * new * (q > 0)}
    pairs = rows = 0
    for x, y in zip(n, t):
        if c["op"] == "tree":          # (the drafts' own pairs: at most a path's)
            p0, y1 = x, x
            see = y * x - (min(_lows(c, x, x + 1), x) * y if c["window"] else 0)
            low = _lows(c, x, x + 1)
        else:
            p0 = x - y
            see = sum(min(x, max(p + 1, c["prefix"])) - min(_lows(c, p, p + 1), x)
                      for p in range(p0, x))
            low = _lows(c, p0, p0 + 1)
        pairs += max(see, 0) * Hkv * G
        rows += max(1, x - low)
    queries = new * Hkv * G
    drafts = 2 * new * Hkv * D * es if c["op"] == "tree" else 0
    return {"bytes": int(2 * Hkv * rows * (D + 4 / c["block"]) + queries * (2 * D * es + 4) + drafts),
            "flops": 4 * D * pairs}


# ------------------------------------------------------------------ the inputs
def _pow2_scale(amax, fmt):
    """The smallest power of two s >= 2^-126 with amax <= qmax * s; 0 for amax 0."""
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [1/2, 1)
    top, lead = (9, 0.875) if fmt == E4M3 else (7, 127 / 128)   # qmax = lead * 2^top
    e = (e - top + (m > lead)).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _encode(x, scale, fmt):
    """x over its scale, rounded to the format's nearest value (ties to even)."""
    y = torch.where(scale > 0, x / torch.where(scale > 0, scale, 1.0), 0.0)
    if fmt == E4M3:
        return y.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(y).to(torch.int8).view(torch.uint8)


def _values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == E4M3 else torch.int8).to(torch.float32)


def _store(c, rows_cap, dev, gen):
    """Empty storage for a cache of the case, [pages, Hkv, page rows, D]."""
    B, Hkv, D, block, page = c["B"], c["Hkv"], c["D"], c["block"], c["page"]
    s = {}
    if page:
        per_seq = -(-rows_cap // page)
        pages = B * per_seq + 3
        s["page_table"] = torch.randperm(pages, generator=gen, device=dev)[: B * per_seq].to(
            torch.int32).view(B, per_seq)
        ps = page
        s["max_len"] = per_seq * page
    else:
        pages, ps = B, -(-rows_cap // block) * block
        s["page_table"] = None
        s["max_len"] = ps
    for x in "kv":
        s[x + "_codes"] = torch.zeros((pages, Hkv, ps, D), dtype=torch.uint8, device=dev)
        s[x + "_scales"] = torch.zeros((pages, Hkv, ps // block), device=dev)
    s["seq_len"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return s


def _table(c, s):
    if s["page_table"] is not None:
        return s["page_table"].long()
    return torch.arange(c["B"], device=s["seq_len"].device).view(-1, 1)


def _channels(gen, dev, Hkv, D):
    """Sizes of a projection's channels: uneven, a few of them large."""
    return torch.exp(0.6 * torch.randn((Hkv, 1, D), generator=gen, device=dev))


def _rows(gen, dev, B, Hkv, N, D, ch):
    """Rows as projections give them: uneven channels, and tokens whose size varies."""
    tok = torch.exp(0.3 * torch.randn((B, Hkv, N, 1), generator=gen, device=dev))
    return torch.randn((B, Hkv, N, D), generator=gen, device=dev) * ch * tok


def _handle(c, s):
    import fp4_kv_cache_rope_gb300 as K
    fmt = K.KV8_E4M3 if c["fmt"] == E4M3 else K.KV8_INT8
    return K.Cache8(c["B"], c["Hkv"], c["D"], s["max_len"], block=c["block"],
                    page_size=c["page"], page_table=s["page_table"],
                    num_pages=s["k_codes"].shape[0] if c["page"] else 0, fmt=fmt,
                    tensors={k: s[k] for k in ("k_codes", "v_codes", "k_scales", "v_scales", "seq_len")})


def prepare(c, seed):
    dev = torch.device("cuda", 0) if torch.cuda.is_available() else torch.device("cpu")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, B, T, N, Hkv, G, D, R = (c[x] for x in ("op", "B", "T", "N", "Hkv", "G", "D", "R"))
    H = Hkv * G
    dt = DTYPES[c["dtype"]]
    n, t = _lengths(c)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cap_rows = N + (c["M"] if op == "path" else 0)
    S = {"c": c, "s": _store(c, cap_rows, dev, gen)}
    s = S["s"]
    kch, vch = (_channels(gen, dev, Hkv, D) for _ in "kv")
    # what the cache holds before the call
    held = [x - y for x, y in zip(n, t)] if op == "rope_append" else n
    hmax = max(held)
    if hmax and op != "rope":
        blk, cap = c["block"], s["max_len"]
        for b in range(B):
            for x, ch in (("k", kch), ("v", vch)):
                rows = _rows(gen, dev, 1, Hkv, hmax, D, ch)
                rows = torch.nn.functional.pad(rows[0, :, :held[b]], (0, 0, 0, cap - held[b]))
                r = rows.view(Hkv, cap // blk, blk, D)
                sc = _pow2_scale(r.abs().amax((2, 3)), c["fmt"])
                codes = _encode(r, sc[..., None, None], c["fmt"]).view(Hkv, cap, D)
                tab = _table(c, s)[b]
                ps = cap // len(tab)
                s[x + "_codes"][tab] = codes.view(Hkv, len(tab), ps, D).transpose(0, 1)
                s[x + "_scales"][tab] = sc.view(Hkv, len(tab), ps // blk).transpose(0, 1)
    s["seq_len"].copy_(ints(held))
    S["len"] = ints(t) if c["ragged"] and T > 1 else None
    S["start"] = ints(held)
    q = torch.randn((B, T, Hkv, G, D), generator=gen, device=dev) * (1.0 / kch).view(Hkv, 1, D)
    q = q * (4.0 if c["cap"] else 1.5)             # (scores that come near the cap)
    # the three parts of a fused projection's output
    fused = torch.cat([q.view(B, T, H, D)] + [_rows(gen, dev, B, Hkv, T, D, ch).transpose(1, 2)
                                              for ch in (kch, vch)], 2).to(dt)
    S["fused"] = fused
    S["q"], S["k"], S["v"] = fused[:, :, :H], fused[:, :, H:H + Hkv], fused[:, :, H + Hkv:]
    S["parent"] = ints(_parents(c, t, seed))
    if R:
        far = max(n) + T + 77
        ang = torch.arange(far, dtype=torch.float64, device=dev)[:, None] * torch.pow(
            10000.0, -2.0 * torch.arange(R // 2, dtype=torch.float64, device=dev) / R)
        S["cos"], S["sin"] = torch.cos(ang).float(), torch.sin(ang).float()
        S["pos"] = None
        if c["where"] == "pos":
            S["pos"] = torch.randint(0, far, (B, T), generator=gen, device=dev, dtype=torch.int32)
        S["k_out"] = torch.zeros((B, T, Hkv, D), dtype=dt, device=dev)
        S["q_out"] = torch.zeros((B, T, H, D), dtype=dt, device=dev)
    if op == "path":
        path, m = torch.zeros((B, c["M"]), dtype=torch.int32), []
        rng = random.Random(seed + 1)
        for b, par in enumerate(S["parent"].tolist()):
            chain = _path_to(par, rng.randrange(t[b])) if c["M"] < T // 2 else list(range(t[b]))
            m.append(min(c["M"], len(chain)))
            path[b, :m[b]] = torch.tensor(chain[:m[b]], dtype=torch.int32)
        S["path"], S["m"] = path.to(dev), ints(m)
    if op in ("scored", "tree"):
        S["slopes"] = None
        if c["slopes"]:
            S["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device=dev) / H).float()
        S["prefix"] = None
        if c["prefix"]:
            S["prefix"] = ints([max(0, c["prefix"] - 17 * b) for b in range(B)])
        S["out"] = torch.zeros((B, T, H, D), dtype=dt, device=dev)
        S["lse"] = torch.zeros((B, T, H), device=dev)
    if own:
        import fp4_kv_cache_rope_gb300 as K
        S["cache"] = _handle(c, s)
        S["ws"] = S["cache"].tree_workspace(T, H) if op == "tree" else S["cache"].workspace(T, H)
        if R:
            S["rope"] = K.Rope(S["cos"], S["sin"], first=c["first"],
                               style=K.ROPE_HALVES if c["style"] == HALVES else K.ROPE_PAIRS)
        if op in ("scored", "tree"):
            S["scores"] = K.Scores(cap=c["cap"], window=c["window"], sink=c["sink"],
                                   slopes=S["slopes"], prefix=S["prefix"])
    return S


# ------------------------------------------------------------- the plain forms
def _gather(c, s, what):
    """[B, Hkv, rows, ...] of a paged array [pages, Hkv, page rows, ...]."""
    x = s[what][_table(c, s)].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])


def _dequantised(c, s, x):
    scale = _gather(c, s, x + "_scales").repeat_interleave(c["block"], 2)
    return _values(_gather(c, s, x + "_codes"), c["fmt"]) * scale[..., None]


def _depths(parent):
    """[B, T] depths of the tokens (a root's is 0)."""
    depth, at = torch.zeros_like(parent), parent
    for _ in range(parent.shape[1]):
        depth = depth + (at >= 0)
        at = torch.where(at >= 0, parent.gather(1, at.clamp(min=0).long()), at)
    return depth


def _new_len(S):
    n = S["start"].long()
    return S["len"].long() if S["len"] is not None else torch.full_like(n, S["c"]["T"])


def _positions(S):
    """[B, T] positions at which rows are rotated."""
    if S["pos"] is not None:
        return S["pos"].long()
    first = S["start"].long().view(-1, 1)
    if S["c"]["where"] == "tree":
        return first + _depths(S["parent"]).long()
    return first + torch.arange(S["c"]["T"], device=first.device)


def _rotate(S, x):
    """Rows x [B, T, heads, D] in 32 bits, each product and sum rounded once."""
    c = S["c"]
    x, f, R = x.float(), c["first"], c["R"]
    p = _positions(S)
    cos, sin = S["cos"][p][:, :, None], S["sin"][p][:, :, None]
    part = x[..., f:f + R]
    a, b = (part[..., : R // 2], part[..., R // 2:]) if c["style"] == HALVES else (part[..., ::2],
                                                                                 part[..., 1::2])
    ya, yb = a * cos - b * sin, a * sin + b * cos
    y = torch.cat([ya, yb], -1) if c["style"] == HALVES else torch.stack([ya, yb], -1).flatten(-2)
    return torch.cat([x[..., :f], y, x[..., f + R:]], -1)


def _real(S, t):
    """[B, T]: the rows that count."""
    return torch.arange(S["c"]["T"], device=t.device) < t.view(-1, 1)


def _plain_rope(S):
    real = _real(S, _new_len(S))[..., None, None]
    return tuple(torch.where(real, _rotate(S, x).to(x.dtype), torch.zeros_like(x))
                 for x in (S["q"], S["k"]))


def _scatter_rows(c, s, what, b, h, p, ok, x):
    """s[what] at positions p of (b, h), where ok."""
    tab = _table(c, s)
    ps = s[what].shape[2]
    p = torch.where(ok, p, 0)
    page = tab.expand(c["B"], -1)[b, p // ps]
    at = (page * c["Hkv"] + h) * ps + p % ps
    flat = s[what].view(-1, *s[what].shape[3:])
    flat[at[ok]] = x[ok]


def _append(S, k, v, t):
    """Rows k, v [B, T, Hkv, D] in 32 bits, t of each sequence, at its start."""
    c, s = S["c"], S["s"]
    B, Hkv, D, blk, T = c["B"], c["Hkv"], c["D"], c["block"], k.shape[1]
    dev = s["seq_len"].device
    start = S["start"].long()
    nb = (T + blk - 2) // blk + 1                  # blocks that T rows can touch
    p = (start // blk * blk).view(-1, 1) + torch.arange(nb * blk, device=dev)
    old = p < start.view(-1, 1)
    i = p - start.view(-1, 1)
    new = (i >= 0) & (i < t.view(-1, 1))
    cap = s["max_len"]
    bh = torch.arange(B, device=dev).view(-1, 1, 1), torch.arange(Hkv, device=dev).view(1, -1, 1)
    sees = lambda m: m.view(B, 1, nb, blk).expand(B, Hkv, nb, blk)  # noqa: E731
    pb, touched = p.view(B, 1, nb, blk)[..., 0].expand(B, Hkv, nb), sees(new).any(-1)
    for x, rows in (("k", k), ("v", v)):
        rows = rows.transpose(1, 2)                # [B, Hkv, T, D]
        at = i.clamp(0, T - 1).view(B, 1, -1, 1).expand(B, Hkv, -1, D)
        rows = torch.where(new.view(B, 1, -1, 1), rows.gather(2, at), 0.0).view(B, Hkv, nb, blk, D)
        pc = p.clamp(max=cap - 1)
        was = _values(_gather(c, s, x + "_codes")[bh[0], bh[1], pc.view(B, 1, -1)], c["fmt"])
        was = was.view(B, Hkv, nb, blk, D)
        had = sees(old).any(-1)
        s0 = _gather(c, s, x + "_scales")[bh[0], bh[1], pb.clamp(max=cap - 1) // blk]
        s0 = torch.where(had, s0, 0.0)
        s1 = torch.maximum(s0, _pow2_scale(rows.abs().amax((3, 4)), c["fmt"]))
        rows = torch.where(sees(old)[..., None], was * s0[..., None, None], rows)
        codes = _encode(rows, s1[..., None, None], c["fmt"])
        ok = (sees(old | new) & touched[..., None]).reshape(B, Hkv, -1)
        b3, h3 = (y.expand(B, Hkv, nb * blk) for y in bh)
        _scatter_rows(c, s, x + "_codes", b3, h3, p.view(B, 1, -1).expand(B, Hkv, -1), ok,
                      codes.view(B, Hkv, nb * blk, D))
        tab, ps = _table(c, s), s[x + "_codes"].shape[2]
        page = tab[bh[0], torch.where(touched, pb, 0) // ps]
        s[x + "_scales"][page[touched], bh[1].expand(B, Hkv, nb)[touched],
                         (pb % ps // blk)[touched]] = s1[touched]
    s["seq_len"].copy_((start + t).int())
    return _stored(c, s)


def _stored(c, s):
    """What the cache holds, as the values that the codes stand for."""
    kind = torch.float8_e4m3fn if c["fmt"] == E4M3 else torch.int8
    return {"k": s["k_codes"].view(kind), "v": s["v_codes"].view(kind),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"], "seq_len": s["seq_len"]}


def _plain_rope_append(S):
    t = _new_len(S)
    real = _real(S, t)[..., None, None]
    q = torch.where(real, _rotate(S, S["q"]).to(S["q"].dtype), torch.zeros_like(S["q"]))
    return {"q": q, **_append(S, _rotate(S, S["k"]), S["v"].float(), t)}


def _plain_path(S):
    at = S["path"].long()[:, :, None, None].expand(-1, -1, S["c"]["Hkv"], S["c"]["D"])
    return _append(S, S["k"].gather(1, at).float(), S["v"].gather(1, at).float(), S["m"].long())


def _change(S, x, dist):
    """Scores x [B, Hkv, T, G, rows] capped and lowered by their distances [B, T, rows]."""
    c = S["c"]
    if c["cap"]:
        x = x.mul_(1.0 / c["cap"]).tanh_().mul_(c["cap"])
    if S["slopes"] is not None:
        slope = S["slopes"].view(c["Hkv"], 1, c["G"], 1)
        x = x.sub_(slope * dist.float().abs()[:, None, :, None, :])
    return x


def _in_window(c, dist, j):
    """dist: the query's position less the row's j."""
    if not c["window"]:
        return torch.ones_like(dist, dtype=torch.bool)
    return (dist < c["window"]) | (j < c["sink"])


def _plain_attn(S):
    c, s = S["c"], S["s"]
    B, T, Hkv, G, D = c["B"], c["T"], c["Hkv"], c["G"], c["D"]
    k = _dequantised(c, s, "k")
    n, t = s["seq_len"].long().view(-1, 1, 1), _new_len(S).view(-1, 1, 1)
    j = torch.arange(k.shape[2], device=k.device)
    i = torch.arange(T, device=k.device).view(1, -1, 1)
    tree = c["op"] == "tree"
    p = n + _depths(S["parent"])[..., None] if tree else n - t + i
    see = (j < n) & (i < t) & _in_window(c, p - j, j)
    if not tree:
        see = see & ((j <= p) | (j < (S["prefix"].view(-1, 1, 1) if S["prefix"] is not None else 0)))
    q = S["q"].float().reshape(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    parts = []                                     # (scores, V) of the cache and of the drafts

    def scores(keys, dist, ok):
        x = torch.matmul(q, keys.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, T, G, -1)
        return _change(S, x, dist).masked_fill_(~ok[:, None, :, None, :], -math.inf)

    parts.append((scores(k, p - j, see), "v"))
    if tree:
        up = S["parent"].long()
        on = torch.zeros((B, T, T), dtype=torch.bool, device=k.device)
        at = torch.arange(T, device=k.device).expand(B, T)
        for _ in range(T):                         # a step towards the root for every token
            on |= torch.zeros_like(on).scatter_(2, at.clamp(min=0)[..., None], (at >= 0)[..., None])
            at = torch.where(at >= 0, up.gather(1, at.clamp(min=0)), at)
        pa = p.transpose(1, 2)                     # [B, 1, T]
        ok = on & (i < t) & _in_window(c, p - pa, pa)
        parts.append((scores(S["k"].float().transpose(1, 2), p - pa, ok),
                      S["v"].float().transpose(1, 2)))
    m = torch.stack([x.amax(-1, keepdim=True) for x, _ in parts]).amax(0)
    m = torch.where(m == -math.inf, 0.0, m)
    total, o = 0.0, 0.0
    for x, v in parts:
        w = x.sub_(m).exp_()
        total = total + w.sum(-1, keepdim=True)
        v = _dequantised(c, s, "v") if isinstance(v, str) else v
        o = o + torch.matmul(w.view(B, Hkv, T * G, -1), v).view(B, Hkv, T, G, D)
    lse = (total.log() + m).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, Hkv * G)
    real = (i < t).squeeze(-1)[..., None]
    lse = torch.where(real, lse, 0.0)
    o = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, D)
    return torch.where(real[..., None], o, 0.0).to(S["q"].dtype), lse


def run(S):
    c = S["c"]
    if own:
        import fp4_kv_cache_rope_gb300 as K
        if c["op"] == "rope":
            K.kv8_rope(S["cache"], S["q"], S["q_out"], S["rope"], S["ws"], k=S["k"], k_out=S["k_out"],
                       q_len=S["len"], pos=S["pos"],
                       parent=S["parent"] if c["where"] == "tree" else None)
            return S["q_out"], S["k_out"]
        if c["op"] == "rope_append":
            K.kv8_append_rope(S["cache"], S["k"], S["v"], S["rope"], S["ws"], q=S["q"],
                              q_out=S["q_out"], new_len=S["len"], start=S["start"], pos=S["pos"])
            return {"q": S["q_out"], **_stored(c, S["s"])}
        if c["op"] == "path":
            K.kv8_append_path(S["cache"], S["k"], S["v"], S["path"], S["ws"], new_len=S["m"],
                              start=S["start"])
            return _stored(c, S["s"])
        if c["op"] == "scored":
            K.kv8_attn_scored(S["cache"], S["q"], S["out"], S["ws"], S["scores"], lse=S["lse"],
                              q_len=S["len"])
        else:
            K.kv8_attn_tree(S["cache"], S["q"], S["k"], S["v"], S["parent"], S["out"], S["ws"],
                            lse=S["lse"], q_len=S["len"], scores=S["scores"])
        return S["out"], S["lse"]
    if c["op"] == "rope":
        return _plain_rope(S)
    if c["op"] == "rope_append":
        return _plain_rope_append(S)
    if c["op"] == "path":
        return _plain_path(S)
    return _plain_attn(S)


# -------------------------------------------------------- the same in 64 bits
def _value64(byte, fmt):
    byte = byte.long()
    if fmt == INT8:
        return torch.where(byte > 127, byte - 256, byte).double()
    e, m = (byte >> 3) & 15, (byte & 7).double()
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where(byte > 127, -mag, mag)


def _nearest64(y, fmt):
    """The format's value nearest to y, ties to the even one; |y| <= qmax."""
    if fmt == INT8:
        return torch.round(y)
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step


def _scale64(amax, fmt):
    """The smallest power of two >= 2^-126 that holds amax; 0 for 0."""
    e = torch.ceil(torch.log2((amax / QMAX[fmt]).clamp(min=2.0 ** -140))).clamp(min=-126.0)
    e = torch.where(amax > QMAX[fmt] * torch.exp2(e), e + 1, e)
    e = torch.where((amax <= QMAX[fmt] * torch.exp2(e - 1)) & (e > -126), e - 1, e)
    return torch.where(amax > 0, torch.exp2(e), torch.zeros_like(amax))


def _pages(s, b):
    return [b] if s["page_table"] is None else s["page_table"][b].tolist()


def _seq64(c, s, b, x):
    """Sequence b's rows [Hkv, rows, D] in 64 bits, and their blocks' scales [Hkv, blocks]."""
    pages = _pages(s, b)
    codes = torch.cat([s[x + "_codes"][p] for p in pages], 1)
    scales = torch.cat([s[x + "_scales"][p] for p in pages], 1).double()
    return _value64(codes, c["fmt"]) * scales.repeat_interleave(c["block"], 1)[..., None], scales


def _rotate64(S, c, x, b, t, pos):
    """Sequence b's first t rows of x in 64 bits, rotated at the positions pos."""
    y = x[b, :t].double().clone()
    R, f = c["R"], c["first"]
    for j in range(R // 2):
        u, v = (f + j, f + R // 2 + j) if c["style"] == HALVES else (f + 2 * j, f + 2 * j + 1)
        cs, sn = S["cos"][pos, j].double()[:, None], S["sin"][pos, j].double()[:, None]
        a, d = x[b, :t, :, u].double(), x[b, :t, :, v].double()
        y[..., u] = a * cs - d * sn
        y[..., v] = a * sn + d * cs
    return y


def _positions64(S, c, b, t, first):
    if S["pos"] is not None:
        return S["pos"][b, :t].tolist()
    if c["where"] == "tree":
        par = S["parent"][b].tolist()
        return [first + len(_path_to(par, i)) - 1 for i in range(t)]
    return [first + i for i in range(t)]


def _exact_append(S, c, rows):
    """rows(b) -> (k, v) [t, Hkv, D] in 64 bits that are appended to sequence b."""
    s, blk, fmt = S["s"], c["block"], c["fmt"]
    e = {x: _value64(s[x + "_codes"], fmt) for x in "kv"}
    e |= {x + "_scales": s[x + "_scales"].double() for x in "kv"}
    ps = s["k_codes"].shape[2]
    for b, first in enumerate(S["start"].tolist()):
        pages = _pages(s, b)
        for x, new in zip("kv", rows(b)):
            new = new.transpose(0, 1)              # [Hkv, t, D]
            t = new.shape[1]
            old, scales = _seq64(c, s, b, x)
            for p in range(first // blk * blk, first + t, blk):
                lo = max(p, first)
                fresh = new[:, lo - first: p + blk - first]
                low = scales[:, p // blk] if p < first else torch.zeros_like(scales[:, 0])
                sc = torch.maximum(low, _scale64(fresh.abs().amax((1, 2)), fmt))
                vals = torch.cat([old[:, p:lo], fresh], 1)
                codes = _nearest64(vals / torch.where(sc > 0, sc, 1.0)[:, None, None], fmt)
                at = p % ps
                e[x][pages[p // ps], :, at:at + vals.shape[1]] = codes
                e[x + "_scales"][pages[p // ps], :, at // blk] = sc
    if fmt == INT8:                                # whole numbers: held to the plain form's alone
        e["k"] = e["v"] = None
    e["seq_len"] = None
    return e


def _exact_attn(S, c):
    s, G, D, H = S["s"], c["G"], c["D"], c["Hkv"] * c["G"]
    n, t = _lengths(c)
    dev = S["q"].device
    out = torch.zeros(S["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(out.shape[:3], dtype=torch.float64, device=dev)
    for b in range(c["B"]):
        nb, tb = n[b], t[b]
        j = torch.arange(nb, device=dev)
        if c["op"] == "tree":
            par = S["parent"][b].tolist()
            paths = [_path_to(par, i) for i in range(tb)]
            p = torch.tensor([nb + len(x) - 1 for x in paths], device=dev)
            own_rows = torch.zeros((tb, tb), dtype=torch.bool, device=dev)
            for i, x in enumerate(paths):
                own_rows[i, x] = True
            see = torch.cat([torch.ones((tb, nb), dtype=torch.bool, device=dev), own_rows], 1)
            j = torch.cat([j, p])
        else:
            p = nb - tb + torch.arange(tb, device=dev)
            top = p + 1
            if S["prefix"] is not None:
                top = torch.maximum(top, S["prefix"][b].long())
            see = j < top[:, None]
        gap = p[:, None] - j
        if c["window"]:
            see = see & ((gap < c["window"]) | (j < c["sink"]))
        ks, vs = (_seq64(c, s, b, x)[0][:, :nb] for x in "kv")
        for h in range(H):
            k, v = ks[h // G], vs[h // G]
            if c["op"] == "tree":
                k = torch.cat([k, S["k"][b, :tb, h // G].double()])
                v = torch.cat([v, S["v"][b, :tb, h // G].double()])
            x = S["q"][b, :tb, h].double() @ k.T / math.sqrt(D)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if S["slopes"] is not None:
                x = x - S["slopes"][h].double() * gap.abs()
            x = x.masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, 1)
            lse[b, :tb, h] = z
            out[b, :tb, h] = torch.exp(x - torch.where(z == -math.inf, 0.0, z)[:, None]) @ v
    return out, lse


def exact(c, seed):
    global own
    was, own = own, False
    try:
        S = prepare(c, seed)
    finally:
        own = was
    n, t = _lengths(c)
    if c["op"] in ("scored", "tree"):
        if sum(x * y for x, y in zip(n, t)) * c["Hkv"] * c["G"] * c["D"] > 4e12:
            return None
        return _exact_attn(S, c)
    first = S["start"].tolist()
    if c["op"] == "path":
        m = S["m"].tolist()
        return _exact_append(S, c, lambda b: tuple(
            x[b][S["path"][b, :m[b]].long()].double() for x in (S["k"], S["v"])))
    where = [_positions64(S, c, b, t[b], first[b]) for b in range(c["B"])]

    def turned(x):
        y = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
        for b in range(c["B"]):
            y[b, :t[b]] = _rotate64(S, c, x, b, t[b], where[b])
        return y
    if c["op"] == "rope":
        return turned(S["q"]), turned(S["k"])
    if sum(t) / c["block"] > 4000:
        return None
    k = turned(S["k"])
    return {"q": turned(S["q"]),
            **_exact_append(S, c, lambda b: (k[b, :t[b]], S["v"][b, :t[b]].double()))}
