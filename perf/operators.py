"""The 8-bit K/V cache's operators: what they compute, on which sizes.

Four operators over one cache of grouped heads, held in 8 bits with one scale
for each block of tokens and head:

  append  quantise new K and V rows into the cache (a block's scale is the
          smallest power of two under which its largest value fits; a row that
          raises it re-expresses the rows already in the block);
  attn    softmax(scale * q k^T) v over the cache, causal at its end, with the
          log of the normaliser;
  mass    add to every cached row, per K/V head, the attention weight that it
          got from the given queries (from their log normalisers);
  evict   keep the first rows, the latest rows and, between them, the rows
          with the largest mass, in order, requantised into the blocks of a
          second cache.

`run` computes them in elementary torch operations in 32 bits, or, with `own`
set, through the package.  `exact` states them once more in 64 bits.
"""
import math

import torch

own = False

E4M3, INT8 = "e4m3", "int8"
QMAX = {E4M3: 448.0, INT8: 127.0}
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- the cases
def _case(name, op, B, T, N, Hkv, G, D, dtype, fmt, block, page, ragged, keep=0, sink=0, recent=0):
    return {"name": name, "op": op, "B": B, "T": T, "N": N, "Hkv": Hkv, "G": G, "D": D,
            "dtype": dtype, "fmt": fmt, "block": block, "page": page, "ragged": ragged,
            "keep": keep, "sink": sink, "recent": recent}


def listed():
    return [
        # one new token for each of 32 sequences that are being answered
        _case("append_token_b32", "append", 32, 1, 2048, 8, 8, 128, "bf16", E4M3, 64, 64, True),
        # the rows of four prompts of different lengths, padded to the longest
        _case("append_prompts_b4", "append", 4, 8192, 8192, 8, 8, 128, "bf16", E4M3, 64, 64, True),
        # one sequence, a short context, an odd group of heads: latency alone
        _case("attn_token_b1", "attn", 1, 1, 1000, 2, 7, 128, "bf16", E4M3, 64, 64, False),
        # a serving batch of different lengths
        _case("attn_token_b32", "attn", 32, 1, 32768, 8, 8, 128, "bf16", E4M3, 64, 64, True),
        # long contexts, contiguous, INT8
        _case("attn_token_long", "attn", 8, 1, 131072, 8, 4, 128, "bf16", INT8, 128, 0, False),
        # five proposed tokens verified at once, small pages
        _case("attn_verify_b16", "attn", 16, 5, 9001, 4, 4, 64, "f16", INT8, 16, 16, True),
        # a chunk of a long prompt over what is cached before it
        _case("attn_chunk_long", "attn", 1, 4096, 16384, 8, 8, 128, "bf16", E4M3, 64, 64, False),
        # whole prompts of odd lengths, padded to the longest
        _case("attn_prompts_b3", "attn", 3, 1501, 1501, 4, 4, 64, "f16", INT8, 32, 64, True),
        # the weights of one decode step, accumulated for a later eviction
        _case("mass_token_b32", "mass", 32, 1, 4096, 8, 8, 128, "bf16", E4M3, 64, 64, True),
        # the weights of a prompt's queries, its whole length
        _case("mass_prompt", "mass", 1, 4096, 4096, 8, 4, 128, "bf16", E4M3, 64, 64, False),
        # prompts cut to a budget before they are answered
        _case("evict_prompts_b4", "evict", 4, 0, 32768, 8, 8, 128, "bf16", E4M3, 64, 64, True,
              4096, 4, 512),
        # a full budget with a few rows over it, one sequence
        _case("evict_step_b1", "evict", 1, 0, 1100, 2, 8, 64, "bf16", INT8, 16, 16, False,
              1024, 4, 64),
    ]


def _cost(c):
    w = work(c)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.8e15


def draw(rng):
    logs = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["append", "attn", "attn", "attn", "mass", "evict"])
        many = rng.random() < 0.5
        B = logs(1, 32)
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8])
        D = rng.choice([64, 128, 128])
        block = rng.choice([16, 32, 64, 128])
        page = rng.choice([0, block, 2 * block, 128])
        N = logs(60, 131072)
        T = min(N, logs(32, 4096) if many else rng.choice([1, 1, 1, 2, 3, 5]))
        keep = sink = recent = 0
        if op == "evict":
            T = 0
            keep = max(8, int(N * rng.uniform(0.1, 0.95)))
            sink, recent = rng.randint(0, 4), rng.randint(0, keep // 2)
        dtype = rng.choice(["bf16", "f16"] + (["f32"] if op == "append" else []))
        c = _case("", op, B, T, N, Hkv, G, D, dtype, rng.choice([E4M3, E4M3, INT8]), block, page,
                  rng.random() < 0.6, keep, sink, recent)
        del c["name"]
        scores = B * Hkv * G * max(T, 1) * N  # the plain form holds them whole
        if _cost(c) <= most and scores <= 1.2e9 and B * Hkv * N * D <= 1.1e9:
            return c


def _lengths(c):
    """(rows held per sequence once the call is done, its new rows or queries)."""
    B, N, T = c["B"], c["N"], c["T"]
    if not c["ragged"]:
        return [N] * B, [T] * B
    n = [max(1, N - (b * N * 5) // (8 * B) - (13 * b) % 61) if b else N for b in range(B)]
    t = [min(x, T if T <= 8 else max(1, T - (b * T * 3) // (4 * B))) for b, x in enumerate(n)]
    return n, t


def work(c):
    B, Hkv, G, D = c["B"], c["Hkv"], c["G"], c["D"]
    n, t = _lengths(c)
    es = 4 if c["dtype"] == "f32" else 2
    rows, new = sum(n), sum(t)
    blocks = sum(-(-x // c["block"]) for x in n)
    if c["op"] == "append":
        touched = sum(-(-x // c["block"]) for x in t)
        return {"bytes": 2 * Hkv * (new * D * (es + 1) + touched * 4) + 8 * B,
                "flops": 4 * Hkv * new * D}
    pairs = sum(y * x - y * (y - 1) // 2 for x, y in zip(n, t)) * Hkv * G
    queries = new * Hkv * G
    if c["op"] == "attn":
        return {"bytes": 2 * Hkv * (rows * D + blocks * 4) + queries * (2 * D * es + 4),
                "flops": 4 * D * pairs}
    if c["op"] == "mass":
        return {"bytes": Hkv * (rows * (D + 4) + blocks * 4) + queries * (D * es + 4),
                "flops": 2 * D * pairs}
    kept = sum(min(x, c["keep"]) for x in n)
    return {"bytes": Hkv * (rows * 4 + kept * (4 * D + 12)), "flops": 2 * Hkv * kept * D}


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
    s["mass"] = torch.zeros((pages, Hkv, ps), device=dev)
    s["seq_len"] = torch.zeros(B, dtype=torch.int32, device=dev)
    return s


def _table(c, s):
    if s["page_table"] is not None:
        return s["page_table"].long()
    return torch.arange(c["B"], device=s["seq_len"].device).view(-1, 1)


def _rows(c, gen, dev, B, Hkv, N, D):
    """K and V rows as projections give them: channels of uneven size, a few of
    them large, and tokens whose size varies."""
    ch = torch.exp(0.6 * torch.randn((Hkv, 1, D), generator=gen, device=dev))
    tok = torch.exp(0.3 * torch.randn((B, Hkv, N, 1), generator=gen, device=dev))
    return torch.randn((B, Hkv, N, D), generator=gen, device=dev) * ch * tok, ch


def _handle(c, s):
    import fp4_kv_cache_rope_gb300 as K
    fmt = K.KV8_E4M3 if c["fmt"] == E4M3 else K.KV8_INT8
    return K.Cache8(c["B"], c["Hkv"], c["D"], s["max_len"], block=c["block"],
                    page_size=c["page"], page_table=s["page_table"],
                    num_pages=s["k_codes"].shape[0] if c["page"] else 0, fmt=fmt,
                    tensors={k: s[k] for k in ("k_codes", "v_codes", "k_scales", "v_scales",
                                               "mass", "seq_len")})


def prepare(c, seed):
    dev = torch.device("cuda", 0) if torch.cuda.is_available() else torch.device("cpu")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    B, T, N, Hkv, G, D = c["B"], c["T"], c["N"], c["Hkv"], c["G"], c["D"]
    H = Hkv * G
    dt = DTYPES[c["dtype"]]
    n, t = _lengths(c)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    S = {"c": c, "s": _store(c, N, dev, gen)}
    s = S["s"]
    # what the cache holds before the call: everything (attn, mass, evict) or
    # the rows in front of the new ones (append)
    held = [x - y for x, y in zip(n, t)] if c["op"] == "append" else n
    hmax = max(held)
    qdir = None
    if hmax:
        blk = c["block"]
        cap = s["max_len"]
        for b in range(B):
            for x in "kv":
                rows, ch = _rows(c, gen, dev, 1, Hkv, hmax, D)
                if x == "k" and b == 0:
                    qdir = 1.0 / ch
                rows = torch.nn.functional.pad(rows[0, :, :held[b]], (0, 0, 0, cap - held[b]))
                r = rows.view(Hkv, cap // blk, blk, D)
                sc = _pow2_scale(r.abs().amax((2, 3)), c["fmt"])
                codes = _encode(r, sc[..., None, None], c["fmt"]).view(Hkv, cap, D)
                tab = _table(c, s)[b]
                ps = cap // len(tab)
                s[x + "_codes"][tab] = codes.view(Hkv, len(tab), ps, D).transpose(0, 1)
                s[x + "_scales"][tab] = sc.view(Hkv, len(tab), ps // blk).transpose(0, 1)
        s["seq_len"].copy_(ints(held))
    S["new_len"] = ints(t) if c["ragged"] and T > 1 else None
    if c["op"] == "append":
        # the K and V parts of a fused projection's output
        both, _ = _rows(c, gen, dev, B, 2 * Hkv, T, D)
        fused = torch.zeros((B, T, H + 2 * Hkv, D), dtype=dt, device=dev)
        fused[:, :, H:] = both.transpose(1, 2).to(dt)
        S["fused"], S["k"], S["v"] = fused, fused[:, :, H:H + Hkv], fused[:, :, H + Hkv:]
        S["start"] = ints(held)
    elif c["op"] in ("attn", "mass"):
        q = torch.randn((B, T, Hkv, G, D), generator=gen, device=dev) * qdir.view(Hkv, 1, D) * 1.5
        S["q"] = q.view(B, T, H, D).to(dt)
        S["out"] = torch.zeros((B, T, H, D), dtype=dt, device=dev)
        S["lse"] = torch.zeros((B, T, H), device=dev)
        if c["op"] == "mass":
            S["lse"] = _plain_attn(S, only_lse=True)
    else:
        w = torch.exp(2.0 * torch.randn(s["mass"].shape, generator=gen, device=dev))
        s["mass"].copy_(torch.where(w < 0.2, 0.0, w))   # many rows never got any weight
        S["dst"] = _store(c, c["keep"], dev, gen)
        S["kept"] = torch.full((B, Hkv, c["keep"]), -1, dtype=torch.int32, device=dev)
    if own:
        S["cache"] = _handle(c, s)
        S["ws"] = S["cache"].workspace(max(T, 1), H)
        if c["op"] == "evict":
            S["dst_cache"] = _handle(c, S["dst"])
    return S


# ------------------------------------------------------------- the plain forms
def _gather(c, s, what):
    """[B, Hkv, rows, ...] of a paged array [pages, Hkv, page rows, ...]."""
    x = s[what][_table(c, s)].transpose(1, 2)
    return x.reshape(x.shape[0], x.shape[1], -1, *x.shape[4:])


def _dequantised(c, s, x):
    scale = _gather(c, s, x + "_scales").repeat_interleave(c["block"], 2)
    return _values(_gather(c, s, x + "_codes"), c["fmt"]) * scale[..., None]


def _visible(c, n, t, T, cap, dev):
    """[B, T, cap]: whether query i of a sequence's t sees row j of its n."""
    j = torch.arange(cap, device=dev)
    i = torch.arange(T, device=dev).view(1, -1, 1)
    n, t = n.view(-1, 1, 1), t.view(-1, 1, 1)
    return (j <= n - t + i) & (i < t) & (j < n)


def _scores(S):
    """Masked logits [B, Hkv, T, G, rows] and who sees whom."""
    c, s = S["c"], S["s"]
    B, T, Hkv, G, D = c["B"], c["T"], c["Hkv"], c["G"], c["D"]
    k = _dequantised(c, s, "k")
    n = s["seq_len"].long()
    t = S["new_len"].long() if S["new_len"] is not None else torch.full_like(n, T)
    see = _visible(c, n, t, T, k.shape[2], k.device)
    q = S["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, T, G, -1)
    return x.masked_fill_(~see[:, None, :, None, :], -math.inf), see, n, t


def _plain_attn(S, only_lse=False):
    c = S["c"]
    B, T, Hkv, G, D = c["B"], c["T"], c["Hkv"], c["G"], c["D"]
    x, see, n, t = _scores(S)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + m).squeeze(-1).permute(0, 2, 1, 3).reshape(B, T, Hkv * G)
    real = (torch.arange(T, device=x.device) < t.view(-1, 1))[..., None]
    lse = torch.where(real, lse, 0.0)
    if only_lse:
        return lse
    v = _dequantised(c, S["s"], "v")
    o = torch.matmul(p.view(B, Hkv, T * G, -1), v).view(B, Hkv, T, G, D)
    o = torch.where(total > 0, o / torch.where(total > 0, total, 1.0), 0.0)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, D)
    return torch.where(real[..., None], o, 0.0).to(S["q"].dtype), lse


def _plain_mass(S):
    c, s = S["c"], S["s"]
    B, T, Hkv, G = c["B"], c["T"], c["Hkv"], c["G"]
    x, see, n, t = _scores(S)
    lse = S["lse"].view(B, T, Hkv, G).permute(0, 2, 1, 3)[..., None]
    w = torch.where(x == -math.inf, 0.0, (x - lse).exp()).sum((2, 3))
    tab = _table(c, s)
    ps = w.shape[2] // tab.shape[1]
    held = torch.arange(w.shape[2], device=w.device) < n.view(-1, 1)
    old = _gather(c, s, "mass")
    w = torch.where(held[:, None], w, old)
    s["mass"][tab] = w.view(B, Hkv, -1, ps).transpose(1, 2)
    return s["mass"]


def _scatter_rows(c, s, what, b, h, p, ok, x):
    """s[what] at positions p of (b, h), where ok."""
    tab = _table(c, s)
    ps = s[what].shape[2]
    p = torch.where(ok, p, 0)
    page = tab.expand(c["B"], -1)[b, p // ps]
    at = (page * c["Hkv"] + h) * ps + p % ps
    flat = s[what].view(-1, *s[what].shape[3:])
    flat[at[ok]] = x[ok]


def _plain_append(S):
    c, s = S["c"], S["s"]
    B, T, Hkv, D, blk = c["B"], c["T"], c["Hkv"], c["D"], c["block"]
    dev = s["seq_len"].device
    start = S["start"].long()
    t = S["new_len"].long() if S["new_len"] is not None else torch.full_like(start, T)
    nb = (T + blk - 2) // blk + 1                  # blocks that T rows can touch
    p = (start // blk * blk).view(-1, 1) + torch.arange(nb * blk, device=dev)
    old = p < start.view(-1, 1)
    i = p - start.view(-1, 1)
    new = (i >= 0) & (i < t.view(-1, 1))
    cap = s["max_len"]
    bh = torch.arange(B, device=dev).view(-1, 1, 1), torch.arange(Hkv, device=dev).view(1, -1, 1)
    sees = lambda m: m.view(B, 1, nb, blk).expand(B, Hkv, nb, blk)  # noqa: E731
    pb, touched = p.view(B, 1, nb, blk)[..., 0].expand(B, Hkv, nb), sees(new).any(-1)
    for x, src in (("k", S["k"]), ("v", S["v"])):
        rows = src.float().transpose(1, 2)         # [B, Hkv, T, D]
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
        flat = s[x + "_scales"]
        tab, ps = _table(c, s), s[x + "_codes"].shape[2]
        page = tab[bh[0], torch.where(touched, pb, 0) // ps]
        flat[page[touched], bh[1].expand(B, Hkv, nb)[touched],
             (pb % ps // blk)[touched]] = s1[touched]
    s["seq_len"].copy_((start + t).int())
    return _stored(c, s)


def _stored(c, s):
    """What the cache holds, as the values that the codes stand for."""
    kind = torch.float8_e4m3fn if c["fmt"] == E4M3 else torch.int8
    return {"k": s["k_codes"].view(kind), "v": s["v_codes"].view(kind),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"], "seq_len": s["seq_len"]}


def _plain_evict(S):
    c, s, d = S["c"], S["s"], S["dst"]
    B, Hkv, D, blk, keep = c["B"], c["Hkv"], c["D"], c["block"], c["keep"]
    mass = _gather(c, s, "mass")
    n = s["seq_len"].long().view(-1, 1, 1)
    j = torch.arange(mass.shape[2], device=mass.device)
    over = n > keep
    always = (j < c["sink"]) | (j >= n - c["recent"]) | ~over
    rank = torch.where(always, math.inf, mass)
    rank = torch.where(j < n, rank, -1.0)          # weights are never negative
    order = rank.sort(dim=2, descending=True, stable=True)[1][..., :keep]
    m = torch.minimum(n, torch.full_like(n, keep)).expand(B, Hkv, 1)
    order = torch.nn.functional.pad(order, (0, keep - order.shape[2]), value=0)
    place = torch.arange(keep, device=mass.device)
    order = torch.where(place < m, order, 1 << 40).sort(2)[0]
    ok = place < m
    S["kept"].copy_(torch.where(ok, order, -1).int())
    nb = -(-keep // blk)
    pad = nb * blk - keep
    src = torch.nn.functional.pad(torch.where(ok, order, 0), (0, pad))
    okp = torch.nn.functional.pad(ok, (0, pad))
    at = torch.arange(nb * blk, device=mass.device).expand(B, Hkv, -1)
    same = ((src == at) | ~okp).view(B, Hkv, nb, blk).all(-1)
    b3 = torch.arange(B, device=mass.device).view(-1, 1, 1).expand(B, Hkv, nb * blk)
    h3 = torch.arange(Hkv, device=mass.device).view(1, -1, 1).expand(B, Hkv, nb * blk)
    whole = okp.view(B, Hkv, nb, blk)[..., 0]      # blocks that hold a row
    for x in "kv":
        codes0 = _gather(c, s, x + "_codes").gather(2, src[..., None].expand(-1, -1, -1, D))
        sc = _gather(c, s, x + "_scales").gather(2, src // blk)
        rows = torch.where(okp[..., None], _values(codes0, c["fmt"]) * sc[..., None], 0.0)
        rows = rows.view(B, Hkv, nb, blk, D)
        s1 = _pow2_scale(rows.abs().amax((3, 4)), c["fmt"])
        s1 = torch.where(same, sc.view(B, Hkv, nb, blk)[..., 0], s1)
        codes = _encode(rows, s1[..., None, None], c["fmt"]).view(B, Hkv, nb * blk, D)
        codes = torch.where(same.repeat_interleave(blk, 2)[..., None], codes0, codes)
        _scatter_rows(c, d, x + "_codes", b3, h3, at, okp, codes)
        ps = d[x + "_codes"].shape[2]
        pb = at.view(B, Hkv, nb, blk)[..., 0]
        page = _table(c, d)[b3[..., :nb], pb // ps]
        d[x + "_scales"][page[whole], h3[..., :nb][whole], (pb % ps // blk)[whole]] = s1[whole]
    _scatter_rows(c, d, "mass", b3, h3, at, okp, mass.gather(2, src))
    d["seq_len"].copy_(m[:, 0, 0].int())
    return {"kept": S["kept"], "mass": d["mass"], **_stored(c, d)}


def run(S):
    c = S["c"]
    if own:
        import fp4_kv_cache_rope_gb300 as K
        if c["op"] == "append":
            K.kv8_append(S["cache"], S["k"], S["v"], S["ws"], new_len=S["new_len"],
                         start=S["start"])
            return _stored(c, S["s"])
        if c["op"] == "attn":
            K.kv8_attn(S["cache"], S["q"], S["out"], S["ws"], lse=S["lse"], q_len=S["new_len"])
            return S["out"], S["lse"]
        if c["op"] == "mass":
            # (the plain form's log normalisers may come transposed)
            K.kv8_mass(S["cache"], S["q"], S["lse"].contiguous(), S["ws"], q_len=S["new_len"],
                       decay=0.0)
            return S["s"]["mass"]
        K.kv8_evict(S["cache"], c["keep"], c["sink"], c["recent"], S["kept"], S["ws"],
                    dst=S["dst_cache"])
        return {"kept": S["kept"], "mass": S["dst"]["mass"], **_stored(c, S["dst"])}
    if c["op"] == "append":
        return _plain_append(S)
    if c["op"] == "attn":
        return _plain_attn(S)
    if c["op"] == "mass":
        return _plain_mass(S)
    return _plain_evict(S)


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


def _block64(rows, low, fmt):
    """(values over the scale, scale) of a block's rows, its scale at least low."""
    amax = float(rows.abs().max()) if rows.numel() else 0.0
    s = 0.0
    if amax > 0:
        s = 2.0 ** max(-126, math.ceil(math.log2(amax / QMAX[fmt])))
        while amax > QMAX[fmt] * s:
            s *= 2
        while s > 2.0 ** -126 and amax <= QMAX[fmt] * s / 2:
            s /= 2
    s = max(s, low)
    return (_nearest64(rows / s, fmt) if s > 0 else torch.zeros_like(rows)), s


def _seq64(c, s, b, h, x):
    """Sequence b's rows of head h in 64 bits, and their blocks' scales."""
    pages = [b] if s["page_table"] is None else s["page_table"][b].tolist()
    codes = torch.cat([s[x + "_codes"][p, h] for p in pages])
    scales = torch.cat([s[x + "_scales"][p, h] for p in pages]).double()
    return _value64(codes, c["fmt"]) * scales.repeat_interleave(c["block"])[:, None], scales


def _exact_attn(S, c):
    s, G, D, T = S["s"], c["G"], c["D"], c["T"]
    n, t = _lengths(c)
    out = torch.zeros(S["q"].shape, dtype=torch.float64, device=S["q"].device)
    lse = torch.zeros(out.shape[:3], dtype=torch.float64, device=out.device)
    mass = s["mass"].double()
    for b in range(c["B"]):
        j = torch.arange(n[b], device=out.device)
        i = torch.arange(t[b], device=out.device)
        hidden = j > (n[b] - t[b] + i)[:, None]
        pages = [b] if s["page_table"] is None else s["page_table"][b].tolist()
        for h in range(c["Hkv"]):
            k = _seq64(c, s, b, h, "k")[0][: n[b]]
            v = _seq64(c, s, b, h, "v")[0][: n[b]] if c["op"] == "attn" else None
            got = torch.zeros(n[b], dtype=torch.float64, device=out.device)
            for g in range(G):
                x = S["q"][b, : t[b], h * G + g].double() @ k.T / math.sqrt(D)
                x = x.masked_fill(hidden, -math.inf)
                if c["op"] == "mass":
                    got += torch.exp(x - S["lse"][b, : t[b], h * G + g].double()[:, None]).sum(0)
                    continue
                z = torch.logsumexp(x, 1)
                lse[b, : t[b], h * G + g] = z
                out[b, : t[b], h * G + g] = torch.exp(x - z[:, None]) @ v
            if c["op"] == "mass":
                ps = mass.shape[2]
                for a, p in enumerate(pages):
                    part = got[a * ps:(a + 1) * ps]
                    mass[p, h, : len(part)] = part
    return mass if c["op"] == "mass" else (out, lse)


def _exact_stored(c, d):
    """Storage of the case's shape for values in 64 bits."""
    e = {x: _value64(d[x + "_codes"], c["fmt"]) for x in "kv"}
    return e | {x + "_scales": d[x + "_scales"].double() for x in "kv"}


def _exact_rows(c, S):
    """append and evict: block by block."""
    s, blk, fmt = S["s"], c["block"], c["fmt"]
    d = s if c["op"] == "append" else S["dst"]
    e = _exact_stored(c, d)
    mass = d["mass"].double()
    n, t = _lengths(c)
    ps = d["k_codes"].shape[2]
    for b in range(c["B"]):
        tab = [b] if d["page_table"] is None else d["page_table"][b].tolist()
        for h in range(c["Hkv"]):
            if c["op"] == "evict":
                stab = [b] if s["page_table"] is None else s["page_table"][b].tolist()
                w = torch.cat([s["mass"][p, h] for p in stab])[: n[b]].double()
                key = w.clone()
                if n[b] > c["keep"]:
                    key[: c["sink"]] = math.inf
                    key[n[b] - c["recent"]:] = math.inf
                take = torch.argsort(key, descending=True, stable=True)[: c["keep"]].sort()[0]
            for x in "kv":
                vals, scales = _seq64(c, s, b, h, x)
                if c["op"] == "append":
                    first = n[b] - t[b]
                    vals = torch.cat([vals[:first], S[x][b, : t[b], h].double()])
                    begin = first // blk * blk
                else:
                    vals, first, begin = vals[take], len(take), 0
                for p in range(begin, len(vals), blk):
                    rows = vals[p:p + blk]
                    low = float(scales[p // blk]) if c["op"] == "append" and p < first else 0.0
                    if c["op"] == "append":
                        new = rows[max(0, first - p):]
                        codes, sc = _block64(rows, max(low, _block64(new, low, fmt)[1]), fmt)
                    else:
                        codes, sc = _block64(rows, 0.0, fmt)
                        own_rows = torch.arange(p, p + len(rows), device=take.device)
                        if torch.equal(take[p:p + blk], own_rows):
                            sc = float(scales[p // blk])
                            codes = rows / sc if sc else rows
                    at = p % ps
                    e[x][tab[p // ps], h, at:at + len(rows)] = codes
                    e[x + "_scales"][tab[p // ps], h, at // blk] = sc
            if c["op"] == "evict":
                for p in range(0, len(take), ps):
                    part = w[take[p:p + ps]]
                    mass[tab[p // ps], h, : len(part)] = part
    if fmt == INT8:                        # whole numbers: held to the plain form's alone
        e["k"] = e["v"] = None
    e["seq_len"] = None
    return e | {"kept": None, "mass": mass} if c["op"] == "evict" else e


def exact(c, seed):
    global own
    was, own = own, False
    try:
        S = prepare(c, seed)
    finally:
        own = was
    if c["op"] in ("attn", "mass"):
        n, t = _lengths(c)
        if sum(x * y for x, y in zip(n, t)) * c["Hkv"] * c["G"] * c["D"] > 4e12:
            return None
        return _exact_attn(S, c)
    n, t = _lengths(c)
    blocks = sum((x if c["op"] == "append" else min(y, c["keep"])) for x, y in zip(t, n))
    if 2 * c["Hkv"] * blocks / c["block"] > 20000:
        return None
    return _exact_rows(c, S)
