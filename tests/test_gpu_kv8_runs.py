"""GPU tests of the 8-bit K/V cache on work that gives every CTA several pieces:
the split kernels' walk over steps, units, heads and sequences, parts that begin
or end inside a unit, and the persistent kernel's rounds over its items.  Sizes
follow the SM count.  The reference is the formulas in fp64 on the GPU."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp4_kv_cache_rope_gb300 as K  # noqa: E402

SMS = torch.cuda.get_device_properties(0).multi_processor_count


def cache_of(B, Hkv, D, lens, block, page, fmt, seed):
    """A cache of random finite codes under power-of-two scales that vary from
    block to block, and its K and V as fp64 [B, Hkv, capacity, D].  V is mostly
    positive, so that what is left out of a sum cannot hide in one that cancels."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    cap = max(max(lens) + 9, 2049)                # above the capacity of one CTA a unit
    if page:
        per = -(-cap // page)
        table = torch.randperm(B * per + 3, generator=gen, device="cuda")[: B * per].view(B, per).int()
        pages, rows, cap = B * per + 3, page, per * page
    else:
        cap = -(-cap // block) * block
        table, pages, rows = None, B, cap
    c = K.Cache8(B, Hkv, D, cap, block=block, page_size=page, page_table=table,
                 num_pages=pages if page else 0, fmt=fmt, mass=True)
    vals = {}
    for s in "kv":
        x = torch.randn(c.k_codes.shape, generator=gen, device="cuda")
        if s == "v":
            x = x.abs() * torch.where(torch.rand(x.shape, generator=gen, device="cuda") < 0.9, 1, -1)
        kind = torch.int8 if fmt == K.KV8_INT8 else torch.float8_e4m3fn
        step = 24.0 if fmt == K.KV8_INT8 else 1.0
        code = (x * step).round().clamp(-127, 127) if fmt == K.KV8_INT8 else x.clamp(-448, 448)
        code = code.to(kind)
        scale = torch.exp2(torch.randint(-1, 2, getattr(c, s + "_scales").shape, generator=gen,
                                         device="cuda").float()) / (32.0 if fmt == K.KV8_INT8 else 1.0)
        getattr(c, s + "_codes").copy_(code.view(torch.uint8))
        getattr(c, s + "_scales").copy_(scale)
        v = code.double() * scale.double().repeat_interleave(block, 2)[..., None]
        at = c.page_table.long() if page else torch.arange(B, device="cuda").view(-1, 1)
        vals[s] = v[at].transpose(1, 2).reshape(B, Hkv, cap, D)
    c.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    return c, vals["k"], vals["v"], gen


def mass_at(c, b):
    """Weights of sequence b in position order, [Hkv, capacity]."""
    if c.page_table is None:
        return c.mass[b]
    return c.mass[c.page_table[b].long()].transpose(0, 1).reshape(c.kv_heads, -1)


def check_run(c, k, v, gen, lens, q_lens, T, G, dtype, chain, decay):
    """kv8_attn, then kv8_mass, against fp64.  chain: fp32 additions that follow
    one another in a sum over the rows, at most.

    A logit is D products summed in fp32 (2^-23 a step for an accumulator that
    cuts off, with the magnitudes' sum L) and its factor's rounding: ds =
    (D + 2) 2^-23 L.  A weight is off by 2 ds (its own logit and the maximum's),
    2^-20 (exp2) and 2^-11 (f16); a sum of them by 2 chain 2^-23 (weights and
    normaliser); a weight is held in steps of 2^-31 of the largest, and the output
    rounded by half a step.  An accumulated weight is off by ds, lse's roundings,
    exp2 and the additions of T G weights.
    """
    B, Hkv, D = c.batch, c.kv_heads, c.dim
    H = Hkv * G
    q = (0.9 * torch.randn((B, T, H, D), generator=gen, device="cuda")).to(dtype)
    out = torch.full_like(q, 7.0)
    lse = torch.full((B, T, H), 7.0, device="cuda")
    ql = torch.tensor(q_lens, dtype=torch.int32, device="cuda")
    ws = c.workspace(T, H)
    ws[256:] = 0xFF
    K.kv8_attn(c, q, out, ws, lse=lse, q_len=ql)
    again, lse2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    K.kv8_attn(c, q, again, ws, lse=lse2, q_len=ql)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    c.mass.fill_(0.25)
    K.kv8_mass(c, q, lse, ws, q_len=ql, decay=decay)
    first = c.mass.clone()
    for _ in range(3):
        c.mass.fill_(0.25)
        K.kv8_mass(c, q, lse, ws, q_len=ql, decay=decay)
        assert torch.equal(c.mass, first)
    assert K.get_status(ws) == 0
    half = 2.0 ** (-8 if dtype == torch.bfloat16 else -11)
    for b in range(B):
        n, t = lens[b], q_lens[b]
        assert (out[b, t:] == 7.0).all() and (lse[b, t:] == 7.0).all()
        m = mass_at(c, b)
        assert (m[:, n:] == 0.25).all()
        if t == 0 or n == 0:
            assert (out[b, :t] == 0).all() and (lse[b, :t] == -math.inf).all()
            assert (m[:, :n] == 0.25 * decay).all()
            continue
        qq = q[b, :t].double().view(t, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, t * G, D)
        kk, vv = k[b, :, :n], v[b, :, :n]
        x = qq @ kk.transpose(1, 2) / math.sqrt(D)
        tok = torch.arange(t * G, device="cuda") // G
        hid = torch.arange(n, device="cuda") > (n - t + tok)[:, None]
        x = x.masked_fill(hid, -math.inf)
        z = torch.logsumexp(x, -1)                           # [Hkv, t G]
        p = torch.where(hid, 0.0, torch.exp(x - torch.where(z == -math.inf, 0.0, z)[..., None]))
        o, a = p @ vv, p @ vv.abs()
        big = ((qq.abs() @ kk.abs().transpose(1, 2)).amax(-1) / math.sqrt(D))
        ds = (D + 2) * 2.0 ** -23 * big
        rel = 2 * ds + 2.0 ** -20 + 2.0 ** -11 + 2 * chain * 2.0 ** -23
        vmax = float(vv.abs().max())
        tol = a * rel[..., None] + (n * 2.0 ** -32 + 2.0 ** -30) * vmax
        tol = tol + half * (o.abs() + tol) + (2.0 ** -25 if half == 2.0 ** -11 else 1e-30)
        got = out[b, :t].double().view(t, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, t * G, D)
        assert ((got - o).abs() <= tol).all(), (b, float(((got - o).abs() / tol).max()))
        gl = lse[b, :t].double().view(t, Hkv, G).permute(1, 0, 2).reshape(Hkv, t * G)
        fin = torch.isfinite(z)
        assert torch.equal(fin, torch.isfinite(gl)) and (gl[~fin] == -math.inf).all()
        ltol = ds + 2.0 ** -20 + chain * 2.0 ** -23 + 2.0 ** -22 * z.abs()
        assert ((gl - z).abs()[fin] <= ltol[fin]).all()
        w = torch.where(hid | ~fin[..., None], 0.0,
                        torch.exp(x - torch.where(fin, gl, 0.0)[..., None])).sum(1)
        top = float(gl[fin].abs().max()) if fin.any() else 0.0
        wrel = (D + 4) * 2.0 ** -23 * float(big.max()) + 2.0 ** -22 * top + 2.0 ** -20 + (
            t * G + 2) * 2.0 ** -23
        want = 0.25 * decay + w
        err = (m[:, :n].double() - want).abs()
        assert (err <= w * wrel + 2 * 2.0 ** -23 * want + 1e-36).all(), (b, float(err.max()))


def ragged(B, total, seed):
    """B lengths that make `total` steps of 128 rows: none and one row (a step
    each), whole steps, a row over, and uneven ones."""
    gen = torch.Generator().manual_seed(seed)
    w = torch.rand(B - 2, generator=gen) ** 2 + 0.05
    steps = [1, 1] + [max(1, int(x)) for x in w / w.sum() * (total - B)]
    steps[-1] += max(0, total - sum(steps))
    lens = [128 * s - int(o) for s, o in zip(steps, torch.randint(0, 128, (B,), generator=gen))]
    lens[0], lens[1], lens[2], lens[3] = 0, 1, 128 * steps[2], 128 * steps[3] - 127
    return lens


# B, Hkv, G, T, D, block, page, dtype, format; the query rows make 1, 2 or 3 tiles of
# eight in one pass, or several passes
FEW = [
    (20, 8, 5, 1, 64, 64, 64, torch.bfloat16, K.KV8_E4M3),
    (40, 4, 1, 1, 128, 16, 48, torch.float16, K.KV8_INT8),
    (9, 8, 4, 4, 64, 16, 16, torch.float16, K.KV8_INT8),
    (35, 3, 8, 2, 128, 32, 32, torch.bfloat16, K.KV8_E4M3),
    (12, 4, 6, 4, 64, 128, 0, torch.float16, K.KV8_E4M3),
    (33, 2, 4, 5, 64, 16, 16, torch.bfloat16, K.KV8_INT8),
    (17, 2, 12, 2, 128, 64, 128, torch.bfloat16, K.KV8_INT8),
    (6, 4, 8, 5, 128, 64, 64, torch.float16, K.KV8_E4M3),
    (36, 2, 16, 4, 64, 32, 96, torch.bfloat16, K.KV8_E4M3),
]


@pytest.mark.parametrize("i", range(len(FEW)))
@pytest.mark.parametrize("many", [3, 5])
def test_several_steps_of_several_units_a_cta(i, many):
    B, Hkv, G, T, D, block, page, dtype, fmt = FEW[i]
    # four CTAs an SM at most: `many` times as many steps and some
    total = (4 * SMS * many + 11) // Hkv
    lens = ragged(B, total, 7 * i + many)
    q_lens = [T if b % 5 else min(T, b % 3) for b in range(B)]
    c, k, v, gen = cache_of(B, Hkv, D, lens, block, page, fmt, 100 + i)
    tiles = -(-T * G // 8)
    # a part has at most many * tiles + 2 steps, a quarter of whose rows a warp adds
    # up; then the warps' and the parts' results
    chain = 32 * (many * tiles * 2 + 2) + 4 + max(lens) // 128 + 2
    check_run(c, k, v, gen, lens, q_lens, T, G, dtype, chain, 0.5 if i % 2 else 0.0)


MANY = [
    (24, 4, 3, 23, 128, 64, 64, torch.bfloat16, K.KV8_E4M3),      # 69 rows
    (40, 2, 2, 50, 64, 16, 48, torch.float16, K.KV8_INT8),        # 100
    (9, 4, 4, 100, 128, 32, 32, torch.float16, K.KV8_INT8),       # 400: four tiles of 128
    (11, 3, 4, 150, 128, 128, 0, torch.bfloat16, K.KV8_E4M3),     # 600: three of 256
    (14, 4, 5, 160, 64, 64, 128, torch.bfloat16, K.KV8_E4M3),     # 800: four of 256
    (34, 2, 7, 75, 128, 16, 16, torch.float16, K.KV8_E4M3),       # 525
    (10, 8, 8, 64, 128, 64, 64, torch.bfloat16, K.KV8_INT8),      # 512
]


@pytest.mark.parametrize("i", range(len(MANY)))
def test_several_items_a_cta(i):
    B, Hkv, G, T, D, block, page, dtype, fmt = MANY[i]
    lens = ragged(B, (5 * SMS + 17) // Hkv + 1, 31 + i)
    q_lens = [min(T, [T, 0, T // 3, T - 1, 1, T // 2][b % 6]) for b in range(B)]
    q_lens[2] = T
    c, k, v, gen = cache_of(B, Hkv, D, lens, block, page, fmt, 200 + i)
    assert sum(max(1, -(-n // 128)) for n in lens) * Hkv >= 5 * SMS
    # the attention's rows are added up by one CTA, or by one of its parts
    check_run(c, k, v, gen, lens, q_lens, T, G, dtype, max(lens) + 16, 1.0 if i % 2 else 0.0)
