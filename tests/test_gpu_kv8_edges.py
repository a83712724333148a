"""GPU tests of the 8-bit K/V cache where a row or a query that must not count
holds what would spoil the others: zero rows moved between blocks whose scales
lie far apart, NaN and infinities in queries without weight."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp4_kv_cache_rope_gb300 as K  # noqa: E402
from oracle import kv8 as O  # noqa: E402
from kv8_tools import Pair, attention_bounds  # noqa: E402


@pytest.mark.parametrize("into", ["place", "cache"])
@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
@pytest.mark.parametrize("block,page,D", [(16, 16, 64), (64, 0, 128), (128, 128, 64)])
def test_evict_keeps_zero_rows_zero_beside_rows_far_smaller(block, page, D, fmt, into):
    """Zero rows come out of a block with a large scale into one whose other rows
    are 2^-20 to 2^-200 as large."""
    for big, small in ((2.0 ** 5, 2.0 ** -15), (2.0 ** 9, 2.0 ** -22), (2.0 ** 9, 2.0 ** -24),
                       (2.0 ** 20, 2.0 ** -25), (2.0 ** 100, 2.0 ** -100)):
        n, keep = 2 * block, block
        p = Pair(1, 2, D, n, block, page, fmt, seed=91)
        ws = p.c.workspace(1, 2)
        k, v = (p.rows(n, 2, "f32") for _ in "kv")
        for x, at in ((k, 0), (v, 1)):
            x[:, :block] = 0
            x[:, at] = big                      # the one row of the first block that is not 0
            x[:, block:] *= small
        p.append(k, v, ws)
        w = np.ones(n)
        w[: 2] = 0.0                            # it goes, zero rows and small ones stay
        w[2 + block // 2: block] = 0.0
        w[n - 2:] = 0.0
        p.set_mass([[w] * 2])
        kept = torch.empty(1, 2, keep, dtype=torch.int32, device="cuda")
        rows = O.evict(w, n, keep, 0, 0)
        d = p
        if into == "cache":
            d = Pair(1, 2, D, keep, block, page, fmt, seed=92)
        K.kv8_evict(p.c, keep, 0, 0, kept, ws, dst=None if d is p else d.c)
        for h in range(2):
            assert kept[0, h].tolist() == rows.tolist()
            for s in "kv":
                d.seq[0, h, s] = p.seq[0, h, s].keep(rows)
        d.len = [keep]
        d.check()
        assert K.get_status(ws) == 0


def test_evict_between_neighbours_in_one_allocation():
    """Two contiguous caches whose arrays lie end to end share nothing."""
    B, Hkv, D, n, keep, block = 2, 2, 64, 128, 48, 16
    p = Pair(B, Hkv, D, n, block, 0, O.E4M3, seed=96)
    d = Pair(B, Hkv, D, n, block, 0, O.E4M3, seed=97)
    both = {}
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "mass", "seq_len"):
        both[name] = torch.cat([getattr(p.c, name), getattr(d.c, name)])
    for i, x in ((0, p), (1, d)):
        x.c = K.Cache8(B, Hkv, D, n, block=block, fmt=O.E4M3,
                       tensors={k: t[i * B:(i + 1) * B] for k, t in both.items()})
    ws = p.c.workspace(1, Hkv)
    p.append(p.rows(100, Hkv, "f32"), p.rows(100, Hkv, "f32"), ws)
    w = p.rng.random((B, Hkv, 100)).astype(np.float32)
    p.set_mass(w)
    kept = torch.empty(B, Hkv, keep, dtype=torch.int32, device="cuda")
    K.kv8_evict(p.c, keep, 2, 9, kept, ws, dst=d.c)
    for b in range(B):
        for h in range(Hkv):
            rows = O.evict(w[b, h], 100, keep, 2, 9)
            for s in "kv":
                d.seq[b, h, s] = p.seq[b, h, s].keep(rows)
    d.len = [keep] * B
    p.check()
    d.check()
    with pytest.raises(K.Csa2Error):
        K.kv8_evict(p.c, keep, 2, 9, kept, ws, dst=p.c)
    p.check()


def _weights(p, q, lse, ws, q_len=None):
    p.c.mass.fill_(3.0)
    K.kv8_mass(p.c, q, lse, ws, q_len=q_len, decay=0.0)
    assert K.get_status(ws) == 0
    return p.c.mass.clone()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,G,D,cap", [(3, 2, 64, 0), (5, 5, 128, 0), (12, 4, 64, 80000), (50, 2, 64, 0),
                                       (90, 3, 128, 0), (310, 2, 128, 0)])
def test_a_query_without_weight_adds_nothing_whatever_it_holds(T, G, D, cap, dtype):
    """lse -inf or +inf: the query adds nothing, be it NaN, infinite or a number."""
    B, Hkv = 2, 2
    lens = [700, 333]
    p = Pair(B, Hkv, D, max(cap, 720), 16, 0 if cap else 16, O.E4M3, seed=93)
    ws = p.c.workspace(T, Hkv * G)
    p.append(p.rows(700, Hkv, "bf16"), p.rows(700, Hkv, "bf16"), ws, lens=lens)
    q = p.rows(T, Hkv * G, dtype, 0.7).cuda()
    out, lse = torch.empty_like(q), torch.empty(B, T, Hkv * G, device="cuda")
    K.kv8_attn(p.c, q, out, ws, lse=lse)
    gone = torch.from_numpy(p.rng.random((B, T, Hkv * G)) < 0.3).cuda()
    gone[0, 0, 0], gone[1, T - 1, 1], gone[1, 0] = True, True, True
    sign = torch.from_numpy(p.rng.random((B, T, Hkv * G)) < 0.5).cuda()
    lse = torch.where(gone, torch.where(sign, math.inf, -math.inf), lse)
    want = _weights(p, q, lse, ws)
    held = torch.zeros_like(want, dtype=torch.bool)
    for b in range(B):
        pages = [b] if p.table is None else p.table[b].tolist()
        left = lens[b]
        for g in pages:
            held[g, :, :max(0, left)] = True
            left -= held.shape[2]
    assert torch.isfinite(want).all() and (want[held] >= 0).all()
    for bad in (math.nan, math.inf, -math.inf):
        spoiled = q.clone()
        spoiled[gone] = bad
        assert torch.equal(_weights(p, spoiled, lse, ws), want), bad
        one = q.clone()
        one[..., 7][gone] = bad
        assert torch.equal(_weights(p, one, lse, ws), want), bad


@pytest.mark.parametrize("T,G,D", [(9, 2, 64), (30, 1, 128), (40, 3, 64), (80, 8, 128)])
def test_queries_in_front_of_the_first_row_add_nothing_whatever_they_hold(T, G, D):
    """More queries than rows: the first ones see none."""
    Hkv, n = 2, T - 4
    p = Pair(1, Hkv, D, 720, 16, 16, O.INT8, seed=94)
    ws = p.c.workspace(T, Hkv * G)
    p.append(p.rows(n, Hkv, "bf16"), p.rows(n, Hkv, "bf16"), ws)
    q = p.rows(T, Hkv * G, "f16", 0.7).cuda()
    out, lse = torch.empty_like(q), torch.empty(1, T, Hkv * G, device="cuda")
    K.kv8_attn(p.c, q, out, ws, lse=lse)
    want = _weights(p, q, lse, ws)
    assert torch.isfinite(want).all()
    q[:, :4] = math.nan
    again = torch.empty_like(lse)
    K.kv8_attn(p.c, q, out, ws, lse=again)
    assert torch.equal(again, lse) and (out[:, :4] == 0).all()
    assert torch.equal(_weights(p, q, again, ws), want)
    again[:, :4] = math.nan                     # nor does their lse count
    assert torch.equal(_weights(p, q, again, ws), want)


@pytest.mark.parametrize("T,G,D", [(5, 3, 64), (8, 1, 128), (6, 5, 128), (60, 3, 64), (90, 8, 128)])
def test_a_nan_query_spoils_only_the_weights_of_rows_that_it_sees(T, G, D):
    Hkv, n = 2, 500
    p = Pair(1, Hkv, D, 720, 32, 32, O.E4M3, seed=95)
    ws = p.c.workspace(T, Hkv * G)
    p.append(p.rows(n, Hkv, "bf16"), p.rows(n, Hkv, "bf16"), ws)
    q = p.rows(T, Hkv * G, "bf16", 0.7).cuda()
    out, lse = torch.empty_like(q), torch.empty(1, T, Hkv * G, device="cuda")
    K.kv8_attn(p.c, q, out, ws, lse=lse)
    _weights(p, q, lse, ws)
    want = [p.at("mass", 0, h)[:n] for h in range(Hkv)]
    q[0, 1, 0, 3] = math.nan                    # token 1, head 0: of the first K/V head
    K.kv8_attn(p.c, q, out, ws, lse=lse)
    assert torch.isnan(lse[0, 1, 0]) and lse.isnan().sum() == 1
    _weights(p, q, lse, ws)
    got = [p.at("mass", 0, h)[:n] for h in range(Hkv)]
    sees = n - T + 2
    assert np.isnan(got[0][:sees]).all()
    assert np.array_equal(got[0][sees:], want[0][sees:])
    assert np.array_equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 5, 70])
def test_attention_takes_every_output_without_overlap(T):
    B, Hkv, G, D = 2, 2, 4, 64
    H = Hkv * G
    p = Pair(B, Hkv, D, 400, 16, 16, O.E4M3, seed=98)
    ws = p.c.workspace(T, H)
    p.append(p.rows(300, Hkv, "bf16"), p.rows(300, Hkv, "bf16"), ws)
    q = p.rows(T, H, "bf16").cuda()
    want = torch.empty_like(q)
    K.kv8_attn(p.c, q, want, ws)
    def full(*s): return torch.full(s, 7.0, dtype=q.dtype, device="cuda")  # noqa: E704
    fused = full(B, T, 3 * H, D)
    for out in (full(T, H, B, D).permute(2, 0, 1, 3), full(H, B, T, D).permute(1, 2, 0, 3),
                full(B, H, T, D).transpose(1, 2), fused[:, :, H:2 * H], full(B, T, H, D + 8)[..., :D],
                full(B, 2 * T, H, D)[:, ::2], full(B, T, 2 * H, D)[:, :, 1::2]):
        K.kv8_attn(p.c, q, out, ws)
        assert torch.equal(out, want)
    assert (fused[:, :, :H] == 7.0).all() and (fused[:, :, 2 * H:] == 7.0).all()
    one = q[:1, :1, :1].expand(B, T, H, D)          # a query that repeats
    K.kv8_attn(p.c, one, want, ws)
    assert torch.isfinite(want).all()
    for shape in ((1, T, H, D), (B, T, 1, D)) + (((B, 1, H, D),) if T > 1 else ()):
        with pytest.raises(K.Csa2Error):
            K.kv8_attn(p.c, q, full(*shape).expand(B, T, H, D), ws)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("T,G,D", [(3, 2, 128), (9, 3, 64), (60, 4, 128), (60, 4, 64), (150, 4, 128)])
def test_weights_of_logits_whose_products_share_a_sign(T, G, D, sign, dtype):
    """Sums that grow steadily lose more to an accumulator that cuts off than sums
    that cancel.  Each product may lose a step of the sum, 2^-23 of it: D 2^-23 of
    the logit, and 4 more for its factor; lse times log2 e, exp2 and the additions
    of T G weights as in any other weight."""
    Hkv, n = 2, 900
    p = Pair(1, Hkv, D, 960, 64, 64, O.E4M3, seed=99)
    ws = p.c.workspace(T, Hkv * G)
    p.append(*(p.rows(n, Hkv, "f32").abs() for _ in "kv"), ws)
    q = sign * p.rows(T, Hkv * G, dtype).abs()
    k = [p.seq[0, h, "k"].values() for h in range(Hkv)]
    lse = np.zeros((T, Hkv * G))
    scale = 25 / max((np.abs(q[0].double().numpy()) @ k[0].T).mean(), 1e-9)
    qn = q[0].double().numpy()
    for h in range(Hkv):
        hs = slice(h * G, (h + 1) * G)
        lse[:, hs] = O.attention(qn[:, hs], k[h], k[h], scale)[1]
    lse = lse.astype(np.float32)
    K.kv8_mass(p.c, q.cuda(), torch.from_numpy(lse)[None].cuda(), ws, softmax_scale=scale, decay=0.0)
    assert K.get_status(ws) == 0
    scale = float(np.float32(scale))
    for h in range(Hkv):
        hs = slice(h * G, (h + 1) * G)
        want = O.mass(qn[:, hs], lse[:, hs].astype(np.float64), k[h], scale)
        big = scale * (np.abs(qn[:, hs]).reshape(-1, D) @ k[h].T).max()
        rel = ((D + 4) * 2.0 ** -23 * big + 2.0 ** -22 * np.abs(lse).max() + 2.0 ** -20
               + (T * G + 2) * 2.0 ** -23)
        got = p.at("mass", 0, h)[:n].astype(np.float64)
        assert (np.abs(got - want) <= rel * want + 1e-36).all(), np.max(np.abs(got - want) / (want + 1e-36)) / rel


def test_lengths_out_of_range_are_clamped():
    """q_len and new_len below 0 and above T, seq_len below 0 and above the capacity."""
    B, Hkv, G, D, cap = 4, 2, 2, 64, 96
    H = Hkv * G
    p = Pair(B, Hkv, D, cap, 16, 16, O.INT8, seed=101)
    ws = p.c.workspace(40, H)
    p.append(p.rows(cap, Hkv, "bf16"), p.rows(cap, Hkv, "bf16"), ws)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for T in (3, 40):
        q = p.rows(T, H, "f16", 0.7).cuda()
        got = []
        for lens, q_len in (([96, 96, 0, 50], [0, T, T, 1]), ([2 ** 30, 97, -7, 50], [-2 ** 31, 2 ** 31 - 1, T + 1, 1])):
            p.c.seq_len.copy_(ints(lens))
            out, lse = torch.full_like(q, 7.0), torch.full((B, T, H), 7.0, device="cuda")
            K.kv8_attn(p.c, q, out, ws, lse=lse, q_len=ints(q_len))
            p.c.mass.fill_(0.5)
            K.kv8_mass(p.c, q, lse, ws, q_len=ints(q_len), decay=0.5)
            assert p.c.seq_len.tolist() == lens
            got.append((out, lse, p.c.mass.clone()))
        assert all(torch.equal(x, y) for x, y in zip(*got))
        assert (got[0][0][0] == 7.0).all() and (got[0][0][2] == 0).all()
        k = p.rows(T, Hkv, "f16").cuda()
        start = ints([10, 20, 30, 40])
        stored = []
        for new in ([0, T, T, 1], [-5, 2 ** 31 - 1, T + 9, 1]):
            K.kv8_append(p.c, k, k, ws, new_len=ints(new), start=start)
            assert p.c.seq_len.tolist() == [10, 20 + T, 30 + T, 41]
            # (bits: unused pages' scales are NaN)
            stored.append([t.view(torch.uint8).clone()
                           for t in (p.c.k_codes, p.c.v_codes, p.c.k_scales, p.c.v_scales)])
        assert all(torch.equal(x, y) for x, y in zip(*stored))
    assert K.get_status(ws) == 0


def test_weights_of_no_queries_decay():
    p = Pair(2, 2, 64, 200, 16, 16, O.E4M3, seed=102)
    ws = p.c.workspace(1, 4)
    p.append(p.rows(130, 2, "bf16"), p.rows(130, 2, "bf16"), ws, lens=[130, 7])
    p.c.mass.fill_(3.0)
    q, lse = torch.zeros(2, 0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 0, 4, device="cuda")
    K.kv8_mass(p.c, q, lse, ws, decay=0.5)
    for b, n in ((0, 130), (1, 7)):
        for h in range(2):
            m = p.at("mass", b, h)
            assert (m[:n] == 1.5).all() and (m[n:] == 3.0).all()
    assert K.get_status(ws) == 0


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("T,G", [(3, 4), (40, 2)])
def test_storage_beyond_4_gib(T, G, paged):
    """K and V of 5 GiB each, of which the last rows are used."""
    B, Hkv, D, block = (40, 8, 128, 64) if not paged else (3, 8, 128, 64)
    H, page = Hkv * G, 64
    cap = 131072 if not paged else 4096
    if paged:
        pages = 5 * 2 ** 30 // (Hkv * page * D)
        table = torch.arange(pages - 1, pages - 1 - B * cap // page, -1, dtype=torch.int32).view(B, -1)
    p = Pair(1 if paged else B, Hkv, D, block, block, 0, O.E4M3, seed=103)
    p.B, p.table = B, table if paged else None
    p.c = K.Cache8(B, Hkv, D, cap, block=block, page_size=page if paged else 0,
                   page_table=table if paged else None, num_pages=pages if paged else 0, fmt=O.E4M3, mass=True)
    assert p.c.k_codes.numel() > 2 ** 32
    p.seq = {(b, h, s): O.Seq(block, O.E4M3, D) for b in range(B) for h in range(Hkv) for s in "kv"}
    lens = [0] * (B - 2) + [300, 131]
    p.len = [0] * B
    ws = p.c.workspace(T, H)
    p.append(p.rows(300, Hkv, "bf16"), p.rows(300, Hkv, "bf16"), ws, lens=lens)
    p.append(p.rows(2, Hkv, "bf16"), p.rows(2, Hkv, "bf16"), ws, lens=[0] * (B - 1) + [2])
    p.check()
    q = p.rows(T, H, "bf16", 0.7)
    out, lse = torch.empty(B, T, H, D, dtype=q.dtype, device="cuda"), torch.empty(B, T, H, device="cuda")
    K.kv8_attn(p.c, q.cuda(), out, ws, lse=lse)
    K.kv8_mass(p.c, q.cuda(), lse, ws, decay=0.0)
    for b in (B - 2, B - 1):
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            ro, rl, tol, ltol = attention_bounds(q[b, :, hs].double().numpy(), p, b, h, G, T, 1 / math.sqrt(D),
                                                 2.0 ** -8)
            assert (np.abs(out[b, :, hs].cpu().double().numpy() - ro) <= tol).all()
            assert (np.abs(lse[b, :, hs].cpu().double().numpy() - rl) <= ltol).all()
            m = p.at("mass", b, h)[: p.len[b]].astype(np.float64)
            assert abs(m.sum() - T * G) < 1e-4 * T * G
    kept = torch.empty(B, Hkv, 100, dtype=torch.int32, device="cuda")
    w = {(b, h): p.at("mass", b, h) for b in (B - 2, B - 1) for h in range(Hkv)}
    K.kv8_evict(p.c, 100, 4, 16, kept, ws)
    for (b, h), x in w.items():
        rows = O.evict(x, p.len[b], 100, 4, 16)
        assert kept[b, h].tolist() == rows.tolist()
        for s in "kv":
            p.seq[b, h, s] = p.seq[b, h, s].keep(rows)
    p.len[B - 2:] = [100, 100]
    p.check()
    assert K.get_status(ws) == 0
