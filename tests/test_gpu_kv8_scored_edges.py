"""The attention with changed scores where its arithmetic is nearest to its limits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import fp4_kv_cache_rope_gb300 as K  # noqa: E402
from oracle import kv8 as O  # noqa: E402
from kv8_tools import Pair  # noqa: E402
from kv8_more_tools import check_attention, ints, scored_want  # noqa: E402
from test_gpu_kv8_scored import filled, run_scored, run_tree, slopes_of  # noqa: E402


def scored(p, q, k=None, v=None, scale=0.0, **args):
    """(out, lse) on the host; with k and v of drafted tokens, each of which follows the one before."""
    B, T, H, _ = q.shape
    ws = p.c.tree_workspace(T, H)
    out, lse = torch.empty(q.shape, dtype=q.dtype, device="cuda"), torch.empty(B, T, H, device="cuda")
    if k is None:
        K.kv8_attn_scored(p.c, q.cuda(), out, ws, K.Scores(**args), lse=lse, softmax_scale=scale)
    else:
        K.kv8_attn_tree(p.c, q.cuda(), k.cuda(), v.cuda(), ints([[t - 1 for t in range(T)]] * B), out, ws, lse=lse,
                        softmax_scale=scale, scores=K.Scores(**args))
    assert K.get_status(ws) == 0
    return out.cpu(), lse.cpu()


def digits(n):
    """n in base 128 with digits from -64 to 63, the last one what is left."""
    d = []
    for _ in range(3):
        low = (n + 64) % 128 - 64
        d.append(low)
        n = (n - low) // 128
    return d + [n]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("drafted", [False, True])
@pytest.mark.parametrize("T,G", [(1, 4), (40, 4)])
def test_the_largest_cap(D, drafted, T, G):
    """Scores over the cap in steps of 2^-18, held exactly: tile after tile of the first, whose
    capped score the second's exceeds by 8 (base 2, the most that the many-row kernel leaves its
    maximum behind), among them the third, a smaller score that comes out above the second by
    1 for the quotient's roundings."""
    first, second, third = 1666109, 2226092, 2218733
    n, cap = 300, 2.0 ** 20
    p = Pair(1, 1, D, n, 16, 16, O.INT8, seed=81, mass=False)
    k = torch.zeros(1, n, 1, D)
    for j in range(n):
        k[0, j, 0, :4] = torch.tensor(digits(first if j < 128 else second if j % 2 else third), dtype=torch.float32)
    k[..., 4] = 64.0                     # the blocks' scales are 1 then
    p.append(k, p.rows(n, 1, "f32"), p.c.workspace(1, 1))
    q = torch.zeros(1, T, G, D)
    q[..., :4] = 128.0 ** torch.arange(4.0)
    q = q.bfloat16()
    kd, vd = (torch.zeros(1, T, 1, D, dtype=torch.bfloat16), p.rows(T, 1, "bf16")) if drafted else (None, None)
    out, lse = scored(p, q, kd, vd, scale=cap * 2.0 ** -18, cap=cap)
    more = {} if kd is None else dict(k=kd[0, :, 0].double().numpy(), v=vd[0, :, 0].double().numpy(),
                                      parent=[t - 1 for t in range(T)])
    check_attention(out[0], lse[0], scored_want(p, q, 0, 0, G, T, cap * 2.0 ** -18, "bf16", cap, **more))


@pytest.mark.parametrize("T,G", [(1, 8), (40, 4)])
@pytest.mark.parametrize("size", [0.1, 0.4, 1.0])
def test_scores_about_and_beyond_the_largest_cap(T, G, size):
    p = filled(2, 2, 128, [700, 130], 64, 64, O.E4M3, seed=82)
    run_scored(p, G, T, "bf16", cap=2.0 ** 20, scale=2.0 ** 20, size=size)


@pytest.mark.parametrize("cap", [30.0, 300.0, 3000.0])
@pytest.mark.parametrize("what", ["key", "query", "front key"])
def test_far_larger_scores_that_are_not_seen_change_no_bits(cap, what):
    """A key becomes 30 times as large, which comes later than some tokens or lies in front
    of all windows, or the last token's query does.  The tokens that share none of the last
    one's 32 query rows keep their bits."""
    T, G, n = 48, 4, 97
    res = []
    for big in (1.0, 30.0):
        p = Pair(1, 1, 128, n, 16, 16, O.E4M3, seed=83, mass=False)
        k, v, q = p.rows(n, 1, "f32"), p.rows(n, 1, "f32"), p.rows(T, G, "f16", 0.02 * cap)
        if what == "key":
            k[0, n - 1] *= big           # alone in its block
        elif what == "query":
            q[0, T - 1] *= big
        else:
            k[0, :16] *= big
        p.append(k, v, p.c.workspace(1, 1))
        res.append(scored(p, q, cap=cap, window=30 if what == "front key" else 0))
    last = T if what == "front key" else T - 32 // G
    for a, b in zip(*res):
        assert torch.equal(a[0, :last], b[0, :last])


@pytest.mark.parametrize("T,G", [(1, 4), (40, 4)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("slope", [2.0 ** 24, 2.0 ** 20, 2.0 ** 14, 1.0])
def test_slopes_that_cancel_huge_logits(T, G, D, slope):
    """One row's score is q.k = slope * (p - j) less the slope's bias: 0, but for the roundings
    of numbers up to 2^31, which are far above 1, and every other row's lies far below.
    Whatever is left of that score, the row's V comes out."""
    n, at = 160, 77
    p = Pair(1, 1, D, n, 16, 16, O.INT8, seed=84, mass=False)
    k = torch.zeros(1, n, 1, D)
    k[..., 0] = (torch.arange(n) - 64.0).view(1, n, 1)
    k[..., 1] = 1.0
    k[..., 2] = 100.0
    k[0, at, 0, 2] = 0.0
    p.append(k, p.rows(n, 1, "f32"), p.c.workspace(1, 1))
    slopes = slope * 2.0 ** -torch.arange(float(G))
    i = torch.arange(float(T)).view(T, 1)

    def queries(first):                  # at first, first + 1, ..
        q = torch.zeros(1, T, G, D)
        q[0, :, :, 0] = -slopes
        q[0, :, :, 1] = slopes * (first + i - 64.0)
        q[0, :, :, 2] = -max(1.0, 2.0 ** -7 * slope)
        assert torch.equal(q, q.bfloat16().float())
        return q.bfloat16()

    for chain in (False, True):
        q = queries(n if chain else n - T)
        more, drafts = {}, {}
        if chain:
            drafts = dict(k=torch.zeros(1, T, 1, D, dtype=torch.bfloat16), v=p.rows(T, 1, "bf16"))
            drafts["k"][..., 2] = 100.0
            more = dict(k=drafts["k"][0, :, 0].double().numpy(), v=drafts["v"][0, :, 0].double().numpy(),
                        parent=[t - 1 for t in range(T)])
        out, lse = scored(p, q, scale=1.0, slopes=slopes.cuda(), **drafts)
        want = scored_want(p, q, 0, 0, G, T, 1.0, "bf16", slopes=slopes.numpy(), **more)
        check_attention(out[0], lse[0], want, chain)


@pytest.mark.parametrize("B,Hkv,G,T", [(1, 1, 1, 256), (3, 2, 2, 256), (2, 1, 1, 64)])
@pytest.mark.parametrize("what", ["none", "window", "all"])
def test_paths_through_every_token(B, Hkv, G, T, what):
    """The longest path that there is; with one query row to a CTA (few rows), and without."""
    p = filled(B, Hkv, 64, [300, 1, 77][:B], 16, 16, O.E4M3, seed=85)
    chain = [i - 1 for i in range(T)]
    args = {"none": {}, "window": dict(window=100, sink=310),
            "all": dict(window=200, sink=5, cap=6.0, slopes=slopes_of(Hkv * G))}[what]
    run_tree(p, G, T, "bf16", size=2.0, parent=[list(chain) for _ in range(B)], **args)
    run_tree(p, G, T, "f16", q_len=[T - 1, T, 3][:B], parent=[list(chain) for _ in range(B)], **args)
