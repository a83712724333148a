"""Refusals of the calls for rotated, scored and drafted tokens, before any launch."""
import ctypes
import math

import pytest
import torch

import fp4_kv_cache_rope_gb300 as K
from test_kv8_refusals import contiguous

BAD, OK = K.CSA2_ERR_INVALID, K.CSA2_OK
WS, SEQ = 256, 1 << 20


def rows(at=1 << 31, heads=8, D=128, T=3, kind=K.BF16, **over):
    s = dict(stride_b=T * heads * D, stride_t=heads * D, stride_h=D)
    s.update(over)
    return K.Csa2Rows(at, s["stride_b"], s["stride_t"], s["stride_h"], kind)


def table(**over):
    f = dict(cos=1 << 22, sin=1 << 23, positions=100, dim=64, first=0, style=K.ROPE_HALVES)
    f.update(over)
    return K.Csa2Rope(*f.values())


def ref(x):
    return None if x is None else ctypes.byref(x)


def rope(c, t, q, qo, k=None, ko=None, T=3, H=8, q_len=None, pos=None, parent=None, ws=WS):
    return K._kv8_rope(ref(c), ref(t), ref(q), H, ref(qo), ref(k), ref(ko), T, q_len, pos, parent, ws, None)


def append_rope(c, t, k, v, T=3, q=None, H=0, qo=None, new_len=None, start=None, pos=None, ws=WS):
    return K._kv8_append_rope(ref(c), ref(t), ref(k), ref(v), T, ref(q), H, ref(qo), new_len, start, pos, ws,
                              None)


def path(c, k, v, T=3, at=512, M=2, new_len=None, start=None, ws=WS):
    return K._kv8_append_path(ref(c), ref(k), ref(v), T, at, M, new_len, start, ws, None)


def scored(c, s, q, out, T=3, H=8, scale=0.0, lse=None, ws=WS):
    return K._kv8_attn_scored(ref(c), ref(q), H, T, None, scale, ref(s), ref(out), lse, ws, None)


def tree(c, q, k, v, out, parent=512, T=3, H=8, scale=0.0, s=None, ws=WS):
    return K._kv8_attn_tree(ref(c), ref(q), H, ref(k), ref(v), parent, T, None, scale, ref(s), ref(out), None,
                            ws, None)


def cache():
    return contiguous(1 << 30, SEQ)


TABLES = [dict(cos=None), dict(sin=None), dict(cos=(1 << 22) + 8), dict(sin=(1 << 22) + 4), dict(positions=0),
          dict(positions=(1 << 21) + 1), dict(dim=8), dict(dim=40), dict(dim=0), dict(dim=144),
          dict(first=-8), dict(first=4), dict(first=72), dict(style=2), dict(style=-1)]


@pytest.mark.parametrize("over", TABLES, ids=lambda o: "-".join(f"{k}{v}" for k, v in o.items()))
def test_tables(over):
    c = cache()
    assert rope(c, table(**over), rows(), rows(1 << 32)) == BAD
    assert append_rope(c, table(**over), rows(heads=4), rows(1 << 33, heads=4)) == BAD
    assert rope(c, None, rows(), rows(1 << 32)) == BAD


def test_rope_arguments():
    c, t = cache(), table()
    q, qo, k, ko = rows(), rows(1 << 32), rows(1 << 33, 4), rows(1 << 34, 4)
    assert rope(c, t, q, qo, T=0) == OK
    for args in [dict(H=0), dict(H=6), dict(T=-1), dict(ws=0), dict(ws=128), dict(q_len=2), dict(pos=6),
                 dict(parent=1026), dict(pos=512, parent=1024), dict(parent=512, T=257)]:
        assert rope(c, t, q, qo, **args) == BAD, args
    for args in [(None, qo), (q, None), (rows(8), qo), (q, rows(1 << 32, kind=K.F16)), (q, rows(1 << 32, stride_h=0)),
                 (q, rows(1 << 32, stride_t=4)), (rows(kind=3), rows(1 << 32, kind=3)), (q, qo, k, None),
                 (q, qo, None, ko), (q, qo, k, rows(1 << 34, 4, stride_b=128)),
                 (q, qo, rows(1 << 33, 4, kind=K.F32), rows(1 << 34, 4, kind=K.F32)),
                 (q, qo, k, rows(1 << 34, 4, kind=K.F16))]:
        assert rope(c, t, *args) == BAD, args


def test_append_rope_arguments():
    c, t = cache(), table()
    k, v, q, qo = rows(1 << 33, 4), rows(1 << 34, 4), rows(), rows(1 << 32)
    assert append_rope(c, t, k, v, T=0) == OK
    assert append_rope(c, t, None, None, T=0) == OK
    for args in [dict(T=-1), dict(ws=0), dict(ws=64), dict(q=q), dict(q=q, H=8), dict(qo=qo, H=8), dict(H=8),
                 dict(q=q, qo=qo, H=6), dict(q=q, qo=rows(1 << 32, kind=K.F16), H=8),
                 dict(q=q, qo=rows(1 << 32, stride_t=0), H=8), dict(new_len=SEQ), dict(start=SEQ + 4),
                 dict(pos=SEQ), dict(pos=SEQ + 4), dict(pos=SEQ - 4 * 6 + 4), dict(pos=510), dict(start=1)]:
        assert append_rope(c, t, k, v, **args) == BAD, args
    for args in [(None, v), (k, None), (k, rows(1 << 34, 4, kind=K.F32)), (rows(12, 4), v)]:
        assert append_rope(c, t, *args) == BAD, args


def test_append_path_arguments():
    c = cache()
    k, v = rows(1 << 33, 4), rows(1 << 34, 4)
    assert path(c, k, v, M=0) == OK and path(c, None, None, T=0, M=0) == OK
    for args in [dict(T=0), dict(T=-1), dict(M=-1), dict(M=(1 << 21) + 1), dict(at=None), dict(at=514),
                 dict(at=SEQ), dict(at=SEQ + 4), dict(at=SEQ - 12), dict(new_len=SEQ), dict(start=SEQ + 4),
                 dict(ws=0)]:
        assert path(c, k, v, **args) == BAD, args
    for args in [(None, v), (k, None), (k, rows(1 << 34, 4, kind=K.F32))]:
        assert path(c, *args) == BAD, args


def test_scores():
    c, q, out = cache(), rows(), rows(1 << 32)
    good = K.Csa2Scores(30.0, 100, 4, 512, 512)
    assert scored(c, good, q, out, T=0) == OK
    assert scored(c, None, q, out) == BAD
    for s in [(-1.0, 0, 0), (2.0 ** -11, 0, 0), (2.0 ** 21, 0, 0), (math.inf, 0, 0), (math.nan, 0, 0), (0.0, -1, 0),
              (0.0, 5, -1), (0.0, 0, 0, 510), (0.0, 0, 0, None, 511)]:
        s = K.Csa2Scores(*s)
        assert scored(c, s, q, out) == BAD and scored(c, s, q, out, T=0) == BAD
        assert tree(c, q, rows(1 << 33, 4), rows(1 << 34, 4), out, s=s) == BAD
    for args in [dict(scale=math.inf), dict(scale=2.0 ** -101), dict(H=6), dict(T=-1), dict(ws=0), dict(lse=2)]:
        assert scored(c, good, q, out, **args) == BAD, args
    for a, b in [(None, out), (q, None), (rows(kind=K.F32), rows(1 << 32, kind=K.F32)), (q, rows(1 << 32, kind=K.F16)),
                 (q, rows(1 << 32, stride_h=64))]:
        assert scored(c, good, a, b) == BAD


def test_trees():
    c, q, k, v, out = cache(), rows(), rows(1 << 33, 4), rows(1 << 34, 4), rows(1 << 32)
    assert tree(c, q, k, v, out, T=0) == OK
    for args in [dict(T=257), dict(T=-1), dict(H=6), dict(parent=None), dict(parent=1), dict(ws=0),
                 dict(scale=2.0 ** 101), dict(s=K.Csa2Scores(0.0, 0, 0, None, 512))]:
        assert tree(c, q, k, v, out, **args) == BAD, args
    f32 = dict(kind=K.F32)
    for a in [(None, k, v, out), (q, None, v, out), (q, k, None, out), (q, k, v, None),
              (q, rows(1 << 33, 4, kind=K.F16), v, out), (q, k, rows(1 << 34, 4, kind=K.F16), out),
              (rows(**f32), rows(1 << 33, 4, **f32), rows(1 << 34, 4, **f32), rows(1 << 32, **f32)),
              (q, k, v, rows(1 << 32, stride_b=0)), (q, rows((1 << 33) + 8, 4), v, out)]:
        assert tree(c, *a) == BAD
    size = K._kv8_tree_workspace_size
    plain = K._kv8_workspace_size(ref(c), 256, 8)
    assert size(ref(c), 257, 8) == 0 and size(ref(c), 3, 6) == 0
    assert size(ref(c), 0, 8) == plain and size(ref(c), 256, 8) >= plain + 2 * 256 * 8 * 132 * 4
    assert size(ref(c), 3, 8) == (plain + 2 * 3 * 8 * 132 * 4 + 255) // 256 * 256


@pytest.mark.parametrize("batch,heads,max_len", [(1, 1, 1 << 20), (2, 8, 131072), (16, 4, 9024), (40, 8, 4096),
                                                 (152, 2, 65536), (3, 5, 50048)])
def test_a_tree_workspace_serves_fewer_tokens(batch, heads, max_len):
    """What a call of T tokens takes is enough for every call of fewer."""
    c = contiguous(1 << 30, SEQ)
    c.batch, c.kv_heads, c.max_len = batch, heads, max_len
    for G in (1, 3, 8, 40):
        sizes = [K._kv8_tree_workspace_size(ref(c), T, heads * G) for T in range(257)]
        assert sizes[0] > 0 and sizes == sorted(sizes), G
        # and it holds the rows, and the parts of the split that T itself gets
        plain = K._kv8_workspace_size(ref(c), 1, heads * G)
        for T in (1, 16, 64, 256):
            parts = 0
            if T * G > 64:
                base = batch * heads * -(-T * G // 256)
                splits = max(1, min(304 // base, -(-max_len // 1024)))
                parts = base * splits * 256 * 130 * 4 if splits > 1 else 0
            assert sizes[T] >= plain + max(batch * T * heads * G * 132 * 4, parts)


# ------------------------------------------------------------------- the binding
def test_handles():
    cos = torch.zeros(10, 8)
    r = K.Rope(cos, cos)
    assert (r.struct.positions, r.struct.dim, r.struct.first, r.struct.style) == (10, 16, 0, K.ROPE_HALVES)
    assert K.Rope(cos.double()[:, ::2], cos.double()[:, ::2]).cos.is_contiguous()
    for a, b in ((cos, cos[:5]), (cos[0], cos[0]), (cos[:0], cos[:0])):
        with pytest.raises(K.Csa2Error, match="cos and sin"):
            K.Rope(a, b)
    with pytest.raises(K.Csa2Error, match="slopes"):
        K.Scores(slopes=torch.zeros(4, dtype=torch.float64))
    with pytest.raises(K.Csa2Error, match="slopes"):
        K.Scores(slopes=torch.zeros(4, 1))
    with pytest.raises(K.Csa2Error, match="prefix"):
        K.Scores(prefix=torch.zeros(8, dtype=torch.int32)[::2])


def test_the_binding_names_what_it_refuses():
    c = K.Cache8(2, 4, 64, 128, block=32, device="cpu")
    ws = torch.zeros(1 << 26, dtype=torch.uint8)
    f = lambda T, H, dt=torch.bfloat16: torch.zeros(2, T, H, 64, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    r = K.Rope(torch.zeros(9, 16), torch.zeros(9, 16))
    no = [
        ("q_out", lambda: K.kv8_rope(c, f(3, 8), f(3, 8, torch.float16), r, ws)),
        ("q_out", lambda: K.kv8_rope(c, f(3, 8), f(4, 8), r, ws)),
        ("k_out", lambda: K.kv8_rope(c, f(3, 8), f(3, 8), r, ws, k=f(3, 4))),
        ("k: T", lambda: K.kv8_rope(c, f(3, 8), f(3, 8), r, ws, k=f(2, 4), k_out=f(3, 4))),
        ("k: shape", lambda: K.kv8_rope(c, f(3, 8), f(3, 8), r, ws, k=f(3, 8), k_out=f(3, 8))),
        ("not both", lambda: K.kv8_rope(c, f(3, 8), f(3, 8), r, ws, pos=i(2, 3), parent=i(2, 3))),
        ("at most 256", lambda: K.kv8_rope(c, f(257, 8), f(257, 8), r, ws, parent=i(2, 257))),
        ("pos", lambda: K.kv8_rope(c, f(3, 8), f(3, 8), r, ws, pos=i(2, 4))),
        ("v: T", lambda: K.kv8_append_rope(c, f(3, 4), f(3, 4, torch.float32), r, ws)),
        ("q_out", lambda: K.kv8_append_rope(c, f(3, 4), f(3, 4), r, ws, q=f(3, 8))),
        ("q: the T", lambda: K.kv8_append_rope(c, f(3, 4), f(3, 4), r, ws, q=f(2, 8), q_out=f(2, 8))),
        ("path", lambda: K.kv8_append_path(c, f(3, 4), f(3, 4), i(2), ws)),
        ("path", lambda: K.kv8_append_path(c, f(3, 4), f(3, 4), i(3, 2), ws)),
        ("no rows", lambda: K.kv8_append_path(c, f(0, 4), f(0, 4), i(2, 2), ws)),
        ("slopes", lambda: K.kv8_attn_scored(c, f(3, 8), f(3, 8), ws, K.Scores(slopes=torch.zeros(4)))),
        ("prefix", lambda: K.kv8_attn_scored(c, f(3, 8), f(3, 8), ws, K.Scores(prefix=i(3)))),
        ("rope: 16 channels from 4", lambda: K.kv8_rope(c, f(3, 8), f(3, 8), K.Rope(torch.zeros(9, 8), torch.zeros(9, 8), first=4), ws)),
        ("rope: 128 channels", lambda: K.kv8_append_rope(c, f(3, 4), f(3, 4), K.Rope(torch.zeros(9, 64), torch.zeros(9, 64)), ws)),
        ("a Scores", lambda: K.kv8_attn_scored(c, f(3, 8), f(3, 8), ws, None)),
        ("a Scores", lambda: K.kv8_attn_tree(c, f(3, 8), f(3, 4), f(3, 4), i(2, 3), f(3, 8), ws, scores=30.0)),
        ("out", lambda: K.kv8_attn_scored(c, f(3, 8), f(3, 4), ws, K.Scores())),
        ("at most 256", lambda: K.kv8_attn_tree(c, f(257, 8), f(257, 4), f(257, 4), i(2, 257), f(257, 8), ws)),
        ("parent", lambda: K.kv8_attn_tree(c, f(3, 8), f(3, 4), f(3, 4), None, f(3, 8), ws)),
        ("parent", lambda: K.kv8_attn_tree(c, f(3, 8), f(3, 4), f(3, 4), i(2, 4), f(3, 8), ws)),
        ("prefix", lambda: K.kv8_attn_tree(c, f(3, 8), f(3, 4), f(3, 4), i(2, 3), f(3, 8), ws,
                                           scores=K.Scores(prefix=i(2)))),
        ("k: T", lambda: K.kv8_attn_tree(c, f(3, 8), f(3, 4, torch.float16), f(3, 4), i(2, 3), f(3, 8), ws)),
        ("workspace", lambda: K.kv8_attn_tree(c, f(3, 8), f(3, 4), f(3, 4), i(2, 3), f(3, 8), ws[:1 << 20])),
        ("KV8_MAX_TREE", lambda: c.tree_workspace(257, 8)),
        ("CUDA device", lambda: K.kv8_attn_tree(c, f(3, 8), f(3, 4), f(3, 4), i(2, 3), f(3, 8), ws)),
    ]
    for text, call in no:
        with pytest.raises(K.Csa2Error, match=text):
            call()
    assert c.tree_workspace(3, 8).numel() > K.kv8_workspace_size(c, 3, 8)
