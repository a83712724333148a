"""CPU pins of the 8-bit K/V cache's oracle, and the refusals of its calls."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fp4_kv_cache_rope_gb300 as K
from oracle import kv8 as O


@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
def test_scale_is_the_smallest_that_holds(fmt):
    rng = np.random.default_rng(1)
    q = O.QMAX[fmt]
    for amax in [q, q * 1.0001, q / 2, q * 2.0 ** -130, 2.0 ** -149, 3.0e38,
                 *np.exp(rng.uniform(-80, 80, 50))]:
        s = O.scale_of(float(amax), fmt)
        assert math.frexp(s)[0] == 0.5 and amax <= q * s
        assert s == 2.0 ** -126 or amax > q * s / 2
    assert O.scale_of(0.0, fmt) == 0.0


def test_nearest_matches_torch():
    x = np.concatenate([np.linspace(-448, 448, 20001), np.random.default_rng(0).standard_normal(5000)])
    x = x.astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(O.nearest(x, O.E4M3), t)
    assert np.array_equal(O.nearest([0.5, 1.5, -2.5, 200.0], O.INT8), [0, 2, -2, 127])


@pytest.mark.parametrize("fmt", [O.E4M3, O.INT8])
def test_append_error_is_half_a_step_of_the_block(fmt):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((70, 64))
    s = O.Seq(32, fmt, 64)
    s.append(x)
    amax = np.array([np.abs(x[i:i + 32]).max() for i in (0, 32, 64)])
    err = np.abs(s.values() - x)
    if fmt == O.INT8:
        assert (err <= np.repeat(s.scales, 32)[:70, None] / 2).all()
    else:
        assert (err <= np.maximum(np.abs(x) / 16, np.repeat(s.scales, 32)[:70, None] * 2.0 ** -10)).all()
    assert (amax <= O.QMAX[fmt] * s.scales).all()


def test_one_by_one_only_differs_by_requantised_rows():
    """E4M3 codes lose nothing when a block's scale doubles unless they are small."""
    rng = np.random.default_rng(3)
    x = rng.standard_normal((64, 64)) * np.exp2(np.arange(64) / 8)[:, None]
    a, b = O.Seq(64, O.E4M3, 64), O.Seq(64, O.E4M3, 64)
    a.append(x)
    for r in x:
        b.append(r[None])
    assert np.array_equal(a.scales, b.scales)
    small = np.abs(x) < a.scales[0] * 2.0 ** -6
    assert np.array_equal(a.values()[~small], b.values()[~small])
    assert (np.abs(a.values() - b.values())[small] <= a.scales[0] * 2.0 ** -9).all()


def test_truncating_append_and_eviction():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((100, 64))
    s = O.Seq(16, O.INT8, 64)
    s.append(x)
    s.append(x[:5], start=40)
    assert len(s.codes) == 45 and len(s.scales) == 3
    w = np.array([5, 1, 1, 9, 1, 0, 7, 7], float)
    assert O.evict(w, 8, 8, 0, 0).tolist() == list(range(8))
    assert O.evict(w, 8, 5, 1, 1).tolist() == [0, 1, 3, 6, 7]
    assert O.evict(np.array([0, np.nan, 2, 2, np.inf, 2]), 6, 4, 0, 0).tolist() == [1, 2, 3, 4]
    kept = np.array([0, 1, 2, 5, 30])
    k = s.keep(kept)
    assert np.abs(k.values() - s.values()[kept]).max() <= k.scales.max() / 2
    same = s.keep(np.r_[np.arange(16), 20, 31])
    assert same.scales[0] == s.scales[0] and np.array_equal(same.codes[:16], s.codes[:16])


def test_attention_and_mass_agree_with_torch():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((3, 2, 64)), rng.standard_normal((9, 64)), rng.standard_normal((9, 64))
    o, lse, _, _ = O.attention(q, k, v, 0.125)
    x = torch.from_numpy(q).permute(1, 0, 2) @ torch.from_numpy(k).T * 0.125
    x = x.masked_fill(torch.arange(9) > torch.arange(6, 9)[:, None], -torch.inf)
    p = torch.softmax(x, -1)
    assert np.allclose(o, (p @ torch.from_numpy(v)).permute(1, 0, 2).numpy())
    assert np.allclose(lse, torch.logsumexp(x, -1).T.numpy())
    assert np.allclose(O.mass(q, lse, k, 0.125), p.sum((0, 1)).numpy())
    # more queries than rows: the first see nothing
    o, lse, _, _ = O.attention(q, k[:2], v[:2], 0.125)
    assert (o[0] == 0).all() and (lse[0] == -np.inf).all() and np.isfinite(lse[1:]).all()


# ------------------------------------------------------------------- refusals
def base():
    return K.Csa2Kv8Cache(2, 4, 128, 64, 0, 0, 1024, 0, K.KV8_E4M3, 256, 256, 256, 256, 256, None, 256)


def test_cache_descriptions():
    assert K.kv8_workspace_size(base(), 1, 8) > 0
    paged = K.Csa2Kv8Cache(2, 4, 128, 16, 48, 30, 1000, 9, K.KV8_INT8, 256, 256, 256, 256, None, 512, 256)
    assert K.kv8_workspace_size(paged, 5, 4) > 0
    for c0, field, value in [
            (base(), "batch", 0), (base(), "batch", 70000), (base(), "kv_heads", 0),
            (base(), "dim", 96), (base(), "block", 48), (base(), "block", 8), (base(), "max_len", 0),
            (base(), "max_len", 1000), (base(), "max_len", 1 << 22), (base(), "format", 2),
            (base(), "k_codes", None), (base(), "v_codes", 264), (base(), "k_scales", 258),
            (base(), "seq_len", None), (base(), "page_size", -16),
            (paged, "page_size", 40), (paged, "page_table", None), (paged, "num_pages", 0),
            (paged, "max_pages_per_seq", 20)]:
        bad = K.Csa2Kv8Cache.from_buffer_copy(c0)
        setattr(bad, field, value)
        assert K.kv8_workspace_size(bad, 1, 8) == 0, (field, value)
    for T, H in [(-1, 8), (1, 0), (1, 6), (1 << 30, 8)]:
        assert K.kv8_workspace_size(base(), T, H) == 0


def test_struct_layout_matches_header(tmp_path):
    import os
    import shutil
    import subprocess
    gcc = shutil.which("gcc") or shutil.which("cc")
    if gcc is None:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    lines, want = [], []
    for st, name in ((K.Csa2Kv8Cache, "csa2_kv8_cache"), (K.Csa2Rows, "csa2_rows")):
        for f in st._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f[0]}));')
            want.append(getattr(st, f[0]).offset)
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(st))
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "csa2.h"\nint main(void){\n'
                   + "\n".join(lines) + "\nreturn 0;}\n")
    subprocess.run([gcc, "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                           text=True).stdout.split()] == want


def test_calls_refuse_before_any_launch():
    c = base()
    r = K.Csa2Rows(256, 1024, 512, 128, K.BF16)

    def rows(**kw):
        x = K.Csa2Rows.from_buffer_copy(r)
        for n, v in kw.items():
            setattr(x, n, v)
        return ctypes.byref(x)

    ok = ctypes.byref(r)
    cp = ctypes.byref(c)
    bad = [
        K._kv8_append(cp, None, ok, 4, None, None, 256, None),
        K._kv8_append(cp, ok, ok, -1, None, None, 256, None),
        K._kv8_append(cp, ok, ok, 4, None, None, None, None),
        K._kv8_append(cp, ok, ok, 4, None, None, 264, None),
        K._kv8_append(cp, ok, ok, 4, 258, None, 256, None),
        K._kv8_append(cp, ok, ok, 4, 256, None, 256, None),       # new_len is seq_len
        K._kv8_append(cp, ok, ok, 4, None, 260, 256, None),       # start overlaps seq_len
        K._kv8_append(cp, ok, rows(type=K.F16), 4, None, None, 256, None),
        K._kv8_append(cp, rows(type=3), rows(type=3), 4, None, None, 256, None),
        K._kv8_append(cp, rows(data=264), ok, 4, None, None, 256, None),
        K._kv8_append(cp, ok, rows(stride_t=516), 4, None, None, 256, None),
        K._kv8_attn(cp, ok, 6, 1, None, 0.0, ok, None, 256, None),
        K._kv8_attn(cp, ok, 8, -1, None, 0.0, ok, None, 256, None),
        K._kv8_attn(cp, ok, 8, 1, None, math.nan, ok, None, 256, None),
        K._kv8_attn(cp, rows(type=K.F32), 8, 1, None, 0.0, rows(type=K.F32), None, 256, None),
        K._kv8_attn(cp, ok, 8, 1, None, 0.0, rows(type=K.F16), None, 256, None),
        K._kv8_attn(cp, ok, 8, 1, None, 0.0, None, None, 256, None),
        K._kv8_attn(cp, ok, 8, 1, None, 0.0, ok, 258, 256, None),
        K._kv8_mass(cp, ok, 8, 1, None, None, 0.0, 1.0, 256, None),
        K._kv8_mass(cp, ok, 8, 1, None, 256, 0.0, 1.5, 256, None),
        K._kv8_mass(cp, ok, 8, 1, None, 256, 0.0, math.nan, 256, None),
        K._kv8_evict(cp, None, 0, 0, 0, 256, 256, None),
        K._kv8_evict(cp, None, 8, 5, 4, 256, 256, None),
        K._kv8_evict(cp, None, 8, -1, 4, 256, 256, None),
        K._kv8_evict(cp, None, 1025, 0, 0, 256, 256, None),
        K._kv8_evict(cp, None, 8, 0, 0, None, 256, None),
        K._kv8_evict(cp, cp, 8, 0, 0, 256, 256, None),      # dst with the same seq_len
    ]
    assert bad == [K.CSA2_ERR_INVALID] * len(bad)
    other = base()
    other.seq_len = 512
    for field, value in [("batch", 3), ("kv_heads", 8), ("dim", 64), ("block", 32),
                         ("format", K.KV8_INT8), ("max_len", 64)]:
        d = K.Csa2Kv8Cache.from_buffer_copy(other)
        setattr(d, field, value)
        assert K._kv8_evict(cp, ctypes.byref(d), 100, 0, 0, 256, 256, None) == K.CSA2_ERR_INVALID
    c.mass = None
    assert K._kv8_mass(cp, ok, 8, 1, None, 256, 0.0, 1.0, 256, None) == K.CSA2_ERR_INVALID
    assert K._kv8_evict(cp, None, 8, 0, 0, 256, 256, None) == K.CSA2_ERR_INVALID
    # nothing to do
    assert K._kv8_append(cp, None, None, 0, None, None, 256, None) == K.CSA2_OK
    assert K._kv8_attn(cp, None, 8, 0, None, 0.0, None, None, 256, None) == K.CSA2_OK


def test_binding_refuses_what_does_not_fit():
    c = K.Cache8(2, 4, 64, 128, block=32, mass=True, device="cpu")
    ws = c.workspace(4, 8)
    k = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16)
    lse = torch.zeros(2, 3, 8)
    kept = torch.zeros(2, 4, 16, dtype=torch.int32)
    i2 = torch.zeros(2, dtype=torch.int32)
    calls = [
        lambda: K.kv8_append(c, k.double(), k, ws),
        lambda: K.kv8_append(c, k[:1], k[:1], ws),
        lambda: K.kv8_append(c, k, k[:, :2], ws),
        lambda: K.kv8_append(c, k, k.half(), ws),
        lambda: K.kv8_append(c, k[..., :32], k[..., :32], ws),
        lambda: K.kv8_append(c, k.transpose(2, 3).contiguous().transpose(2, 3), k, ws),
        lambda: K.kv8_append(c, torch.zeros(2, 3, 4, 65, dtype=torch.bfloat16)[..., 1:], k, ws),
        lambda: K.kv8_append(c, k, k, ws, new_len=i2.long()),
        lambda: K.kv8_append(c, k, k, ws, start=i2[:1]),
        lambda: K.kv8_append(c, k, k, ws[:256]),
        lambda: K.kv8_attn(c, q.float(), q.float(), ws),
        lambda: K.kv8_attn(c, q[:, :, :6], q[:, :, :6].clone(), ws),
        lambda: K.kv8_attn(c, q, q[:, :2], ws),
        lambda: K.kv8_attn(c, q, q.clone(), ws, lse=lse.half()),
        lambda: K.kv8_attn(c, q, q.clone(), ws, q_len=torch.zeros(3, dtype=torch.int32)),
        lambda: K.kv8_mass(c, q, None, ws),
        lambda: K.kv8_mass(c, q, lse[:, :2], ws),
        lambda: K.kv8_evict(c, 17, 0, 0, kept, ws),
        lambda: K.kv8_evict(c, 16, 0, 0, None, ws),
        lambda: K.Cache8(2, 4, 64, 100, block=32, device="cpu"),
        lambda: K.Cache8(2, 4, 64, 128, block=32, page_size=32, num_pages=9, device="cpu"),
        lambda: K.Cache8(2, 4, 64, 128, block=32, device="cpu", tensors={"seq_len": i2}),
        lambda: K.Cache8(2, 4, 100, 128, block=32, device="cpu").workspace(1, 4),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(K.Csa2Error):
            call()
            pytest.fail(f"call {i} was not refused")
    no_mass = K.Cache8(2, 4, 64, 128, block=32, device="cpu")
    for call in (lambda: K.kv8_mass(no_mass, q, lse, ws), lambda: K.kv8_evict(no_mass, 16, 0, 0, kept, ws)):
        with pytest.raises(K.Csa2Error):
            call()
