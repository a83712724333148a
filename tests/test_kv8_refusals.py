"""Refusals of the 8-bit K/V cache's calls, before any launch: arguments whose
memory overlaps where the kernels read and write it without an order, and
numbers that the kernels cannot work with."""
import ctypes
import math

import pytest
import torch

import fp4_kv_cache_rope_gb300 as K


def contiguous(at, seq_len):
    """A contiguous cache of 2 x 4 x 1024 rows, its arrays one after another from
    `at` on: 1 MiB of K, of V, 2 x 512 bytes of scales, 32 KiB of weights."""
    mib = 1 << 20
    return K.Csa2Kv8Cache(2, 4, 128, 64, 0, 0, 1024, 0, K.KV8_E4M3, at, at + mib, at + 2 * mib,
                          at + 2 * mib + 512, at + 2 * mib + 1024, None, seq_len)


def evict(a, b):
    return K._kv8_evict(ctypes.byref(a), ctypes.byref(b), 100, 0, 0, 256, 256, None)


def test_evict_refuses_another_cache_over_its_own_storage():
    base = 1 << 30
    size = (2 << 20) + 1024 + 2 * 4 * 1024 * 4
    src = contiguous(base, 1 << 20)
    for at in (base, base + 256, base - 256, base + (1 << 20), base - (1 << 20), base + (2 << 20),
               base + size - 16, base - size + 16):
        assert evict(src, contiguous(at, 1 << 21)) == K.CSA2_ERR_INVALID, at
    # one array of one over another of the other
    for field, value in [("k_codes", src.v_codes), ("v_codes", src.k_codes + (1 << 20) - 16),
                         ("k_scales", src.mass), ("v_scales", src.k_scales), ("mass", src.v_codes + 64),
                         ("mass", src.v_scales - 4)]:
        d = contiguous(1 << 33, 1 << 21)
        setattr(d, field, value)
        assert evict(src, d) == K.CSA2_ERR_INVALID, field
    # a contiguous cache inside a paged one's pool, either way round
    pool = K.Csa2Kv8Cache.from_buffer_copy(src)
    pool.page_size, pool.max_pages_per_seq, pool.num_pages, pool.page_table = 64, 16, 32, 512
    inside = contiguous(1 << 33, 1 << 21)
    inside.k_codes = pool.k_codes + (1 << 20) - 128
    assert evict(pool, inside) == K.CSA2_ERR_INVALID
    assert evict(inside, pool) == K.CSA2_ERR_INVALID
    # seq_len apart by one of two entries
    for off in (-4, 0, 4):
        assert evict(src, contiguous(1 << 33, (1 << 20) + off)) == K.CSA2_ERR_INVALID, off


def test_attention_refuses_outputs_whose_rows_overlap():
    """q may repeat rows; out may not."""
    c = contiguous(1 << 30, 1 << 20)
    c.dim, B, T, H = 64, 2, 3, 8
    D = c.dim
    q = K.Csa2Rows(1 << 31, 0, 0, 0, K.BF16)

    def attn(sb, st, sh, T=T, H=H):
        out = K.Csa2Rows(1 << 32, sb, st, sh, K.BF16)
        return K._kv8_attn(ctypes.byref(c), ctypes.byref(q), H, T, None, 0.0, ctypes.byref(out), None, 256,
                           None)

    for strides in [(0, H * D, D), (T * H * D, 0, D), (T * H * D, H * D, 0), (T * H * D, H * D, 8),
                    (T * H * D, D, D), (H * D, H * D, D), (T * H * D - 8, H * D, D),
                    (T * H * D, H * D, -8), (D, 2 * D, 6 * D + 8 - D), (1 << 62, H * D, D),
                    (-(1 << 63), H * D, D), (0, 0, 0)]:
        assert attn(*strides) == K.CSA2_ERR_INVALID, strides


def test_softmax_scales_out_of_range():
    c = contiguous(1 << 30, 1 << 20)
    r = K.Csa2Rows(1 << 31, 8 * 128, 8 * 128, 128, K.BF16)
    for scale in (math.inf, math.nan, 3.0e38, 2.0 ** 101, 1e-40, 2.0 ** -101):
        assert K._kv8_attn(ctypes.byref(c), ctypes.byref(r), 8, 1, None, scale, ctypes.byref(r), None, 256,
                           None) == K.CSA2_ERR_INVALID, scale
        assert K._kv8_mass(ctypes.byref(c), ctypes.byref(r), 8, 1, None, 256, scale, 1.0, 256,
                           None) == K.CSA2_ERR_INVALID, scale
    # no query rows: nothing is launched for a scale that is taken
    for scale in (0.0, -1.0, 2.0 ** -100, 0.125, 2.0 ** 100):
        assert K._kv8_attn(ctypes.byref(c), None, 8, 0, None, scale, None, None, 256, None) == K.CSA2_OK


@pytest.mark.parametrize("missing", ["k_codes", "v_codes", "k_scales", "v_scales", "seq_len"])
def test_a_cache_over_given_storage_names_what_is_missing(missing):
    c = K.Cache8(2, 4, 64, 128, block=32, mass=True, device="cpu")
    given = {n: getattr(c, n) for n in ("k_codes", "v_codes", "k_scales", "v_scales", "mass", "seq_len")}
    assert K.Cache8(2, 4, 64, 128, block=32, tensors=given).mass is c.mass
    for gone in ({n: t for n, t in given.items() if n != missing}, given | {missing: None}):
        with pytest.raises(K.Csa2Error, match=missing):
            K.Cache8(2, 4, 64, 128, block=32, tensors=gone)
