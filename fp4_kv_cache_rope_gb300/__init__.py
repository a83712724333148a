"""Python binding of libcsa2 (CSA2 sparse attention over an FP4 global KV cache).

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libcsa2.so`` behind the C ABI declared in ``include/csa2.h``.  Tensors are
passed as ``torch.Tensor`` (device memory) and the current torch CUDA stream
is used unless a stream is given.  There is no CPU fallback: importing this
module fails loudly when the library has not been built.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcsa2.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
    )

_lib = ctypes.CDLL(LIB_PATH)

CSA2_OK, CSA2_ERR_INVALID, CSA2_ERR_CUDA, CSA2_ERR_UNSUPPORTED, CSA2_ERR_TIMEOUT, CSA2_ERR_DEVICE = range(6)
DEV_BAD_INDEX, DEV_BAD_PAGE, DEV_OVERFLOW, DEV_TIMEOUT, DEV_BAD_POOL, DEV_BAD_ALIGN = (
    0x1, 0x2, 0x4, 0x8, 0x10, 0x20)
DEV_NONFINITE, DEV_BAD_TREE = 0x40, 0x80
MAX_TOPK = 2048
POOL_BLOCKS = 2048
BLOCK = 8

_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64


class Csa2Cache(ctypes.Structure):
    _fields_ = [
        ("batch", _i32), ("dim", _i32), ("rope_dim", _i32), ("idx_dim", _i32),
        ("page_size", _i32), ("max_pages_per_seq", _i32), ("max_len", _i32), ("num_pages", _i32),
        ("kv_codes", _p), ("code_stride", _i64),
        ("kv_scales", _p), ("scale_stride", _i64),
        ("idx_k", _p), ("idxk_stride", _i64),
        ("page_table", _p), ("seq_len", _p),
        ("rope_cos", _p), ("rope_sin", _p),
        ("idx_format", _i32), ("idx_scales", _p), ("idx_scale_stride", _i64),
    ]


IDX_E4M3, IDX_MXFP4 = 0, 1


class Csa2Kv8Cache(ctypes.Structure):
    _fields_ = [
        ("batch", _i32), ("kv_heads", _i32), ("dim", _i32), ("block", _i32), ("page_size", _i32),
        ("max_pages_per_seq", _i32), ("max_len", _i32), ("num_pages", _i32), ("format", _i32),
        ("k_codes", _p), ("v_codes", _p), ("k_scales", _p), ("v_scales", _p), ("mass", _p),
        ("page_table", _p), ("seq_len", _p),
    ]


class Csa2Rows(ctypes.Structure):
    _fields_ = [("data", _p), ("stride_b", _i64), ("stride_t", _i64), ("stride_h", _i64),
                ("type", _i32)]


class Csa2Rope(ctypes.Structure):
    _fields_ = [("cos", _p), ("sin", _p), ("positions", _i32), ("dim", _i32), ("first", _i32),
                ("style", _i32)]


class Csa2Scores(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("window", _i32), ("sink", _i32), ("slopes", _p),
                ("prefix", _p)]


KV8_E4M3, KV8_INT8 = 0, 1
ROPE_HALVES, ROPE_PAIRS = 0, 1
KV8_MAX_TREE = 256
BF16, F16, F32 = 0, 1, 2


def _sig(name, args, res=_i32):
    f = getattr(_lib, name)
    f.argtypes = args
    f.restype = res
    return f


_CP = ctypes.POINTER(Csa2Cache)
_workspace_size = _sig("csa2_workspace_size", [_CP, _i32, _i32], ctypes.c_size_t)
_entry_bytes = _sig("csa2_entry_bytes", [_i32], _i64)
_fp8_quant = _sig("csa2_fp8_quant", [_p, _i64, _p, _p])
_quant_append = _sig("csa2_quant_append", [_CP, _p, _p, _i32, _p, _p])
_quant_append_pairs = _sig("csa2_quant_append_pairs", [_CP, _p, _p, _p, _i32, _p, _p])
_index_full = _sig("csa2_index_full", [_CP, _p, _p, _i32, _i32, _p, _p, _i32, _i32,
                                       _p, _p, _p, _p, _p, _p])
_index_full_noalloc = _sig("csa2_index_full_noalloc", [_CP, _p, _p, _i32, _i32, _p, _p, _i32,
                                                       _i32, _p, _p, _p, _p, _p, _p])
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024
_index_reindex = _sig("csa2_index_reindex", [_CP, _p, _p, _i32, _i32, _p, _p, _p, _p, _i32,
                                             _i32, _p, _p, _p, _p])
_attn_decode = _sig("csa2_attn_decode", [_CP, _p, _i32, _p, _p, _i32, _p, _p, _i32,
                                         ctypes.c_float, _p, _p, _p])
_attn_decode_layers = _sig("csa2_attn_decode_layers", [_CP, _i32, _p, _i32, _p, _p, _i32, _p, _p,
                                                       _i32, ctypes.c_float, _p, _p, _p])
_attn_prefill = _sig("csa2_attn_prefill", [_CP, _p, _i32, _i32, _p, _p, _p, _i32, _p, _i32,
                                           ctypes.c_float, _p, _p, _p])
_get_status = _sig("csa2_get_status", [_p, ctypes.POINTER(ctypes.c_uint32), _p])
_reset_status = _sig("csa2_reset_status", [_p, _p])
_status_string = _sig("csa2_status_string", [_i32], ctypes.c_char_p)
_set_launch_events = _sig("csa2_set_launch_events", [_i32, _p, _p])
_set_wait_limit = _sig("csa2_set_wait_limit", [ctypes.c_uint64])
_C8P, _RP = ctypes.POINTER(Csa2Kv8Cache), ctypes.POINTER(Csa2Rows)
_kv8_workspace_size = _sig("csa2_kv8_workspace_size", [_C8P, _i32, _i32], ctypes.c_size_t)
_kv8_append = _sig("csa2_kv8_append", [_C8P, _RP, _RP, _i32, _p, _p, _p, _p])
_kv8_attn = _sig("csa2_kv8_attn", [_C8P, _RP, _i32, _i32, _p, ctypes.c_float, _RP, _p, _p, _p])
_kv8_mass = _sig("csa2_kv8_mass", [_C8P, _RP, _i32, _i32, _p, _p, ctypes.c_float, ctypes.c_float,
                                   _p, _p])
_kv8_evict = _sig("csa2_kv8_evict", [_C8P, _C8P, _i32, _i32, _i32, _p, _p, _p])
_OP, _SP = ctypes.POINTER(Csa2Rope), ctypes.POINTER(Csa2Scores)
_kv8_rope = _sig("csa2_kv8_rope", [_C8P, _OP, _RP, _i32, _RP, _RP, _RP, _i32, _p, _p, _p, _p, _p])
_kv8_append_rope = _sig("csa2_kv8_append_rope", [_C8P, _OP, _RP, _RP, _i32, _RP, _i32, _RP, _p, _p,
                                                 _p, _p, _p])
_kv8_append_path = _sig("csa2_kv8_append_path", [_C8P, _RP, _RP, _i32, _p, _i32, _p, _p, _p, _p])
_kv8_attn_scored = _sig("csa2_kv8_attn_scored", [_C8P, _RP, _i32, _i32, _p, ctypes.c_float, _SP, _RP,
                                                 _p, _p, _p])
_kv8_tree_workspace_size = _sig("csa2_kv8_tree_workspace_size", [_C8P, _i32, _i32], ctypes.c_size_t)
_kv8_attn_tree = _sig("csa2_kv8_attn_tree", [_C8P, _RP, _i32, _RP, _RP, _p, _i32, _p, ctypes.c_float,
                                             _SP, _RP, _p, _p, _p])
KERNEL_QUANT, KERNEL_INDEXER, KERNEL_SELECT, KERNEL_ATTENTION = 0, 1, 2, 3

EXPORTED = ["csa2_workspace_size", "csa2_entry_bytes", "csa2_fp8_quant", "csa2_quant_append",
            "csa2_index_full", "csa2_index_reindex", "csa2_attn_decode", "csa2_attn_prefill",
            "csa2_get_status", "csa2_reset_status", "csa2_status_string",
            "csa2_set_launch_events", "csa2_index_full_noalloc", "csa2_quant_append_pairs",
            "csa2_set_wait_limit", "csa2_attn_decode_layers", "csa2_kv8_workspace_size",
            "csa2_kv8_append", "csa2_kv8_attn", "csa2_kv8_mass", "csa2_kv8_evict", "csa2_kv8_rope",
            "csa2_kv8_append_rope", "csa2_kv8_append_path", "csa2_kv8_attn_scored",
            "csa2_kv8_tree_workspace_size", "csa2_kv8_attn_tree"]


class Csa2Error(RuntimeError):
    pass


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code, what):
    if code != CSA2_OK:
        raise Csa2Error(f"{what}: {status_string(code)} ({code})")
    return code


def status_string(code: int) -> str:
    return _status_string(int(code)).decode()


def entry_bytes(dim: int) -> int:
    return int(_entry_bytes(dim))


def workspace_size(cache: "Cache | Csa2Cache", max_rows: int, heads: int) -> int:
    c = cache.struct if isinstance(cache, Cache) else cache
    return int(_workspace_size(ctypes.byref(c), max_rows, heads))


def fp8_quant(x, out, stream=None):
    """fp32 -> E4M3 codes (RNE, saturating at 448, sign copied)."""
    _check(_fp8_quant(_ptr(x), x.numel(), _ptr(out), _stream(stream)), "csa2_fp8_quant")


def quant_append(cache, kv, idx_k_in, T, ws, stream=None):
    _check(_quant_append(ctypes.byref(cache.struct), _ptr(kv), _ptr(idx_k_in), T, _ptr(ws),
                         _stream(stream)), "csa2_quant_append")


def quant_append_pairs(cache, kv, z, idx_k_in, T, ws, stream=None):
    """Append T entries per sequence, each compressed from 2 source rows (m = 2)."""
    _check(_quant_append_pairs(ctypes.byref(cache.struct), _ptr(kv), _ptr(z), _ptr(idx_k_in), T,
                               _ptr(ws), _stream(stream)), "csa2_quant_append_pairs")


def index_full(cache, q_idx, w, hi, tq, q_pos, batch_ids, n_batch, k, out_idx, out_cnt,
               pool_blocks, pool_cnt, ws, stream=None):
    _check(_index_full(ctypes.byref(cache.struct), _ptr(q_idx), _ptr(w), hi, tq, _ptr(q_pos),
                       _ptr(batch_ids), n_batch, k, _ptr(out_idx), _ptr(out_cnt),
                       _ptr(pool_blocks), _ptr(pool_cnt), _ptr(ws), _stream(stream)),
           "csa2_index_full")


def index_full_noalloc(cache, q_idx, w, hi, tq, q_pos, batch_ids, n_batch, k, out_idx, out_cnt,
                       pool_blocks, pool_cnt, status, stream=None):
    """index_full for callers that may not allocate device memory: the scratch
    is a fixed array inside the library; ``status`` (a 4-byte device tensor or
    None) receives the call's device status word."""
    _check(_index_full_noalloc(ctypes.byref(cache.struct), _ptr(q_idx), _ptr(w), hi, tq,
                               _ptr(q_pos), _ptr(batch_ids), n_batch, k, _ptr(out_idx),
                               _ptr(out_cnt), _ptr(pool_blocks), _ptr(pool_cnt), _ptr(status),
                               _stream(stream)), "csa2_index_full_noalloc")


def index_reindex(cache, q_idx, w, hi, tq, q_pos, pool_blocks, pool_cnt, batch_ids, n_batch, k,
                  out_idx, out_cnt, ws, stream=None):
    _check(_index_reindex(ctypes.byref(cache.struct), _ptr(q_idx), _ptr(w), hi, tq, _ptr(q_pos),
                          _ptr(pool_blocks), _ptr(pool_cnt), _ptr(batch_ids), n_batch, k,
                          _ptr(out_idx), _ptr(out_cnt), _ptr(ws), _stream(stream)),
           "csa2_index_reindex")


def attn_decode(cache, q, heads, idx, cnt, kcap, swa, swa_cnt, window, softmax_scale, out, ws,
                stream=None):
    _check(_attn_decode(ctypes.byref(cache.struct), _ptr(q), heads, _ptr(idx), _ptr(cnt), kcap,
                        _ptr(swa), _ptr(swa_cnt), window, float(softmax_scale), _ptr(out),
                        _ptr(ws), _stream(stream)), "csa2_attn_decode")


MAX_ATTN_LAYERS = 8


def attn_decode_layers(cache, qs, heads, idx, cnt, kcap, swas, swa_cnt, window, softmax_scale,
                       outs, ws, stream=None):
    """csa2_attn_decode_layers: qs, swas, outs are sequences of one tensor per
    layer (the host pointer arrays are built here)."""
    n = len(qs)
    if not 1 <= n <= MAX_ATTN_LAYERS or len(outs) != n or len(swas) != n:
        raise Csa2Error("csa2_attn_decode_layers: 1..%d layers, one q, swa and out each"
                        % MAX_ATTN_LAYERS)
    arr = ctypes.c_void_p * n
    qa, sa, oa = arr(*[_ptr(x) for x in qs]), arr(*[_ptr(x) for x in swas]), arr(*[_ptr(x) for x in outs])
    _check(_attn_decode_layers(ctypes.byref(cache.struct), n, ctypes.cast(qa, ctypes.c_void_p),
                               heads, _ptr(idx), _ptr(cnt), kcap, ctypes.cast(sa, ctypes.c_void_p),
                               _ptr(swa_cnt), window, float(softmax_scale),
                               ctypes.cast(oa, ctypes.c_void_p), _ptr(ws), _stream(stream)),
           "csa2_attn_decode_layers")


def attn_prefill(cache, q, heads, tq, q_pos, idx, cnt, kcap, swa, window, softmax_scale, out, ws,
                 stream=None):
    _check(_attn_prefill(ctypes.byref(cache.struct), _ptr(q), heads, tq, _ptr(q_pos), _ptr(idx),
                         _ptr(cnt), kcap, _ptr(swa), window, float(softmax_scale), _ptr(out),
                         _ptr(ws), _stream(stream)), "csa2_attn_prefill")


def set_launch_events(family, begin=None, end=None):
    """Bracket the family's main kernel with torch.cuda.Event records (or stop)."""
    b = begin.cuda_event if begin is not None else None
    e = end.cuda_event if end is not None else None
    _check(_set_launch_events(family, b, e), "csa2_set_launch_events")


def set_wait_limit(ns: int = 0):
    """Limit of the kernels' bounded on-chip waits in ns (0 = the 2 s default)."""
    _check(_set_wait_limit(int(ns)), "csa2_set_wait_limit")


def get_status(ws, stream=None) -> int:
    v = ctypes.c_uint32(0)
    code = _get_status(_ptr(ws), ctypes.byref(v), _stream(stream))
    if code not in (CSA2_OK, CSA2_ERR_DEVICE):
        _check(code, "csa2_get_status")
    return int(v.value)


def reset_status(ws, stream=None):
    _check(_reset_status(_ptr(ws), _stream(stream)), "csa2_reset_status")


class Cache:
    """Device storage of one shared global cache plus its C description.

    Row strides are the smallest multiples of 16 bytes that hold a row:
    codes D/2, scales round_up(D/16, 16), indexer key di (E4M3).  With
    ``idx_format=IDX_MXFP4`` (di = 128) the indexer key is 64 code bytes per
    row and a separate array holds its 4 E8M0 scale bytes per row.
    """

    def __init__(self, batch, dim, rope_dim, idx_dim, max_len, rope_cos, rope_sin,
                 page_size=0, page_table=None, num_pages=0, device="cuda",
                 idx_format=IDX_E4M3):
        import torch
        self.batch, self.dim, self.rope_dim, self.idx_dim = batch, dim, rope_dim, idx_dim
        self.max_len, self.page_size = max_len, page_size
        self.idx_format = idx_format
        self.code_stride = (dim // 2 + 15) // 16 * 16
        self.scale_stride = (dim // 16 + 15) // 16 * 16
        if idx_format == IDX_MXFP4:
            self.idxk_stride = (idx_dim // 2 + 31) // 32 * 32
            self.idx_scale_stride = idx_dim // 32
        else:
            self.idxk_stride = (idx_dim + 15) // 16 * 16
            self.idx_scale_stride = 0
        if page_size:
            self.num_pages = num_pages
            rows = num_pages * page_size
            self.page_table = page_table.to(device=device, dtype=torch.int32).contiguous()
            self.max_pages = self.page_table.shape[1]
        else:
            self.num_pages = 0
            rows = batch * max_len
            self.page_table = None
            self.max_pages = 0
        self.rows = rows
        self.codes = torch.zeros((rows, self.code_stride), dtype=torch.uint8, device=device)
        self.scales = torch.zeros((rows, self.scale_stride), dtype=torch.uint8, device=device)
        self.idx_k = torch.zeros((rows, self.idxk_stride), dtype=torch.uint8, device=device)
        self.idx_scales = (torch.zeros((rows, self.idx_scale_stride), dtype=torch.uint8,
                                       device=device) if idx_format == IDX_MXFP4 else None)
        self.seq_len = torch.zeros(batch, dtype=torch.int32, device=device)
        self.rope_cos = rope_cos.to(device=device, dtype=torch.float32).contiguous()
        self.rope_sin = rope_sin.to(device=device, dtype=torch.float32).contiguous()
        self.struct = Csa2Cache(
            batch, dim, rope_dim, idx_dim, page_size, self.max_pages, max_len, self.num_pages,
            self.codes.data_ptr(), self.code_stride, self.scales.data_ptr(), self.scale_stride,
            self.idx_k.data_ptr(), self.idxk_stride,
            self.page_table.data_ptr() if self.page_table is not None else None,
            self.seq_len.data_ptr(), self.rope_cos.data_ptr(), self.rope_sin.data_ptr(),
            idx_format, self.idx_scales.data_ptr() if self.idx_scales is not None else None,
            self.idx_scale_stride)

    def physical_row(self, b, t):
        """Host mirror of the row mapping (for reading rows back in tests)."""
        if not self.page_size:
            return b * self.max_len + t
        pt = self.page_table_host()
        return int(pt[b, t // self.page_size]) * self.page_size + t % self.page_size

    def page_table_host(self):
        if not hasattr(self, "_pt_host"):
            self._pt_host = self.page_table.cpu().numpy()
        return self._pt_host

    def workspace(self, max_rows, heads):
        import torch
        n = workspace_size(self, max_rows, heads)
        if n == 0:
            raise Csa2Error("invalid cache description")
        ws = torch.zeros(n, dtype=torch.uint8, device=self.codes.device)
        return ws


# ------------------------------------------------------- the 8-bit K/V cache
def kv8_workspace_size(cache: "Cache8 | Csa2Kv8Cache", T: int, heads: int) -> int:
    c = cache.struct if isinstance(cache, Cache8) else cache
    return int(_kv8_workspace_size(ctypes.byref(c), T, heads))


def kv8_tree_workspace_size(cache: "Cache8 | Csa2Kv8Cache", T: int, heads: int) -> int:
    c = cache.struct if isinstance(cache, Cache8) else cache
    return int(_kv8_tree_workspace_size(ctypes.byref(c), T, heads))


class Cache8:
    """Device storage of a K/V cache of grouped heads in 8 bits plus its C
    description (csa2_kv8_cache): codes with one power-of-two scale for each
    block of rows and head.

    ``tensors`` gives existing storage instead of new: a dict of k_codes and
    v_codes (uint8 [pages, kv_heads, page rows, dim]), k_scales and v_scales
    (fp32 [pages, kv_heads, page rows / block]), seq_len (int32 [batch]) and,
    where weights are accumulated, mass (fp32 [pages, kv_heads, page rows]).
    pages and page rows are num_pages and page_size, or, contiguous
    (page_size 0), batch and max_len.
    """

    def __init__(self, batch, kv_heads, dim, max_len, block=64, page_size=0, page_table=None,
                 num_pages=0, fmt=KV8_E4M3, mass=False, device="cuda", tensors=None):
        import torch
        self.batch, self.kv_heads, self.dim, self.max_len = batch, kv_heads, dim, max_len
        self.block, self.page_size, self.fmt = block, page_size, fmt
        self.int32, self.float32, self.needs = torch.int32, torch.float32, {}
        self.kinds = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}
        self.cuda = torch.cuda, torch._C._cuda_getCurrentRawStream
        pages, rows = (num_pages, page_size) if page_size else (batch, max_len)
        if page_size and page_table is None:
            raise Csa2Error("Cache8: a paged cache needs a page table")
        if not page_size and page_table is not None:
            raise Csa2Error("Cache8: a contiguous cache (page_size 0) has no page table")
        if min(batch, kv_heads, dim, max_len, block, pages, rows) < 1 or rows % block:
            raise Csa2Error("invalid cache description")
        shapes = {"k_codes": (torch.uint8, (pages, kv_heads, rows, dim)),
                  "v_codes": (torch.uint8, (pages, kv_heads, rows, dim)),
                  "k_scales": (torch.float32, (pages, kv_heads, rows // block)),
                  "v_scales": (torch.float32, (pages, kv_heads, rows // block)),
                  "mass": (torch.float32, (pages, kv_heads, rows)),
                  "seq_len": (torch.int32, (batch,))}
        if tensors is None:
            tensors = {n: torch.zeros(shape, dtype=dt, device=device)
                       for n, (dt, shape) in shapes.items() if n != "mass" or mass}
        if tensors.get("seq_len") is None:
            raise Csa2Error("Cache8: the given storage lacks seq_len")
        device = tensors["seq_len"].device
        for n, (dt, shape) in shapes.items():
            t = tensors.get(n)
            if t is None and n == "mass":
                continue
            if t is None or t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous() \
                    or t.device != device:
                raise Csa2Error(f"Cache8: {n} must be a contiguous {dt} tensor of shape {shape} "
                                f"on {device}")
        for n in shapes:
            setattr(self, n, tensors.get(n))
        self.device, self.num_pages = device, num_pages if page_size else 0
        self.index = device.index if device.type == "cuda" else None
        if page_size:
            self.page_table = page_table.to(device=device, dtype=torch.int32).contiguous()
            if self.page_table.dim() != 2 or self.page_table.shape[0] != batch:
                raise Csa2Error("Cache8: the page table is [batch, pages per sequence]")
        else:
            self.page_table = None
        self.struct = Csa2Kv8Cache(
            batch, kv_heads, dim, block, page_size,
            self.page_table.shape[1] if page_size else 0, max_len, self.num_pages, fmt,
            _ptr(self.k_codes), _ptr(self.v_codes), _ptr(self.k_scales), _ptr(self.v_scales),
            _ptr(self.mass), _ptr(self.page_table), _ptr(self.seq_len))

    def workspace(self, T, heads):
        """Workspace for calls of at most T query rows per sequence and `heads` heads."""
        import torch
        n = kv8_workspace_size(self, T, heads)
        if n == 0:
            raise Csa2Error("invalid cache description")
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    def tree_workspace(self, T, heads):
        """Workspace for kv8_attn_tree with at most T drafted tokens per sequence and `heads`
        heads, and for the other calls too."""
        import torch
        n = kv8_tree_workspace_size(self, T, heads)
        if n == 0:
            raise Csa2Error("invalid cache description, or more drafted tokens than KV8_MAX_TREE")
        return torch.zeros(n, dtype=torch.uint8, device=self.device)


def _int32(name, x):
    """x, which a C structure would cut to 32 bits."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise Csa2Error(f"{name}: {x} is not a 32-bit number")
    return x


class Rope:
    """Cosines and sines [positions, dim / 2] of the position rotation of `dim` channels
    from channel `first` on; pair j is the channels first + j and first + dim / 2 + j
    (ROPE_HALVES) or first + 2 j and first + 2 j + 1 (ROPE_PAIRS).  Kept as fp32 on
    `device` (default: where `cos` is)."""

    def __init__(self, cos, sin, first=0, style=ROPE_HALVES, device=None):
        import torch
        device = torch.device(cos.device if device is None else device)
        if cos.dim() != 2 or cos.shape != sin.shape or cos.shape[0] < 1:
            raise Csa2Error("Rope: cos and sin are [positions, dim / 2]")
        self.cos = cos.to(device=device, dtype=torch.float32).contiguous()
        self.sin = sin.to(device=device, dtype=torch.float32).contiguous()
        if (self.cos.data_ptr() | self.sin.data_ptr()) & 15:
            self.cos, self.sin = self.cos.clone(), self.sin.clone()
        self.device = self.cos.device
        self.struct = Csa2Rope(_ptr(self.cos), _ptr(self.sin), _int32("Rope: positions", cos.shape[0]),
                               _int32("Rope: dim", 2 * cos.shape[1]), _int32("Rope: first", first),
                               _int32("Rope: style", style))


class Scores:
    """What a model does to its attention's scores, for a query at position p and a row
    at position j: x = cap * tanh(x / cap) (cap > 0), x = x - slopes[head] * |p - j|
    (slopes: fp32 [heads]); and which rows a query sees: j <= p or j < prefix[b]
    (prefix: int32 [batch]), and, with window > 0, j > p - window or j < sink."""

    def __init__(self, cap=0.0, window=0, sink=0, slopes=None, prefix=None):
        import torch
        for name, x, dt in (("slopes", slopes, torch.float32), ("prefix", prefix, torch.int32)):
            if x is not None and (x.dtype != dt or x.dim() != 1 or not x.is_contiguous()):
                raise Csa2Error(f"Scores: {name} is a contiguous {dt} vector")
        # (a smaller cap could become 0, which is none, in fp32)
        if cap != 0 and not 2.0 ** -10 <= cap <= 2.0 ** 20:
            raise Csa2Error(f"Scores: cap {cap}; it takes 0 for none, or 2^-10 .. 2^20")
        self.slopes, self.prefix = slopes, prefix
        self.struct = Csa2Scores(cap, _int32("Scores: window", window), _int32("Scores: sink", sink),
                                 _ptr(slopes), _ptr(prefix))


# The calls below are made once per layer and token, so their checks are kept to
# a few attribute reads, and a refusal's text is put together only when it is raised.
def _kv8_rows(cache, x, name, heads=None, wide=False):
    """(struct, T) of a [batch, T, heads, dim] tensor whose last dimension is contiguous."""
    kind, shape = cache.kinds.get(x.dtype), x.shape
    if kind is None or (kind == F32 and not wide):
        raise Csa2Error(f"{name}: {x.dtype}; it takes bfloat16, float16"
                        + (" or float32" if wide else ""))
    if len(shape) != 4 or shape[0] != cache.batch or shape[3] != cache.dim or (
            heads is not None and shape[2] != heads):
        raise Csa2Error(f"{name}: shape {tuple(shape)}; it takes [batch {cache.batch}, T, "
                        f"{'heads' if heads is None else heads}, dim {cache.dim}]")
    if x.device != cache.device:
        raise Csa2Error(f"{name}: on {x.device}, the cache on {cache.device}")
    T = shape[1]
    if T == 0 or shape[2] == 0:
        return Csa2Rows(None, 0, 0, 0, kind), T
    sb, st, sh, sd = x.stride()
    at, part = x.data_ptr(), 3 if kind == F32 else 7   # strides in steps of 16 bytes
    if sd != 1 or at & 15 or (sb | st | sh) & part:
        # the stride of a dimension of one element is not used
        sb, st, sh = (v if n > 1 else 0 for v, n in zip((sb, st, sh), shape))
        if sd != 1 or at & 15 or (sb | st | sh) & part:
            raise Csa2Error(f"{name}: the last dimension must be contiguous and every row start "
                            "on a multiple of 16 bytes")
    return Csa2Rows(at, sb, st, sh, kind), T


def _kv8_arg(cache, x, name, dtype, shape):
    """Pointer of an optional contiguous tensor of this type and shape on the cache's device."""
    if x is None:
        return None
    if x.dtype != getattr(cache, dtype) or x.shape != shape or not x.is_contiguous() \
            or x.device != cache.device:
        raise Csa2Error(f"{name}: it takes a contiguous {dtype} tensor of shape {shape} on "
                        f"{cache.device}")
    return x.data_ptr()


def _kv8_ws(cache, ws, T=0, heads=None, tree=False):
    heads = cache.kv_heads if heads is None else heads
    need = cache.needs.get((T, heads, tree))
    if need is None:
        need = (kv8_tree_workspace_size if tree else kv8_workspace_size)(cache, T, heads)
        if need == 0:
            raise Csa2Error(f"the cache does not take a call of {T} query rows and {heads} heads")
        if len(cache.needs) > 256:
            cache.needs.clear()
        cache.needs[T, heads, tree] = need
    if ws.device != cache.device or ws.numel() * ws.element_size() < need or not ws.is_contiguous():
        raise Csa2Error(f"workspace: it takes {need} contiguous bytes on {cache.device}")
    return ws.data_ptr()


def _kv8_run(cache, what, call, stream, *args):
    """call(*args, stream) with the cache's device current."""
    if cache.index is None:
        raise Csa2Error("the cache is not on a CUDA device")
    cuda, raw = cache.cuda
    if cuda.current_device() != cache.index:
        with cuda.device(cache.index):
            return _kv8_run(cache, what, call, stream, *args)
    if stream is None:
        stream = raw(cache.index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    code = call(*args, stream)
    if code:
        _check(code, what)


def kv8_append(cache, k, v, ws, new_len=None, start=None, stream=None):
    """Quantise and append the rows k, v [batch, T, kv_heads, dim] (bf16, f16 or
    fp32): new_len[b] of them (int32 [batch], default T) from position start[b]
    on (int32 [batch], default seq_len)."""
    rk, T = _kv8_rows(cache, k, "k", cache.kv_heads, True)
    rv, Tv = _kv8_rows(cache, v, "v", cache.kv_heads, True)
    if T != Tv or rk.type != rv.type:
        raise Csa2Error("k and v: one T and one type")
    nl = _kv8_arg(cache, new_len, "new_len", "int32", (cache.batch,))
    sp = _kv8_arg(cache, start, "start", "int32", (cache.batch,))
    _kv8_run(cache, "csa2_kv8_append", _kv8_append, stream, ctypes.byref(cache.struct),
             ctypes.byref(rk), ctypes.byref(rv), T, nl, sp, _kv8_ws(cache, ws))


def kv8_attn(cache, q, out, ws, lse=None, q_len=None, softmax_scale=0.0, stream=None):
    """Attention of the queries q [batch, T, heads, dim] (bf16 or f16) of each
    sequence's last q_len[b] rows (int32 [batch], default T) over the cache, into
    out (as q) and lse (fp32 [batch, T, heads], optional)."""
    rq, T = _kv8_rows(cache, q, "q")
    H = q.shape[2]
    ro, To = _kv8_rows(cache, out, "out", H)
    if To != T or ro.type != rq.type:
        raise Csa2Error("out: shape and type of q")
    ls = _kv8_arg(cache, lse, "lse", "float32", (cache.batch, T, H))
    ql = _kv8_arg(cache, q_len, "q_len", "int32", (cache.batch,))
    _kv8_run(cache, "csa2_kv8_attn", _kv8_attn, stream, ctypes.byref(cache.struct),
             ctypes.byref(rq), H, T, ql, softmax_scale, ctypes.byref(ro), ls,
             _kv8_ws(cache, ws, T, H))


def kv8_mass(cache, q, lse, ws, q_len=None, softmax_scale=0.0, decay=1.0, stream=None):
    """cache.mass = decay * cache.mass + the weight that each row got from the
    queries q, given the lse that kv8_attn returned for them.  Pages that two
    sequences share lose updates: weights need pages of their own."""
    rq, T = _kv8_rows(cache, q, "q")
    H = q.shape[2]
    if cache.mass is None or lse is None:
        raise Csa2Error("csa2_kv8_mass: the cache holds no mass, or no lse given")
    ls = _kv8_arg(cache, lse, "lse", "float32", (cache.batch, T, H))
    ql = _kv8_arg(cache, q_len, "q_len", "int32", (cache.batch,))
    _kv8_run(cache, "csa2_kv8_mass", _kv8_mass, stream, ctypes.byref(cache.struct),
             ctypes.byref(rq), H, T, ql, ls, softmax_scale, decay, _kv8_ws(cache, ws, T, H))


def kv8_evict(cache, keep, sink, recent, kept, ws, dst=None, stream=None):
    """Cut every sequence to at most `keep` rows: the first `sink`, the last
    `recent`, and the heaviest by cache.mass between them, in place or into the
    cache `dst`, which shares no storage with `cache` (two paged ones: no page).
    kept (int32 [batch, kv_heads, keep]): their former positions."""
    kp = _kv8_arg(cache, kept, "kept", "int32", (cache.batch, cache.kv_heads, keep))
    if kp is None or cache.mass is None:
        raise Csa2Error("csa2_kv8_evict: it takes `kept`, and a cache with mass")
    if dst is not None and dst.device != cache.device:
        raise Csa2Error(f"dst: on {dst.device}, the cache on {cache.device}")
    _kv8_run(cache, "csa2_kv8_evict", _kv8_evict, stream, ctypes.byref(cache.struct),
             None if dst is None else ctypes.byref(dst.struct), keep, sink, recent, kp,
             _kv8_ws(cache, ws))


def _kv8_alike(cache, x, name, heads, first, of, T, kind, wide=False):
    """(struct) of rows of x, which has the T and the type of `first`, the operand called `of`."""
    if x.dtype is first.dtype and x.shape == (cache.batch, T, heads, cache.dim) \
            and x.device == cache.device and T:
        sb, st, sh, sd = x.stride()
        at = x.data_ptr()
        if sd == 1 and not (at & 15 or (sb | st | sh) & (3 if kind == F32 else 7)):
            return Csa2Rows(at, sb, st, sh, kind)
    r, Tx = _kv8_rows(cache, x, name, heads, wide)
    if Tx != T or r.type != kind:
        raise Csa2Error(f"{name}: T and type of {of}")
    return r


def _kv8_table(cache, rope):
    if rope.device != cache.device:
        raise Csa2Error(f"rope: on {rope.device}, the cache on {cache.device}")
    r = rope.struct
    if r.dim % 16 or r.first % 8 or r.first < 0 or r.first + r.dim > cache.dim:
        raise Csa2Error(f"rope: {r.dim} channels from {r.first} on; it takes a multiple of 16 from a "
                        f"multiple of 8 on, within dim {cache.dim}")
    return ctypes.byref(r)


def _kv8_scores(cache, scores, H):
    if not isinstance(scores, Scores):
        raise Csa2Error("scores: it takes a Scores")
    if scores.slopes is not None:
        _kv8_arg(cache, scores.slopes, "slopes", "float32", (H,))
    if scores.prefix is not None:
        _kv8_arg(cache, scores.prefix, "prefix", "int32", (cache.batch,))
    return ctypes.byref(scores.struct)


def kv8_rope(cache, q, q_out, rope, ws, k=None, k_out=None, q_len=None, pos=None, parent=None,
             stream=None):
    """Rotate the first q_len[b] rows (int32 [batch], default T) of q [batch, T, heads, dim]
    into q_out and, if given, of k [batch, T, kv_heads, dim] into k_out (bf16, f16 or fp32,
    one type; an output may be its input).  Their positions: pos[b, i] (int32 [batch, T]), or
    seq_len[b] + the depth of drafted token i in the tree parent[b] (int32 [batch, T]), or
    seq_len[b] + i."""
    rq, T = _kv8_rows(cache, q, "q", None, True)
    H = q.shape[2]
    ro = _kv8_alike(cache, q_out, "q_out", H, q, "q", T, rq.type, True)
    if (k is None) != (k_out is None):
        raise Csa2Error("k and k_out go together")
    rk = rko = None
    if k is not None:
        rk = ctypes.byref(_kv8_alike(cache, k, "k", cache.kv_heads, q, "q", T, rq.type, True))
        rko = ctypes.byref(_kv8_alike(cache, k_out, "k_out", cache.kv_heads, q, "q", T, rq.type, True))
    if pos is not None and parent is not None:
        raise Csa2Error("pos or parent, not both")
    if parent is not None and T > KV8_MAX_TREE:
        raise Csa2Error(f"a tree has at most {KV8_MAX_TREE} drafted tokens")
    ql = _kv8_arg(cache, q_len, "q_len", "int32", (cache.batch,))
    ps = _kv8_arg(cache, pos, "pos", "int32", (cache.batch, T))
    pa = _kv8_arg(cache, parent, "parent", "int32", (cache.batch, T))
    _kv8_run(cache, "csa2_kv8_rope", _kv8_rope, stream, ctypes.byref(cache.struct),
             _kv8_table(cache, rope), ctypes.byref(rq), H, ctypes.byref(ro), rk, rko, T, ql, ps, pa,
             _kv8_ws(cache, ws))


def kv8_append_rope(cache, k, v, rope, ws, q=None, q_out=None, new_len=None, start=None, pos=None,
                    stream=None):
    """kv8_append of the rows k, rotated at the positions pos (int32 [batch, T], default
    start[b] + i), and v; with q [batch, T, heads, dim] (bf16, f16 or fp32) the step's
    queries are rotated at the same positions into q_out, which may be q."""
    rk, T = _kv8_rows(cache, k, "k", cache.kv_heads, True)
    rv = _kv8_alike(cache, v, "v", cache.kv_heads, k, "k", T, rk.type, True)
    if (q is None) != (q_out is None):
        raise Csa2Error("q and q_out go together")
    rq = ro = None
    H = 0
    if q is not None:
        x, Tq = _kv8_rows(cache, q, "q", None, True)
        H = q.shape[2]
        if Tq != T:
            raise Csa2Error("q: the T of k and v")
        rq = ctypes.byref(x)
        ro = ctypes.byref(_kv8_alike(cache, q_out, "q_out", H, q, "q", T, x.type, True))
    nl = _kv8_arg(cache, new_len, "new_len", "int32", (cache.batch,))
    sp = _kv8_arg(cache, start, "start", "int32", (cache.batch,))
    ps = _kv8_arg(cache, pos, "pos", "int32", (cache.batch, T))
    _kv8_run(cache, "csa2_kv8_append_rope", _kv8_append_rope, stream, ctypes.byref(cache.struct),
             _kv8_table(cache, rope), ctypes.byref(rk), ctypes.byref(rv), T, rq, H, ro, nl, sp, ps,
             _kv8_ws(cache, ws))


def kv8_append_path(cache, k, v, path, ws, new_len=None, start=None, stream=None):
    """kv8_append of chosen rows of k, v [batch, T, kv_heads, dim]: the i-th new row of a
    sequence is row path[b, i] (int32 [batch, M]); new_len[b] of them (default M).  The drafted
    tokens on an accepted path, with the keys that kv8_attn_tree took."""
    rk, T = _kv8_rows(cache, k, "k", cache.kv_heads, True)
    rv = _kv8_alike(cache, v, "v", cache.kv_heads, k, "k", T, rk.type, True)
    if len(path.shape) != 2:
        raise Csa2Error("path: it takes [batch, M]")
    M = path.shape[1]
    if T == 0 and M > 0:
        raise Csa2Error("path: there are no rows to choose from")
    pt = _kv8_arg(cache, path, "path", "int32", (cache.batch, M))
    nl = _kv8_arg(cache, new_len, "new_len", "int32", (cache.batch,))
    sp = _kv8_arg(cache, start, "start", "int32", (cache.batch,))
    _kv8_run(cache, "csa2_kv8_append_path", _kv8_append_path, stream, ctypes.byref(cache.struct),
             ctypes.byref(rk), ctypes.byref(rv), T, pt, M, nl, sp, _kv8_ws(cache, ws))


def kv8_attn_scored(cache, q, out, ws, scores, lse=None, q_len=None, softmax_scale=0.0, stream=None):
    """kv8_attn with what `scores` (Scores) does to the scores and to which rows count; query
    i of a sequence is at position seq_len[b] - q_len[b] + i.  kv8_mass does not take its lse."""
    rq, T = _kv8_rows(cache, q, "q")
    H = q.shape[2]
    ro = _kv8_alike(cache, out, "out", H, q, "q", T, rq.type)
    ls = _kv8_arg(cache, lse, "lse", "float32", (cache.batch, T, H))
    ql = _kv8_arg(cache, q_len, "q_len", "int32", (cache.batch,))
    _kv8_run(cache, "csa2_kv8_attn_scored", _kv8_attn_scored, stream, ctypes.byref(cache.struct),
             ctypes.byref(rq), H, T, ql, softmax_scale, _kv8_scores(cache, scores, H),
             ctypes.byref(ro), ls, _kv8_ws(cache, ws, T, H))


def kv8_attn_tree(cache, q, k, v, parent, out, ws, lse=None, q_len=None, softmax_scale=0.0,
                  scores=None, stream=None):
    """Attention of drafted tokens, which are not in the cache: token i of a sequence's first
    q_len[b] (default T <= KV8_MAX_TREE) sees all rows of the cache, itself and the tokens that
    it follows, parent[b, i] (int32 [batch, T]; an earlier token, or -1) and so on.  q [batch,
    T, heads, dim], k and v [batch, T, kv_heads, dim] (bf16 or f16, rotated as kv8_rope with
    `parent` does); out, lse as kv8_attn; scores without a prefix; ws: cache.tree_workspace."""
    rq, T = _kv8_rows(cache, q, "q")
    H = q.shape[2]
    rk = _kv8_alike(cache, k, "k", cache.kv_heads, q, "q", T, rq.type)
    rv = _kv8_alike(cache, v, "v", cache.kv_heads, q, "q", T, rq.type)
    ro = _kv8_alike(cache, out, "out", H, q, "q", T, rq.type)
    if T > KV8_MAX_TREE:
        raise Csa2Error(f"a tree has at most {KV8_MAX_TREE} drafted tokens")
    if parent is None:
        raise Csa2Error("csa2_kv8_attn_tree: it takes `parent`")
    if isinstance(scores, Scores) and scores.prefix is not None:
        raise Csa2Error("csa2_kv8_attn_tree: scores without a prefix")
    pa = _kv8_arg(cache, parent, "parent", "int32", (cache.batch, T))
    ls = _kv8_arg(cache, lse, "lse", "float32", (cache.batch, T, H))
    ql = _kv8_arg(cache, q_len, "q_len", "int32", (cache.batch,))
    _kv8_run(cache, "csa2_kv8_attn_tree", _kv8_attn_tree, stream, ctypes.byref(cache.struct),
             ctypes.byref(rq), H, ctypes.byref(rk), ctypes.byref(rv), pa, T, ql, softmax_scale,
             None if scores is None else _kv8_scores(cache, scores, H), ctypes.byref(ro), ls,
             _kv8_ws(cache, ws, T, H, tree=True))
