"""ctypes binding of libkascade.so (the C ABI in include/kascade.h).

Argument marshalling only: every step of the computation runs in the CUDA
library.  Tensors are torch CUDA tensors (used for device memory and
streams); the library raises if it was not built.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

__all__ = ["Shape", "KascadeError", "lib", "OP_SELECT", "OP_SPARSE_DECODE", "OP_SPARSE_PREFILL",
           "OP_DENSE", "workspace_bytes", "index_count", "index_offsets", "Workspace", "select",
           "sparse_decode", "sparse_prefill", "dense_ref", "status_str", "launch_count", "EXPORTS", "LIB_PATH",
           "select_decode_static", "select_decode_static_error", "refine_select", "OP_REFINE",
           "index_overlap", "plan_anchors", "sparse_decode_paged", "select_varlen", "sparse_decode_varlen",
           "Q8Cache", "page_tables", "q8_append", "q8_gather", "sparse_decode_q8", "OP_SPARSE_DECODE_Q8",
           "CACHE_E4M3", "CACHE_INT8"]

LIB_PATH = os.environ.get("KASCADE_LIB") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkascade.so")

OP_SELECT, OP_SPARSE_DECODE, OP_SPARSE_PREFILL, OP_DENSE, OP_REFINE, OP_SELECT_VARLEN = 0, 1, 2, 3, 4, 5
OP_SPARSE_DECODE_Q8 = 6
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TOO_LARGE = 0, 1, 2, 3, 4, 5
FLAG_PDL, FLAG_INPUTS_STABLE, FLAG_CHECK_INDICES, FLAG_TEST_DROP_LOAD = 1, 2, 4, 1 << 30
DEVERR_SCORE_POOL, DEVERR_DECODE_MERGE, DEVERR_PREFILL_ATTN, DEVERR_DECODE_SELECT = 2, 3, 4, 5
DEVERR_DECODE_GATHER, DEVERR_INDEX_LIST, DEVERR_PAGE = 6, 7, 8
SELECT_GQA, SELECT_PER_HEAD, SELECT_ALL_HEADS = 0, 1, 2
DTYPE_BF16, DTYPE_F32, DTYPE_F16 = 0, 1, 2
CACHE_E4M3, CACHE_INT8 = 0, 1

EXPORTS = ("kascade_workspace_bytes", "kascade_index_count", "kascade_index_offsets",
           "kascade_workspace_init", "kascade_select", "kascade_sparse_decode",
           "kascade_sparse_prefill", "kascade_dense_ref", "kascade_workspace_error",
           "kascade_status_str", "kascade_select_decode_static", "kascade_select_decode_static_max_bytes",
           "kascade_launch_count", "kascade_select_decode_static_error", "kascade_refine_select",
           "kascade_index_overlap", "kascade_plan_anchors", "kascade_sparse_decode_paged",
           "kascade_select_varlen", "kascade_sparse_decode_varlen", "kascade_page_tables", "kascade_q8_append",
           "kascade_q8_gather", "kascade_sparse_decode_q8")


class KascadeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_str(status)} (status {status})")
        self.status = status


class Shape(ctypes.Structure):
    """kascade_shape: B, Hq, Hkv, d, q_len (1 = decode), kv_len, tile, frac."""
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("q_len", ctypes.c_int32), ("kv_len", ctypes.c_int32), ("tile", ctypes.c_int32),
                ("topk_num", ctypes.c_int32), ("topk_den", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("select_mode", ctypes.c_int32), ("dtype", ctypes.c_int32)]

    @classmethod
    def make(cls, batch, hq, hkv, d, q_len, kv_len, frac=(10, 100), tile=32, flags=0, mode=0, dtype=0):
        return cls(batch, hq, hkv, d, q_len, kv_len, tile, frac[0], frac[1], flags, mode, dtype)

    def with_flags(self, flags: int) -> "Shape":
        return Shape(self.batch, self.num_q_heads, self.num_kv_heads, self.head_dim, self.q_len,
                     self.kv_len, self.tile, self.topk_num, self.topk_den, flags, self.select_mode, self.dtype)

    @property
    def n_lists(self) -> int:
        """Index lists per batch row under the shape's selection mode."""
        return {SELECT_PER_HEAD: self.num_q_heads, SELECT_ALL_HEADS: 1}.get(self.select_mode, self.num_kv_heads)

    @property
    def decode(self) -> bool:
        return self.q_len == 1


class _Q8CacheArgs(ctypes.Structure):
    """kascade_q8_cache."""
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("scale_block", ctypes.c_int32), ("type", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m sparse_attention_long_anchor_b200.build`")
    so = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    SP = ctypes.POINTER(Shape)
    so.kascade_workspace_bytes.argtypes = [SP, ctypes.c_int]
    so.kascade_workspace_bytes.restype = ctypes.c_size_t
    so.kascade_index_count.argtypes = [SP]
    so.kascade_index_count.restype = ctypes.c_int64
    so.kascade_index_offsets.argtypes = [SP, ctypes.POINTER(ctypes.c_int64)]
    so.kascade_index_offsets.restype = ctypes.c_int
    so.kascade_workspace_init.argtypes = [P, ctypes.c_size_t, P]
    so.kascade_workspace_init.restype = ctypes.c_int
    so.kascade_select.argtypes = [SP, P, P, P, P, ctypes.c_size_t, P]
    so.kascade_select.restype = ctypes.c_int
    for fn in (so.kascade_sparse_decode, so.kascade_sparse_prefill):
        fn.argtypes = [SP, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        fn.restype = ctypes.c_int
    so.kascade_dense_ref.argtypes = [SP, P, P, P, ctypes.c_int, P, P, P, ctypes.c_size_t, P]
    so.kascade_dense_ref.restype = ctypes.c_int
    so.kascade_workspace_error.argtypes = [P, ctypes.POINTER(ctypes.c_int), ctypes.c_int, P]
    so.kascade_workspace_error.restype = ctypes.c_int
    so.kascade_select_varlen.argtypes = [SP, P, P, P, P, P, ctypes.c_size_t, P]
    so.kascade_select_varlen.restype = ctypes.c_int
    so.kascade_sparse_decode_varlen.argtypes = [SP, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    so.kascade_sparse_decode_varlen.restype = ctypes.c_int
    so.kascade_sparse_decode_paged.argtypes = [SP, P, P, P, P, ctypes.c_int32, ctypes.c_int32, P, P, P, P, P,
                                               ctypes.c_size_t, P]
    so.kascade_sparse_decode_paged.restype = ctypes.c_int
    I, L, CP = ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(_Q8CacheArgs)
    so.kascade_page_tables.argtypes = [I, I, I, P, P, P, I, P, P, P, P, I, P, P]
    so.kascade_page_tables.restype = ctypes.c_int
    so.kascade_q8_append.argtypes = [CP, P, P, L, L, L, L, I, I, P, P, ctypes.c_size_t, P]
    so.kascade_q8_append.restype = ctypes.c_int
    so.kascade_q8_gather.argtypes = [CP, I, I, P, I, P, I, P, P, P, ctypes.c_size_t, P]
    so.kascade_q8_gather.restype = ctypes.c_int
    so.kascade_sparse_decode_q8.argtypes = [SP, CP, P, P, I, P, P, P, P, P, P, ctypes.c_size_t, P]
    so.kascade_sparse_decode_q8.restype = ctypes.c_int
    so.kascade_index_overlap.argtypes = [SP, P, P, P, P]
    so.kascade_index_overlap.restype = ctypes.c_int
    so.kascade_plan_anchors.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.c_int32, ctypes.c_int32,
                                        ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_double)]
    so.kascade_plan_anchors.restype = ctypes.c_int
    so.kascade_refine_select.argtypes = [SP, P, P, P, ctypes.c_int32, P, P, P, ctypes.c_size_t, P]
    so.kascade_refine_select.restype = ctypes.c_int
    so.kascade_select_decode_static.argtypes = [SP, P, P, P, P]
    so.kascade_select_decode_static.restype = ctypes.c_int
    so.kascade_select_decode_static_error.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.c_int, P]
    so.kascade_select_decode_static_error.restype = ctypes.c_int
    so.kascade_select_decode_static_max_bytes.argtypes = []
    so.kascade_select_decode_static_max_bytes.restype = ctypes.c_size_t
    so.kascade_launch_count.argtypes = [SP, ctypes.c_int]
    so.kascade_launch_count.restype = ctypes.c_int
    so.kascade_status_str.argtypes = [ctypes.c_int]
    so.kascade_status_str.restype = ctypes.c_char_p
    return so


lib = _load()


def status_str(status: int) -> str:
    return lib.kascade_status_str(status).decode()


def launch_count(shape: "Shape", op: int) -> int:
    """Kernels that `op` launches for `shape` on the current device."""
    n = lib.kascade_launch_count(ctypes.byref(shape), op)
    if n < 0:
        raise KascadeError(ERR_INVALID_ARG, "kascade_launch_count")
    return n


def _check(status: int, where: str):
    if status != OK:
        raise KascadeError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the raw handle of the current stream without building a Stream object
# (a per-call host cost of the eager API); the public call where absent
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def workspace_bytes(shape: Shape, op: int) -> int:
    return int(lib.kascade_workspace_bytes(ctypes.byref(shape), op))


def index_count(shape: Shape) -> int:
    n = int(lib.kascade_index_count(ctypes.byref(shape)))
    if n < 0:
        raise KascadeError(ERR_INVALID_ARG, "kascade_index_count")
    return n


def index_offsets(shape: Shape) -> np.ndarray:
    """Tile offsets of one index row (the call's tiles: a rolling chunk's own)."""
    n_t = 1 if shape.decode else -(-shape.kv_len // 32) - (shape.kv_len - shape.q_len) // 32
    out = np.zeros(n_t + 1, dtype=np.int64)
    _check(lib.kascade_index_offsets(ctypes.byref(shape), out.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))),
           "kascade_index_offsets")
    return out


class Workspace:
    """A zero-initialised device workspace large enough for the given ops."""

    def __init__(self, shape: Shape, ops=(OP_SELECT, OP_SPARSE_DECODE, OP_SPARSE_PREFILL, OP_DENSE, OP_REFINE),
                 device="cuda", nbytes=None):
        need = nbytes if nbytes is not None else max([workspace_bytes(shape, op) for op in ops] + [256])
        self.buf = torch.zeros(need + 256, dtype=torch.uint8, device=device)
        base = self.buf.data_ptr()
        self.ptr = (base + 255) // 256 * 256
        self.nbytes = need

    def args(self):
        return self.ptr, self.nbytes

    def error(self, clear=True, stream=None) -> int:
        """The device error word (0 = no kernel gave up on a bounded wait)."""
        out = ctypes.c_int(0)
        _check(lib.kascade_workspace_error(self.ptr, ctypes.byref(out), int(clear), _stream(stream)),
               "kascade_workspace_error")
        return out.value


def _ws(ws, shape, op):
    if ws is None:
        if op != OP_SELECT and not shape.flags & FLAG_CHECK_INDICES:
            return None, 0       # attention calls run without an error word
        ws = Workspace(shape, (op,))
    return ws.args()


def select(shape: Shape, q, k, idx=None, ws=None, stream=None):
    """kascade_select: anchor Top-k index sets (int32, ascending)."""
    if idx is None:
        idx = torch.empty(index_count(shape), dtype=torch.int32, device=q.device)
    p, n = _ws(ws, shape, OP_SELECT)
    _check(lib.kascade_select(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(idx), p, n, _stream(stream)),
           "kascade_select")
    return idx


def refine_select(shape: Shape, q, k, pool, pool_len: int, head_map=None, idx=None, ws=None, stream=None):
    """kascade_refine_select: a refined decode layer's own Top-k from the
    proposal layer's pool [B, Hkv, pool_len]."""
    if idx is None:
        idx = torch.empty(index_count(shape), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = Workspace(shape, (OP_REFINE,))
    p, n = ws.args()
    _check(lib.kascade_refine_select(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(pool), int(pool_len),
                                     _ptr(head_map), _ptr(idx), p, n, _stream(stream)), "kascade_refine_select")
    return idx


def index_overlap(shape: Shape, a, b, counts=None, stream=None):
    """kascade_index_overlap: |a and b| per (batch row, list), summed over tiles."""
    if counts is None:
        counts = torch.empty(shape.batch * shape.n_lists, dtype=torch.int64, device=a.device)
    _check(lib.kascade_index_overlap(ctypes.byref(shape), _ptr(a), _ptr(b), _ptr(counts), _stream(stream)),
           "kascade_index_overlap")
    return counts


def plan_anchors(sim, n_anchors: int):
    """kascade_plan_anchors: (anchor layers, objective) for a host
    similarity matrix sim[a][l]."""
    sim = np.ascontiguousarray(np.asarray(sim, dtype=np.float64))
    n = sim.shape[0]
    out = (ctypes.c_int32 * max(n_anchors, 1))()
    obj = ctypes.c_double(0.0)
    _check(lib.kascade_plan_anchors(sim.ctypes.data_as(ctypes.POINTER(ctypes.c_double)), n, n_anchors, out,
                                    ctypes.byref(obj)), "kascade_plan_anchors")
    return list(out)[:n_anchors], obj.value


def select_decode_static(shape: Shape, q, k, idx=None, stream=None):
    """kascade_select_decode_static: decode anchor selection with the library's
    fixed scratch array instead of a workspace (nothing is allocated)."""
    if idx is None:
        idx = torch.empty(index_count(shape), dtype=torch.int32, device=q.device)
    _check(lib.kascade_select_decode_static(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(idx), _stream(stream)),
           "kascade_select_decode_static")
    return idx


def select_decode_static_error(clear=True, stream=None) -> int:
    """The device error word of kascade_select_decode_static on the current
    device (0 = no kernel gave up on a bounded wait)."""
    out = ctypes.c_int(0)
    _check(lib.kascade_select_decode_static_error(ctypes.byref(out), int(clear), _stream(stream)),
           "kascade_select_decode_static_error")
    return out.value


def _attn(fn, name, shape, q, k, v, idx, head_map, o, lse, ws, stream, op):
    if o is None:
        o = torch.empty_like(q)
    p, n = _ws(ws, shape, op)
    _check(fn(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(head_map), _ptr(o),
              _ptr(lse), p, n, _stream(stream)), name)
    return o


def sparse_decode(shape: Shape, q, k, v, idx, head_map=None, o=None, lse=None, ws=None, stream=None):
    """kascade_sparse_decode: kv head h attends over anchor list head_map[h]."""
    return _attn(lib.kascade_sparse_decode, "kascade_sparse_decode", shape, q, k, v, idx, head_map, o, lse,
                 ws, stream, OP_SPARSE_DECODE)


def select_varlen(shape: Shape, q, k, kv_lens, idx=None, ws=None, stream=None):
    """kascade_select_varlen: decode selection with a context length per batch
    row (lists padded with -1 to the layout of kv_len)."""
    if idx is None:
        idx = torch.empty(index_count(shape), dtype=torch.int32, device=q.device)
    if ws is None:
        ws = Workspace(shape, (OP_SELECT_VARLEN,))
    p, n = ws.args()
    _check(lib.kascade_select_varlen(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(kv_lens), _ptr(idx), p, n,
                                     _stream(stream)), "kascade_select_varlen")
    return idx


def sparse_decode_varlen(shape: Shape, q, k, v, kv_lens, idx, head_map=None, o=None, lse=None, ws=None,
                         stream=None):
    """kascade_sparse_decode_varlen: sparse (idx None: dense) decode with a
    context length per batch row."""
    if o is None:
        o = torch.empty_like(q)
    p, n = _ws(ws, shape, OP_SPARSE_DECODE)
    _check(lib.kascade_sparse_decode_varlen(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(kv_lens),
                                            _ptr(idx), _ptr(head_map), _ptr(o), _ptr(lse), p, n, _stream(stream)),
           "kascade_sparse_decode_varlen")
    return o


def sparse_decode_paged(shape: Shape, q, k_pages, v_pages, page_table, page_size: int, idx, head_map=None, o=None,
                        lse=None, ws=None, stream=None):
    """kascade_sparse_decode_paged: sparse (or, with idx None, dense) decode
    over pages [num_pages, Hkv, page_size, d] named by page_table [B, max_pages]."""
    if o is None:
        o = torch.empty_like(q)
    p, n = _ws(ws, shape, OP_SPARSE_DECODE)
    _check(lib.kascade_sparse_decode_paged(ctypes.byref(shape), _ptr(q), _ptr(k_pages), _ptr(v_pages),
                                           _ptr(page_table), int(page_size), int(page_table.shape[-1]), _ptr(idx),
                                           _ptr(head_map), _ptr(o), _ptr(lse), p, n, _stream(stream)),
           "kascade_sparse_decode_paged")
    return o


def sparse_prefill(shape: Shape, q, k, v, idx, head_map=None, o=None, lse=None, ws=None, stream=None):
    """kascade_sparse_prefill: causal tile-level sparse attention."""
    return _attn(lib.kascade_sparse_prefill, "kascade_sparse_prefill", shape, q, k, v, idx, head_map, o,
                 lse, ws, stream, OP_SPARSE_PREFILL)


def dense_ref(shape: Shape, q, k, v, causal=True, o=None, lse=None, ws=None, stream=None):
    """kascade_dense_ref: dense (causal) attention."""
    if o is None:
        o = torch.empty_like(q)
    p, n = _ws(ws, shape, OP_DENSE)
    _check(lib.kascade_dense_ref(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), int(bool(causal)), _ptr(o),
                                 _ptr(lse), p, n, _stream(stream)), "kascade_dense_ref")
    return o


# ---------------------------------------------------------------- 8-bit paged cache

_CACHE_TYPES = {torch.float8_e4m3fn: CACHE_E4M3, torch.int8: CACHE_INT8}
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32, torch.float16: DTYPE_F16}


def _need(ok, where: str, status: int = ERR_INVALID_ARG):
    if not ok:
        raise KascadeError(status, where)


def _dense(t, dtype, numel, index, where: str):
    """t's address; raises unless t is a contiguous tensor of this type and size on CUDA device `index`."""
    if t.dtype is not dtype or t.numel() != numel or t.get_device() != index or not t.is_contiguous():
        raise KascadeError(ERR_INVALID_ARG, where)
    return t.data_ptr()


def _here(index, stream):
    """The handle of the stream of a call that runs as things are, on the
    current device `index` and its current stream; None if it does not."""
    if stream is not None or index < 0 or index != torch.cuda.current_device():
        return None
    return _raw_stream(index) if _raw_stream is not None else torch.cuda.current_stream(index).cuda_stream


def _on(device, stream, where):
    """A context in which `device` is the current one and an explicit `stream`
    torch's current stream, so that what the call allocates belongs to the
    stream that its kernels run on."""
    if stream is None:
        return torch.cuda.device(device)
    if isinstance(stream, int):
        # (0 is the legacy default stream, which torch's default stream is)
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    _need(stream.device == device, where)
    return torch.cuda.stream(stream)   # switches the device too


class Q8Cache:
    """An 8-bit paged KV cache: k_pages, v_pages [num_pages, Hkv, page_size, d]
    (torch.float8_e4m3fn or torch.int8) and scales [num_pages, Hkv,
    page_size / scale_block, 2] in fp32, the (K, V) scale of each block of rows.
    Keeps the tensors it is given; their addresses must not change."""

    def __init__(self, k_pages, v_pages, scales):
        where = "Q8Cache"
        _need(k_pages.dim() == 4 and scales.dim() == 4 and k_pages.dtype in _CACHE_TYPES, where)
        n, h, page, d = k_pages.shape
        blocks = scales.shape[2]
        _need(n > 0 and h > 0 and page > 0 and d > 0 and blocks > 0 and page % blocks == 0, where)
        _need(v_pages.shape == k_pages.shape and scales.shape == (n, h, blocks, 2), where)
        self.device, self.index = k_pages.device, k_pages.get_device()   # (index -1: not a CUDA device)
        kp = _dense(k_pages, k_pages.dtype, n * h * page * d, self.index, where)
        vp = _dense(v_pages, k_pages.dtype, n * h * page * d, self.index, where)
        sp = _dense(scales, torch.float32, n * h * blocks * 2, self.index, where)
        self.k_pages, self.v_pages, self.scales = k_pages, v_pages, scales
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = n, h, page, d
        self.scale_block = page // blocks
        self.args = _Q8CacheArgs(kp, vp, sp, n, h, d, page, self.scale_block, _CACHE_TYPES[k_pages.dtype])
        self.ref = ctypes.byref(self.args)

    @classmethod
    def empty(cls, num_pages: int, num_kv_heads: int, head_dim: int, page_size: int = 64, scale_block: int = None,
              dtype=torch.float8_e4m3fn, device="cuda") -> "Q8Cache":
        """A zeroed cache; one scale pair per page unless scale_block says otherwise."""
        block = min(page_size, 256) if scale_block is None else scale_block
        _need(dtype in _CACHE_TYPES and block > 0 and page_size % block == 0, "Q8Cache.empty")
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
        return cls(k, v, torch.zeros(*shape[:2], page_size // block, 2, device=device))


def page_tables(page_size: int, kv_lens, new_lens, free_pages, page_table, capacity: int, out=None, stream=None):
    """kascade_page_tables: extends page_table [B, max_pages] in place for
    new_lens [B] more tokens behind kv_lens [B], with pages from free_pages.
    Returns (kv_lens_out [B], offsets [B + 1], slot_map [capacity], info [2]),
    `out` if it is given (four buffers, none of them kv_lens)."""
    where = "kascade_page_tables"
    dev, i32 = page_table.get_device(), torch.int32
    _need(page_table.dim() == 2 and dev >= 0, where)
    raw = _here(dev, stream)
    if raw is None:
        with _on(page_table.device, stream, where):
            return page_tables(page_size, kv_lens, new_lens, free_pages, page_table, capacity, out)
    n, width = page_table.shape
    if out is None:
        # one allocation; the slots first, on its 16-byte aligned start
        buf = torch.empty(capacity + 2 * n + 3, dtype=i32, device=page_table.device)
        slot_map, lens_out, offsets, info = torch.split_with_sizes(buf, (capacity, n, n + 1, 2))
        out = (lens_out, offsets, slot_map, info)
        sp = buf.data_ptr()
        lp = sp + 4 * capacity
        op, ip = lp + 4 * n, lp + 8 * n + 4
    else:
        lens_out, offsets, slot_map, info = out
        lp, op = _dense(lens_out, i32, n, dev, where), _dense(offsets, i32, n + 1, dev, where)
        sp, ip = _dense(slot_map, i32, capacity, dev, where), _dense(info, i32, 2, dev, where)
    free = free_pages.numel()
    status = lib.kascade_page_tables(
        n, page_size, width, _dense(kv_lens, i32, n, dev, where), _dense(new_lens, i32, n, dev, where),
        _dense(free_pages, i32, free, dev, where), free, _dense(page_table, i32, n * width, dev, where), lp, op, sp,
        capacity, ip, raw)
    if status:
        raise KascadeError(status, where)
    return out


def q8_append(cache: Q8Cache, k, v, slot_map, ws=None, stream=None):
    """kascade_q8_append: quantises k, v [T, Hkv, d] (bf16, fp16 or fp32, any
    strides of whole 16 bytes with the last dim dense) into the slots of
    slot_map [T]."""
    where = "kascade_q8_append"
    dev = cache.index
    raw = _here(dev, stream)
    if raw is None:
        _need(dev >= 0, where)
        with _on(cache.device, stream, where):
            return q8_append(cache, k, v, slot_map, ws)
    dtype = k.dtype
    shape = k.shape
    if (len(shape) != 3 or v.shape != shape or v.dtype is not dtype or dtype not in _DTYPES
            or k.get_device() != dev or v.get_device() != dev):
        raise KascadeError(ERR_INVALID_ARG, where)
    t, heads, d = shape
    if heads != cache.num_kv_heads or d != cache.head_dim:
        raise KascadeError(ERR_INVALID_ARG, where)
    (kt, kh, kd), (vt, vh, vd) = k.stride(), v.stride()
    _need(kd == 1 and vd == 1, where, ERR_UNSUPPORTED)
    p, n = ws.args() if ws is not None else (None, 0)
    status = lib.kascade_q8_append(cache.ref, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh, _DTYPES[dtype], t,
                                   _dense(slot_map, torch.int32, t, dev, where), p, n, raw)
    if status:
        raise KascadeError(status, where)


def q8_gather(cache: Q8Cache, page_table, n_ctx: int, kv_lens=None, k=None, v=None, dtype=None, ws=None, stream=None):
    """kascade_q8_gather: the cache's rows as slabs (k, v) [B, Hkv, n_ctx, d].
    Rows from kv_lens[b] on stay as they are in the given k and v, and are zero
    in slabs that the call makes (both, of `dtype`, bf16 by default, unless one
    of the two is given)."""
    where = "kascade_q8_gather"
    dev, i32 = cache.index, torch.int32
    _need(page_table.dim() == 2 and dev >= 0, where)
    raw = _here(dev, stream)
    if raw is None:
        with _on(cache.device, stream, where):
            return q8_gather(cache, page_table, n_ctx, kv_lens, k, v, dtype, ws)
    b, width = page_table.shape
    shape = (b, cache.num_kv_heads, n_ctx, cache.head_dim)
    if k is None and v is None:
        make = torch.empty if kv_lens is None else torch.zeros
        k, v = (make(shape, dtype=dtype or torch.bfloat16, device=cache.device) for _ in range(2))
    one = (v if k is None else k).dtype
    _need(one in _DTYPES and (k is None or k.shape == shape) and (v is None or v.shape == shape), where)
    total = b * shape[1] * n_ctx * shape[3]
    p, n = ws.args() if ws is not None else (None, 0)
    status = lib.kascade_q8_gather(
        cache.ref, b, n_ctx, _dense(page_table, i32, b * width, dev, where), width,
        None if kv_lens is None else _dense(kv_lens, i32, b, dev, where), _DTYPES[one],
        None if k is None else _dense(k, one, total, dev, where),
        None if v is None else _dense(v, one, total, dev, where), p, n, raw)
    if status:
        raise KascadeError(status, where)
    return k, v


def sparse_decode_q8(shape: Shape, q, cache: Q8Cache, page_table, idx=None, head_map=None, kv_lens=None, o=None,
                     lse=None, ws=None, stream=None):
    """kascade_sparse_decode_q8: sparse (idx None: dense) decode of q
    [B, Hq, 1, d] over an 8-bit paged cache, page_table [B, max_pages]."""
    where = "kascade_sparse_decode_q8"
    dev, i32 = cache.index, torch.int32
    raw = _here(dev, stream)
    if raw is None:
        _need(dev >= 0, where)
        with _on(cache.device, stream, where):
            return sparse_decode_q8(shape, q, cache, page_table, idx, head_map, kv_lens, o, lse, ws)
    b, hq, lists = shape.batch, shape.num_q_heads, shape.n_lists
    n_q = b * hq * shape.head_dim
    dt = torch.float16 if shape.dtype == DTYPE_F16 else torch.bfloat16
    _need(page_table.dim() == 2, where)
    width = page_table.shape[1]
    qp = _dense(q, dt, n_q, dev, where)
    if o is None:
        o = torch.empty_like(q)
        op = o.data_ptr()
    else:
        op = _dense(o, dt, n_q, dev, where)
    if ws is None:
        ws = Workspace(shape, (OP_SPARSE_DECODE_Q8,), device=cache.device)
    p, n = ws.args()
    if idx is not None:   # B lists K entries, K = ceil(frac N)
        count = -(-shape.topk_num * shape.kv_len // max(shape.topk_den, 1))
        idx = _dense(idx, i32, b * lists * count, dev, where)
    status = lib.kascade_sparse_decode_q8(
        ctypes.byref(shape), cache.ref, qp, _dense(page_table, i32, b * width, dev, where), width,
        None if kv_lens is None else _dense(kv_lens, i32, b, dev, where), idx,
        None if head_map is None else _dense(head_map, i32, lists, dev, where), op,
        None if lse is None else _dense(lse, torch.float32, b * hq, dev, where), p, n, raw)
    if status:
        raise KascadeError(status, where)
    return o
