"""ctypes binding of libdsa.so (include/dsa.h): argument marshalling only.

Every function here forwards torch tensors' device pointers and the current
CUDA stream to the C ABI of the same name and raises DsaError on a non-OK
status. Every step of the DSA forward path runs in the library's CUDA
kernels; there is no Python or CPU fallback. Importing this module loads the
library and fails loudly if it has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdsa.so")

DSA_OK = 0
DSA_ERR_INVALID_ARG = 1
DSA_ERR_UNSUPPORTED = 2
DSA_ERR_WORKSPACE_TOO_SMALL = 3
DSA_ERR_CUDA = 4
DSA_ERR_DEVICE_BOUNDS = 5
DSA_ERR_TIMEOUT = 6

DSA_F32, DSA_E4M3, DSA_BF16 = 0, 1, 2
DSA_KV_CONTIGUOUS, DSA_KV_PAGED = 0, 1
DSA_OP_INDEXER_SCORES, DSA_OP_TOPK, DSA_OP_SPARSE_MQA, DSA_OP_FORWARD = 0, 1, 2, 3

DSA_OP_SELECT = 4
DSA_OP_KV8_MQA, DSA_OP_KV8_ACCUMULATE = 5, 6

EXPORTED = ["dsa_indexer_scores", "dsa_topk", "dsa_sparse_mqa_fwd", "dsa_select", "dsa_forward",
            "dsa_workspace_size", "dsa_check_status", "dsa_status_string",
            "dsa_last_cuda_error", "dsa_launch_counter", "dsa_version", "dsa_select_noalloc",
            "dsa_set_wait_limit_ns", "dsa_dense_mqa_fwd", "dsa_select_scored", "dsa_indexer_kl",
            "dsa_sparse_mqa_bwd", "dsa_kv8_store", "dsa_kv8_mqa_fwd", "dsa_kv8_accumulate",
            "dsa_kv8_evict"]


class DsaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} ({status_string(status)})")


class KvLayout(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("ld_block_table", ctypes.c_int64),
                ("max_pages", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("ctx_lens", ctypes.c_void_p), ("q_seq", ctypes.c_void_p),
                ("q_pos", ctypes.c_void_p), ("n_seq", ctypes.c_int32)]
    tensors = sizes = None    # of paged_layout; sequences, keys of the longest, pages
    fits, dev = False, -1     # one sequence a query, all as the C side reads it; on which device


class IndexerIn(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_q", ctypes.c_int32), ("n_keys", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("ld_q", ctypes.c_int64), ("q_scale", ctypes.c_void_p),
                ("k", ctypes.c_void_p), ("ld_k", ctypes.c_int64), ("k_scale", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("ld_w", ctypes.c_int64), ("kv", KvLayout)]


class AttnIn(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("n_q", ctypes.c_int32), ("n_keys", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("d_qk", ctypes.c_int32), ("d_v", ctypes.c_int32),
                ("scale", ctypes.c_float),
                ("q", ctypes.c_void_p), ("ld_q", ctypes.c_int64),
                ("kv", ctypes.c_void_p), ("ld_kv", ctypes.c_int64),
                ("v", ctypes.c_void_p), ("ld_v", ctypes.c_int64),
                ("kv_layout", KvLayout)]


class Kv8Cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("ld", ctypes.c_int64), ("exps", ctypes.c_void_p),
                ("n_keys", ctypes.c_int32), ("kv", KvLayout)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_attention_long_tcgen05_b200._build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    F32 = ctypes.c_float
    sig = {
        "dsa_indexer_scores": [ctypes.POINTER(IndexerIn), P, I32, P, I64, I32, P, SZ, P],
        "dsa_topk": [P, I64, P, I32, I32, P, I64, P],
        "dsa_sparse_mqa_fwd": [ctypes.POINTER(AttnIn), P, I64, I32, P, P, P, SZ, P],
        "dsa_select": [ctypes.POINTER(IndexerIn), I32, P, I64, P, SZ, P],
        "dsa_dense_mqa_fwd": [ctypes.POINTER(AttnIn), P, P, P],
        "dsa_select_scored": [ctypes.POINTER(IndexerIn), I32, P, I64, P, I64, P, SZ, P],
        "dsa_indexer_kl": [ctypes.POINTER(AttnIn), P, I64, I32, P, P, I64, P, P, I64, P],
        "dsa_sparse_mqa_bwd": [ctypes.POINTER(AttnIn), P, I64, I32, P, P, P, P, P, I64, P, P],
        "dsa_forward": [ctypes.POINTER(IndexerIn), ctypes.POINTER(AttnIn), I32, P, P, P, P, SZ, P],
        "dsa_kv8_store": [ctypes.POINTER(Kv8Cache), I32, P, I64, P, I32, P],
        "dsa_kv8_mqa_fwd": [ctypes.POINTER(AttnIn), P, P, I64, I32, P, P, P, SZ, P],
        "dsa_kv8_accumulate": [ctypes.POINTER(AttnIn), P, P, I64, I32, P, F32, P, I64, P, SZ, P],
        "dsa_kv8_evict": [ctypes.POINTER(Kv8Cache), P, I64, P, P, I64, I32, I32, I32, P, I64, P, P,
                          I64, P, I64, P],
        "dsa_launch_counter": [],
        "dsa_set_wait_limit_ns": [I64],
        "dsa_select_noalloc": [ctypes.POINTER(IndexerIn), I32, P, I64, P],
        "dsa_workspace_size": [I32, ctypes.POINTER(IndexerIn), ctypes.POINTER(AttnIn), I32, I32,
                               I32, ctypes.POINTER(SZ)],
        "dsa_check_status": [P],
        "dsa_status_string": [ctypes.c_int],
        "dsa_last_cuda_error": [],
        "dsa_version": [],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = {"dsa_status_string": ctypes.c_char_p,
                     "dsa_launch_counter": ctypes.c_int64}.get(name, ctypes.c_int32)
    return lib


LIB = _load()


def status_string(status: int) -> str:
    return LIB.dsa_status_string(int(status)).decode()


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        # torch.cuda.current_stream().cuda_stream without building a Stream object
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != DSA_OK:
        raise DsaError(status, what + (f" (cudaError {LIB.dsa_last_cuda_error()})"
                                       if status == DSA_ERR_CUDA else ""))


# ------------------------------------------------------------ struct builders

class _Keep:
    """A C struct plus the tensors whose pointers it holds; for the 8-bit cache also
    the device of all of them and the sizes that the calls' other tensors need."""

    def __init__(self, struct, tensors, dev=-1, sizes=None):
        self.struct = struct
        self.tensors = tensors
        self.dev = dev
        self.sizes = sizes


def paged_layout(block_table: torch.Tensor, ctx_lens: torch.Tensor, num_pages: int,
                 q_seq: Optional[torch.Tensor] = None,
                 q_pos: Optional[torch.Tensor] = None) -> KvLayout:
    """PAGED key side: block_table [n_seq, max_pages] and ctx_lens [n_seq]
    int32; optional q_seq / q_pos [n_q] int32 (sequence and position of each
    query; by default query b is the newest token of sequence b). The caller
    keeps the tensors alive while the layout is in use."""
    rows, cols = block_table.shape
    ld, one = block_table.stride()
    n_seq = ctx_lens.shape[0]
    lay = KvLayout(DSA_KV_PAGED, 64, block_table.data_ptr(), ld, cols, num_pages, ctx_lens.data_ptr(),
                   q_seq.data_ptr() if q_seq is not None else None,
                   q_pos.data_ptr() if q_pos is not None else None, n_seq)
    lay.tensors = (block_table, ctx_lens, q_seq, q_pos)
    lay.sizes = (n_seq, cols * 64, num_pages)
    lay.dev = dev = block_table.get_device()
    lay.fits = (q_seq is q_pos is None and block_table.dtype is ctx_lens.dtype is torch.int32 and one == 1 and
                rows >= n_seq and ctx_lens.is_contiguous() and ctx_lens.get_device() == dev)
    return lay


def indexer_in(q, k, w, q_scale=None, k_scale=None, n_keys=None, kv: Optional[KvLayout] = None):
    """q [n_q, H_I, d_I] (uint8 e4m3 codes or float32), k [n_keys, d_I] or paged
    [pages, 64, d_I], w [n_q, H_I]; scales [n_q] / [n_keys or pages*64]."""
    fp8 = q.dtype == torch.uint8
    n_q, heads, dim = q.shape
    kv = kv if kv is not None else KvLayout(DSA_KV_CONTIGUOUS, 0, None, 0, 0, 0, None)
    ld_k = k.stride(-2)
    s = IndexerIn(DSA_E4M3 if fp8 else DSA_F32, n_q,
                  (n_keys if n_keys is not None else k.shape[0]) if kv.kind == DSA_KV_CONTIGUOUS
                  else 0,
                  heads, dim, q.data_ptr(), q.stride(0),
                  q_scale.data_ptr() if q_scale is not None else None,
                  k.data_ptr(), ld_k, k_scale.data_ptr() if k_scale is not None else None,
                  w.data_ptr(), w.stride(0), kv)
    return _Keep(s, [q, k, w, q_scale, k_scale])


def attn_in(q, kv, scale, d_v, v=None, kv_layout: Optional[KvLayout] = None):
    """q [n_q, H, d_qk], kv [n_keys, d_qk] or paged [pages, 64, d_qk] (bf16 or
    float32), optional separate v [n_keys, d_v] (float32 only)."""
    bf16 = q.dtype == torch.bfloat16
    n_q, heads, d_qk = q.shape
    lay = kv_layout if kv_layout is not None else KvLayout(DSA_KV_CONTIGUOUS, 0, None, 0, 0, 0,
                                                           None)
    paged = lay.kind == DSA_KV_PAGED
    n_keys = 0 if paged else kv.shape[0]
    st = q.stride()
    s = AttnIn(DSA_BF16 if bf16 else DSA_F32, n_q, n_keys,
               heads, d_qk, d_v, float(scale), q.data_ptr(), st[0], kv.data_ptr(),
               kv.stride()[-2], v.data_ptr() if v is not None else None,
               v.stride(0) if v is not None else 0, lay)
    if kv.dtype is not torch.uint8:
        return _Keep(s, [q, kv, v])
    # the 8-bit cache
    if not paged and kv.dim() != 2:
        raise DsaError(DSA_ERR_INVALID_ARG, "attn_in: kv must be [n_keys, 576] without a paged layout")
    if st[2] != 1 or (heads > 1 and st[1] != d_qk):
        raise DsaError(DSA_ERR_INVALID_ARG, "attn_in: q's heads must follow one another")
    n_seq, keys, blocks, dev = _cache_fits(lay, paged, kv, n_keys, n_q, "attn_in: kv")
    return _Keep(s, [q, kv, v, lay], dev if q.get_device() == dev else -1,
                 (n_q, n_q * heads, blocks, n_seq or n_q, keys))


def kv8_cache(codes: torch.Tensor, exps: torch.Tensor, kv: Optional[KvLayout] = None,
              n_keys: Optional[int] = None):
    """The latent cache in 8 bits: codes uint8 [pages, 64, 576] with a paged
    layout, or [n_keys, 576]; exps int8, one per page or per 64 rows. Rows may be
    further apart than 576 bytes, pages not further than their 64 rows."""
    lay = kv if kv is not None else KvLayout(DSA_KV_CONTIGUOUS, 0, None, 0, 0, 0, None)
    paged = lay.kind == DSA_KV_PAGED
    if not paged and n_keys is None and codes.dim() != 2:
        raise DsaError(DSA_ERR_INVALID_ARG, "kv8_cache: codes must be [n_keys, 576] without a paged layout or n_keys")
    n = 0 if paged else n_keys if n_keys is not None else codes.shape[0]
    n_seq, keys, blocks, dev = _cache_fits(lay, paged, codes, n, 0, "kv8_cache: codes")
    if not (exps.dtype is _I8 and exps.numel() >= blocks and exps.is_contiguous()):
        _flat(exps, _I8, blocks, "kv8_cache: exps")
    if exps.get_device() != dev:
        dev = -1
    s = Kv8Cache(codes.data_ptr(), codes.stride()[-2], exps.data_ptr(), n, lay)
    return _Keep(s, [codes, exps, lay], dev, (n_seq, keys, blocks))


# The C side sees addresses only: what the 8-bit cache's calls are given is checked
# here, or it would be misread, or written past its end. The calls test everything in
# one expression, which takes a microsecond; these functions, for which a Python call
# each would take several, say what did not fit.

_I8, _I32, _F32, _BF16, _U8 = torch.int8, torch.int32, torch.float32, torch.bfloat16, torch.uint8


def _need(t: Optional[torch.Tensor], dtype, what: str):
    if t is not None and t.dtype != dtype:
        raise DsaError(DSA_ERR_INVALID_ARG, f"{what} must be {dtype}, got {t.dtype}")


def _flat(t: Optional[torch.Tensor], dtype, n: int, what: str):
    """n elements in a row."""
    _need(t, dtype, what)
    if t is not None and (t.numel() < n or not t.is_contiguous()):
        raise DsaError(DSA_ERR_INVALID_ARG, f"{what} must be {n} contiguous elements")


def _matrix(t: Optional[torch.Tensor], dtype, rows: int, cols: int, what: str):
    """At least rows x cols, the rows any distance apart."""
    _need(t, dtype, what)
    if t is not None and (t.dim() != 2 or t.shape[0] < rows or t.shape[1] < cols or
                          (cols > 1 and t.stride(1) != 1)):
        raise DsaError(DSA_ERR_INVALID_ARG, f"{what} must be [{rows}, {cols}] at least, each row contiguous")


def _rows(t: torch.Tensor, width: int, lay: KvLayout, n_keys: int, what: str):
    """uint8 rows of `width` for every key or page, at one distance throughout."""
    _need(t, _U8, what)
    shape, stride = t.shape, t.stride()
    n = n_keys if lay.kind == DSA_KV_CONTIGUOUS else lay.num_pages * 64
    if not 2 <= len(shape) <= 3 or shape[-1] != width or stride[-1] != 1 or t.numel() < n * width:
        raise DsaError(DSA_ERR_INVALID_ARG, f"{what} must hold {n} rows of {width} contiguous elements")
    if len(shape) == 3 and ((lay.kind == DSA_KV_PAGED and shape[1] != 64) or
                            (shape[0] > 1 and stride[0] != shape[1] * stride[1])):
        raise DsaError(DSA_ERR_INVALID_ARG, f"{what} must be pages of 64 rows that follow one another")


def _cache_fits(lay: KvLayout, paged: bool, codes: torch.Tensor, n_keys: int, n_q: int, what: str):
    """Sequences, keys of the longest, blocks, and the device of the codes and the
    layout (-1: several)."""
    dev = codes.get_device()
    if not paged:
        _rows(codes, 576, lay, n_keys, what)
        return 1, n_keys, -(-n_keys // 64), dev
    shape, stride = codes.shape, codes.stride()
    n_seq, keys, pages = lay.sizes or (lay.n_seq, lay.max_pages * 64, lay.num_pages)
    if not (len(shape) == 3 and codes.dtype is _U8 and shape[2] == 576 and stride[2] == 1 and shape[1] == 64 and
            stride[0] == 64 * stride[1] and shape[0] >= pages):
        _rows(codes, 576, lay, n_keys, what)
    if lay.fits:
        return n_seq, keys, pages, dev if dev == lay.dev else -1
    if lay.tensors is not None:               # (a layout that the caller has filled in has none)
        table, lens, q_seq, q_pos = lay.tensors
        _matrix(table, _I32, n_seq, keys // 64, "paged_layout: block_table")
        _flat(lens, _I32, n_seq, "paged_layout: ctx_lens")
        _flat(q_seq, _I32, n_q, "paged_layout: q_seq")
        _flat(q_pos, _I32, n_q, "paged_layout: q_pos")
        if any(t is not None and t.get_device() != dev for t in lay.tensors):
            dev = -1
    return n_seq, keys, pages, dev


def _elsewhere(what: str):
    raise DsaError(DSA_ERR_INVALID_ARG, what + ": its tensors are not all on the current device")


def _stream_on(dev: int, stream, what: str):
    """The stream's handle; dev: the device of a call's tensors, which must be the current one."""
    if dev < 0 or dev != torch.cuda.current_device():
        _elsewhere(what)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


# ------------------------------------------------------------ the C ABI calls

def dsa_workspace_size(op, ind: Optional[_Keep] = None, attn: Optional[_Keep] = None,
                       n_rows: int = 0, n_cols: int = 0, k: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(LIB.dsa_workspace_size(op, ctypes.byref(ind.struct) if ind else None,
                                  ctypes.byref(attn.struct) if attn else None,
                                  n_rows, n_cols, k, ctypes.byref(out)), "dsa_workspace_size")
    return out.value


def dsa_indexer_scores(ind: _Keep, rows: Optional[torch.Tensor], n_rows: int,
                       scores: torch.Tensor, n_cols: int, ws: Optional[torch.Tensor] = None,
                       stream=None):
    _check(LIB.dsa_indexer_scores(ctypes.byref(ind.struct), _ptr(rows), n_rows, _ptr(scores),
                                  scores.stride(0), n_cols, _ptr(ws),
                                  0 if ws is None else ws.numel() * ws.element_size(),
                                  _stream(stream)), "dsa_indexer_scores")


def dsa_topk(scores: torch.Tensor, row_pos: torch.Tensor, k: int, idx: torch.Tensor,
             stream=None):
    _check(LIB.dsa_topk(_ptr(scores), scores.stride(0), _ptr(row_pos), scores.shape[0], k,
                        _ptr(idx), idx.stride(0), _stream(stream)), "dsa_topk")


def dsa_sparse_mqa_fwd(attn: _Keep, idx: torch.Tensor, k: int, out: torch.Tensor,
                       lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                       stream=None):
    _check(LIB.dsa_sparse_mqa_fwd(ctypes.byref(attn.struct), _ptr(idx), idx.stride(0), k,
                                  _ptr(out), _ptr(lse), _ptr(ws),
                                  0 if ws is None else ws.numel() * ws.element_size(),
                                  _stream(stream)), "dsa_sparse_mqa_fwd")


def dsa_dense_mqa_fwd(attn: _Keep, out: torch.Tensor, lse: Optional[torch.Tensor] = None,
                      stream=None):
    _check(LIB.dsa_dense_mqa_fwd(ctypes.byref(attn.struct), _ptr(out), _ptr(lse),
                                 _stream(stream)), "dsa_dense_mqa_fwd")


def dsa_select_scored(ind: _Keep, k: int, idx: torch.Tensor, sel_scores: torch.Tensor,
                      ws: torch.Tensor, stream=None):
    _check(LIB.dsa_select_scored(ctypes.byref(ind.struct), k, _ptr(idx), idx.stride(0),
                                 _ptr(sel_scores), sel_scores.stride(0), _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)),
           "dsa_select_scored")


def dsa_indexer_kl(attn: _Keep, idx: torch.Tensor, k: int, lse: torch.Tensor,
                   sel_scores: torch.Tensor, loss: torch.Tensor, grad: torch.Tensor,
                   stream=None):
    _check(LIB.dsa_indexer_kl(ctypes.byref(attn.struct), _ptr(idx), idx.stride(0), k, _ptr(lse),
                              _ptr(sel_scores), sel_scores.stride(0), _ptr(loss), _ptr(grad),
                              grad.stride(0), _stream(stream)), "dsa_indexer_kl")


def dsa_sparse_mqa_bwd(attn: _Keep, idx: torch.Tensor, k: int, out: torch.Tensor,
                       lse: torch.Tensor, d_out: torch.Tensor, d_q: torch.Tensor,
                       d_kv: torch.Tensor, delta: torch.Tensor, stream=None):
    """Gradient of dsa_sparse_mqa_fwd: writes d_q and delta, ADDS into d_kv."""
    _check(LIB.dsa_sparse_mqa_bwd(ctypes.byref(attn.struct), _ptr(idx), idx.stride(0), k,
                                  _ptr(out), _ptr(lse), _ptr(d_out), _ptr(d_q), _ptr(d_kv),
                                  d_kv.stride(0), _ptr(delta), _stream(stream)),
           "dsa_sparse_mqa_bwd")


def dsa_kv8_store(cache: _Keep, rows: torch.Tensor, cu_rows: Optional[torch.Tensor] = None,
                  stream=None):
    """Quantises rows [n, 576] (bf16 or float32) into the cache as the newest
    tokens: rows cu_rows[b]..cu_rows[b+1]-1 of each sequence b, one row per
    sequence without cu_rows, or the last n rows of a contiguous cache."""
    dtype, shape, stride = rows.dtype, rows.shape, rows.stride()
    if dtype is not _BF16 and dtype is not _F32:
        raise DsaError(DSA_ERR_UNSUPPORTED, f"dsa_kv8_store: rows of {dtype}")
    if len(shape) != 2 or shape[1] != 576 or stride[1] != 1:
        raise DsaError(DSA_ERR_INVALID_ARG, "dsa_kv8_store: rows must be [n, 576], each row contiguous")
    dev = rows.get_device()
    if dev != cache.dev:
        dev = -1
    if cu_rows is not None:
        n = cache.sizes[0] + 1
        if not (cu_rows.dtype is _I32 and cu_rows.numel() >= n and cu_rows.is_contiguous()):
            _flat(cu_rows, _I32, n, "dsa_kv8_store: cu_rows")
        if cu_rows.get_device() != dev:
            dev = -1
    _check(LIB.dsa_kv8_store(ctypes.byref(cache.struct), DSA_BF16 if dtype is _BF16 else DSA_F32,
                             rows.data_ptr(), stride[0], _ptr(cu_rows), shape[0],
                             _stream_on(dev, stream, "dsa_kv8_store")), "dsa_kv8_store")


def _kv8_reads(attn: _Keep, kv_exp, idx, k, lse, ws, what: str):
    """Checks what attention and its weights are given alike; the device, or -1."""
    if attn.sizes is None:
        _need(attn.tensors[1], _U8, what + ": kv")
    n_q, n_lse, blocks, _, _ = attn.sizes
    dev = attn.dev
    if not (kv_exp.dtype is _I8 and kv_exp.numel() >= blocks and kv_exp.is_contiguous()):
        _flat(kv_exp, _I8, blocks, what + ": kv_exp")
    if not ws.is_contiguous():
        _flat(ws, ws.dtype, 0, what + ": ws")
    ok = kv_exp.get_device() == dev and ws.get_device() == dev
    if lse is not None:
        if not (lse.dtype is _F32 and lse.numel() >= n_lse and lse.is_contiguous()):
            _flat(lse, _F32, n_lse, what + ": lse")
        ok = ok and lse.get_device() == dev
    if idx is not None:
        if not (idx.dtype is _I32 and idx.dim() == 2 and idx.shape[0] >= n_q and idx.shape[1] >= k and
                idx.stride()[1] == 1):
            _matrix(idx, _I32, n_q, k, what + ": idx")
        ok = ok and idx.get_device() == dev
    return dev if ok else -1


def dsa_kv8_mqa_fwd(attn: _Keep, kv_exp: torch.Tensor, idx: Optional[torch.Tensor], k: int,
                    out: torch.Tensor, lse: Optional[torch.Tensor], ws: torch.Tensor,
                    stream=None):
    """Attention over the 8-bit cache: attn from attn_in with the codes as kv;
    idx None (k 0): every preceding key."""
    dev = _kv8_reads(attn, kv_exp, idx, k, lse, ws, "dsa_kv8_mqa_fwd")
    n = attn.sizes[1] * 512
    if not (out.dtype is _BF16 and out.numel() >= n and out.is_contiguous()):
        _flat(out, _BF16, n, "dsa_kv8_mqa_fwd: out")
    if out.get_device() != dev:
        dev = -1
    _check(LIB.dsa_kv8_mqa_fwd(ctypes.byref(attn.struct), kv_exp.data_ptr(), _ptr(idx),
                               0 if idx is None else idx.stride()[0], k, out.data_ptr(), _ptr(lse),
                               ws.data_ptr(), ws.numel() * ws.element_size(),
                               _stream_on(dev, stream, "dsa_kv8_mqa_fwd")), "dsa_kv8_mqa_fwd")


def dsa_kv8_accumulate(attn: _Keep, kv_exp: torch.Tensor, idx: Optional[torch.Tensor], k: int,
                       lse: torch.Tensor, decay: float, acc: torch.Tensor, ws: torch.Tensor,
                       stream=None):
    """acc [n_seq, >= keys] = decay * acc + each cached token's attention weight."""
    dev = _kv8_reads(attn, kv_exp, idx, k, lse, ws, "dsa_kv8_accumulate")
    shape, stride, n = acc.shape, acc.stride(), attn.sizes
    if not (acc.dtype is _F32 and len(shape) == 2 and shape[0] >= n[3] and shape[1] >= n[4] and stride[1] == 1):
        _matrix(acc, _F32, n[3], n[4], "dsa_kv8_accumulate: acc")
    if acc.get_device() != dev:
        dev = -1
    _check(LIB.dsa_kv8_accumulate(ctypes.byref(attn.struct), kv_exp.data_ptr(), _ptr(idx),
                                  0 if idx is None else idx.stride()[0], k, _ptr(lse), decay,
                                  acc.data_ptr(), stride[0], ws.data_ptr(),
                                  ws.numel() * ws.element_size(),
                                  _stream_on(dev, stream, "dsa_kv8_accumulate")), "dsa_kv8_accumulate")


def dsa_kv8_evict(cache: _Keep, acc: torch.Tensor, budget: int, sink: int, recent: int,
                  dst_table: torch.Tensor, new_lens: torch.Tensor, kept: torch.Tensor,
                  acc_out: torch.Tensor, idx_codes: Optional[torch.Tensor] = None,
                  idx_scales: Optional[torch.Tensor] = None, stream=None):
    """Keeps `budget` tokens of each sequence and moves them into the pages of
    dst_table; optionally the indexer's key cache (codes [pages, 64, 128], scales
    [pages, 64]) along with them."""
    n, keys, pages = cache.sizes
    sa, sd, sk, so = acc.shape, dst_table.shape, kept.shape, acc_out.shape
    ta, td, tk, to = acc.stride(), dst_table.stride(), kept.stride(), acc_out.stride()
    if not (acc.dtype is _F32 and acc_out.dtype is _F32 and dst_table.dtype is _I32 and kept.dtype is _I32 and
            new_lens.dtype is _I32 and new_lens.numel() >= n and new_lens.is_contiguous() and
            len(sa) == len(sd) == len(sk) == len(so) == 2 and min(sa[0], sd[0], sk[0], so[0]) >= n and
            sa[1] >= keys and 64 * sd[1] >= budget <= sk[1] and budget <= so[1] and
            ta[1] == td[1] == tk[1] == to[1] == 1):
        _matrix(acc, _F32, n, keys, "dsa_kv8_evict: acc")
        _matrix(dst_table, _I32, n, -(-budget // 64), "dsa_kv8_evict: dst_table")
        _flat(new_lens, _I32, n, "dsa_kv8_evict: new_lens")
        _matrix(kept, _I32, n, budget, "dsa_kv8_evict: kept")
        _matrix(acc_out, _F32, n, budget, "dsa_kv8_evict: acc_out")
    dev = cache.dev
    if not (acc.get_device() == dst_table.get_device() == new_lens.get_device() == kept.get_device() ==
            acc_out.get_device() == dev):
        dev = -1
    if idx_codes is not None:
        _rows(idx_codes, 128, cache.struct.kv, 0, "dsa_kv8_evict: idx_codes")
        if idx_codes.get_device() != dev:
            dev = -1
    if idx_scales is not None:
        _flat(idx_scales, _F32, pages * 64, "dsa_kv8_evict: idx_scales")
        if idx_scales.get_device() != dev:
            dev = -1
    _check(LIB.dsa_kv8_evict(ctypes.byref(cache.struct), _ptr(idx_codes),
                             0 if idx_codes is None else idx_codes.stride()[-2], _ptr(idx_scales),
                             acc.data_ptr(), ta[0], budget, sink, recent, dst_table.data_ptr(), td[0],
                             new_lens.data_ptr(), kept.data_ptr(), tk[0], acc_out.data_ptr(), to[0],
                             _stream_on(dev, stream, "dsa_kv8_evict")), "dsa_kv8_evict")


def dsa_select(ind: _Keep, k: int, idx: torch.Tensor, ws: torch.Tensor, stream=None):
    _check(LIB.dsa_select(ctypes.byref(ind.struct), k, _ptr(idx), idx.stride(0), _ptr(ws),
                          ws.numel() * ws.element_size(), _stream(stream)), "dsa_select")


def dsa_select_noalloc(ind: _Keep, k: int, idx: torch.Tensor, stream=None):
    """dsa_select without a workspace, for callers that cannot allocate device
    memory: the library's fixed 16 MiB per-GPU scratch holds the score rows.
    Calls on one device must not overlap (they share that scratch)."""
    _check(LIB.dsa_select_noalloc(ctypes.byref(ind.struct), k, _ptr(idx), idx.stride(0),
                                  _stream(stream)), "dsa_select_noalloc")


def dsa_set_wait_limit_ns(ns: int):
    """Bound of the pipeline waits of the indexer and of the 8-bit cache's attention
    and weights (ns <= 0: the 1 s default)."""
    _check(LIB.dsa_set_wait_limit_ns(int(ns)), "dsa_set_wait_limit_ns")


def dsa_launch_counter() -> int:
    return int(LIB.dsa_launch_counter())


def dsa_forward(ind: _Keep, attn: _Keep, k: int, idx_out: Optional[torch.Tensor],
                out: torch.Tensor, lse: Optional[torch.Tensor], ws: torch.Tensor, stream=None):
    _check(LIB.dsa_forward(ctypes.byref(ind.struct), ctypes.byref(attn.struct), k,
                           _ptr(idx_out), _ptr(out), _ptr(lse), _ptr(ws),
                           ws.numel() * ws.element_size(), _stream(stream)), "dsa_forward")


def dsa_check_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status."""
    return int(LIB.dsa_check_status(_stream(stream)))


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte aligned device buffer of at least nbytes (torch allocations are)."""
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
