"""GB300-native sparse MLA (DeepSeek sparse attention) hot path.

Thin Python binding of ``libhs.so`` (C ABI in ``include/hs.h``): the functions below have the
C names, take torch CUDA tensors, marshal pointers and sizes, and call the library on the
current (or given) CUDA stream. Every step of the computation runs in the library's sm_103a
kernels; there is no fallback. If the library is missing, import succeeds but every call raises
``HSError`` telling how to build it (``python -m dsa_sparse_mla_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

__all__ = ["HSError", "lib_path", "load", "hs_abi_version", "hs_check_flag", "hs_indexer_scores", "hs_topk",
           "hs_indexer_topk",
           "hs_sparse_mla_fwd", "hs_sparse_mla_workspace_size", "hs_sparse_mla_fwd_static", "hs_hisparse_resolve",
           "hs_hisparse_touch_host", "hs_kv_append", "hs_kv_offload", "hs_rope", "hs_rope_inv_freq", "hs_paged_mla_fwd",
           "hs_paged_mla_workspace_size", "hs_kv_copy_pages", "hs_kv_fork", "hs_kv_free", "hs_kv_compact",
           "hs_kv_compact_workspace_size", "FLAGS"]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libhs.so")
_lib = None

FLAGS = {"BAD_INDEX": 0x01, "BAD_LENGTH": 0x02, "BAD_BLOCK": 0x04, "NOT_ASCENDING": 0x08, "BAD_STATE": 0x10,
         "TIMEOUT": 0x20, "RANGE": 0x40, "NO_PAGES": 0x80}
_STATUS = {0: "HS_OK", 1: "HS_ERR_INVALID", 2: "HS_ERR_UNSUPPORTED", 3: "HS_ERR_CUDA", 4: "HS_ERR_DEVICE_FLAG",
           5: "HS_ERR_TIMEOUT"}


class HSError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("%s: %s" % (_STATUS.get(status, status), message))
        self.status = status


_P = ctypes.c_void_p
_i32, _i64, _f32, _f64 = ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_double


class _IndexerArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("B", _i32), ("Hi", _i32), ("Di", _i32), ("q", _P), ("q_scale", _P), ("weights", _P),
                ("k_cache", _P), ("k_scale", _P), ("nblk", _i64), ("block_table", _P), ("bt_stride", _i32),
                ("token_req", _P), ("token_kvlen", _P), ("scores", _P), ("ld", _i64), ("err_flag", _P)]


class _MlaArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("k", _i32), ("q", _P), ("kv_pool", _P), ("R", _i64), ("idx", _P),
                ("block_table", _P), ("bt_stride", _i32), ("token_req", _P), ("softmax_scale", _f32),
                ("out", _P), ("lse", _P), ("err_flag", _P), ("workspace", _P), ("workspace_bytes", ctypes.c_uint64),
                ("idx_row", _P), ("idx_rows", _i32), ("token_kvlen", _P)]


class _ResolveArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("k", _i32), ("S", _i32), ("step", _i32), ("idx", _P), ("seq_len", _P),
                ("resident_start", _P), ("block_table", _P), ("bt_stride", _i32), ("host_rows", _P),
                ("kv_pool", _P), ("R", _i64), ("slot_row", _P), ("slot_token", _P), ("slot_stamp", _P),
                ("tok2slot", _P), ("ld_t2s", _i64), ("out_rows", _P), ("counters", _P), ("err_flag", _P)]


def lib_path() -> str:
    return _LIB_PATH


def load():
    """Load libhs.so once. Raises HSError if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise HSError(2, "libhs.so not found at %s; build it with `python -m dsa_sparse_mla_gb300.build`"
                          % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        lib.hs_abi_version.restype = ctypes.c_int
        lib.hs_status_str.argtypes = [ctypes.c_int]
        lib.hs_status_str.restype = ctypes.c_char_p
        lib.hs_last_error.restype = ctypes.c_char_p
        lib.hs_check_flag.argtypes = [_P, _P, _P]
        lib.hs_indexer_scores.argtypes = [ctypes.POINTER(_IndexerArgs), _P]
        lib.hs_topk.argtypes = [_P, _i64, _P, _i32, _i32, _P, _P, _P]
        lib.hs_indexer_topk.argtypes = [ctypes.POINTER(_IndexerArgs), _i32, _P, _P]
        lib.hs_sparse_mla_fwd.argtypes = [ctypes.POINTER(_MlaArgs), _P]
        lib.hs_sparse_mla_workspace_size.argtypes = [_i32, ctypes.POINTER(ctypes.c_uint64)]
        lib.hs_sparse_mla_fwd_static.argtypes = [ctypes.POINTER(_MlaArgs), _P]
        lib.hs_hisparse_resolve.argtypes = [ctypes.POINTER(_ResolveArgs), _P]
        lib.hs_hisparse_touch_host.argtypes = [_i32, _P, _P, _P, _P, _P]
        lib.hs_kv_append.argtypes = [ctypes.POINTER(_AppendArgs), _P]
        lib.hs_kv_offload.argtypes = [ctypes.POINTER(_OffloadArgs), _P]
        lib.hs_rope.argtypes = [_P, _P]
        lib.hs_rope_inv_freq.argtypes = [_i32, _f64, _i32, _f64, _i32, _f64, _f64, _P, _P]
        lib.hs_paged_mla_fwd.argtypes = [_P, _P]
        lib.hs_paged_mla_workspace_size.argtypes = [_i32, _i32, _i32, _i64, ctypes.POINTER(ctypes.c_uint64)]
        lib.hs_kv_copy_pages.argtypes = [_P, _P]
        lib.hs_kv_fork.argtypes = [_P, _P]
        lib.hs_kv_free.argtypes = [_P, _P]
        lib.hs_kv_compact.argtypes = [_P, _P]
        lib.hs_kv_compact_workspace_size.argtypes = [_i64, ctypes.POINTER(ctypes.c_uint64)]
        for f in ("hs_rope", "hs_rope_inv_freq", "hs_paged_mla_fwd", "hs_paged_mla_workspace_size", "hs_kv_copy_pages", "hs_kv_fork",
                  "hs_kv_free", "hs_kv_compact", "hs_kv_compact_workspace_size"):
            getattr(lib, f).restype = ctypes.c_int
        for f in ("hs_check_flag", "hs_indexer_scores", "hs_topk", "hs_indexer_topk", "hs_sparse_mla_fwd", "hs_sparse_mla_workspace_size",
                  "hs_sparse_mla_fwd_static", "hs_hisparse_resolve", "hs_hisparse_touch_host", "hs_kv_append", "hs_kv_offload"):
            getattr(lib, f).restype = ctypes.c_int
        _lib = lib
    return _lib


def _check(status: int):
    if status:
        raise HSError(status, load().hs_last_error().decode(errors="replace"))


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _dev(t, name, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise HSError(1, "%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise HSError(1, "%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise HSError(1, "%s must be %s (got %s)" % (name, dtype, t.dtype))
    return t


def _stream(stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


_CODES = {_P: "P", _i32: "i", _i64: "q", _f32: "f", _f64: "d", ctypes.c_uint64: "Q"}


def _packer(cls):
    """Packs an args struct's fields (pointers as integers, 0 for none) into bytes of its C layout, which a call reads in
    place: a few times cheaper than filling the ctypes structure."""
    return struct.Struct("@" + "".join(_CODES[t] for _, t in cls._fields_) + "0P").pack


def _tensor(t, name, dtype):
    """The address of a contiguous CUDA tensor of this type."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise HSError(1, "%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise HSError(1, "%s must be %s (got %s)" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise HSError(1, "%s must be contiguous" % name)
    return t.data_ptr()


def hs_abi_version() -> int:
    return int(load().hs_abi_version())


def hs_check_flag(err_flag: torch.Tensor, stream=None) -> int:
    """Synchronise `stream` and return the raw device error bits (0 = none)."""
    out = ctypes.c_int32(0)
    st = load().hs_check_flag(_ptr(_dev(err_flag, "err_flag", torch.int32)), ctypes.addressof(out), _stream(stream))
    if st not in (0, 4, 5):
        _check(st)
    return int(out.value)


def _indexer_args(q, q_scale, weights, k_cache, k_scale, block_table, token_req, token_kvlen, scores, err_flag,
                  num_requests):
    _dev(q, "q", torch.uint8), _dev(q_scale, "q_scale", torch.float32), _dev(weights, "weights", torch.float32)
    _dev(k_cache, "k_cache", torch.uint8), _dev(k_scale, "k_scale", torch.float32)
    _dev(block_table, "block_table", torch.int32), _dev(token_req, "token_req", torch.int32)
    _dev(token_kvlen, "token_kvlen", torch.int32), _dev(scores, "scores", torch.float32)
    _dev(err_flag, "err_flag", torch.int32)
    T, Hi, Di = q.shape
    return _IndexerArgs(T, num_requests if num_requests is not None else block_table.shape[0], Hi, Di, _ptr(q),
                        _ptr(q_scale), _ptr(weights), _ptr(k_cache), _ptr(k_scale), k_cache.shape[0],
                        _ptr(block_table), block_table.shape[1], _ptr(token_req), _ptr(token_kvlen), _ptr(scores),
                        scores.shape[1], _ptr(err_flag))


def hs_indexer_scores(q, q_scale, weights, k_cache, k_scale, block_table, token_req, token_kvlen, scores, err_flag,
                      num_requests: int | None = None, stream=None):
    """Lightning-indexer scores into ``scores`` (float32 [T, ld]); see include/hs.h."""
    a = _indexer_args(q, q_scale, weights, k_cache, k_scale, block_table, token_req, token_kvlen, scores, err_flag,
                      num_requests)
    _check(load().hs_indexer_scores(ctypes.byref(a), _stream(stream)))


def hs_indexer_topk(q, q_scale, weights, k_cache, k_scale, block_table, token_req, token_kvlen, scores, k: int, idx,
                    err_flag, num_requests: int | None = None, stream=None):
    """Indexer scores and their top-k in one call (``scores`` is scratch, undefined afterwards);
    the indices go to ``idx`` (int32 [T, k]), as hs_indexer_scores + hs_topk would write them."""
    a = _indexer_args(q, q_scale, weights, k_cache, k_scale, block_table, token_req, token_kvlen, scores, err_flag,
                      num_requests)
    _dev(idx, "idx", torch.int32)
    if tuple(idx.shape) != (q.shape[0], k):
        raise HSError(1, "idx must have shape [T, k]")
    _check(load().hs_indexer_topk(ctypes.byref(a), k, _ptr(idx), _stream(stream)))


def hs_topk(scores, token_kvlen, k: int, idx, err_flag, stream=None):
    """Top-k indices (ascending, -1 padded) into ``idx`` (int32 [T, k])."""
    _dev(scores, "scores", torch.float32), _dev(token_kvlen, "token_kvlen", torch.int32)
    _dev(idx, "idx", torch.int32), _dev(err_flag, "err_flag", torch.int32)
    T, ld = scores.shape
    if idx.shape != (T, k):
        raise HSError(1, "idx must have shape [T, k]")
    _check(load().hs_topk(_ptr(scores), ld, _ptr(token_kvlen), T, k, _ptr(idx), _ptr(err_flag), _stream(stream)))


def hs_sparse_mla_workspace_size(H: int) -> int:
    """Bytes of workspace hs_sparse_mla_fwd needs for H heads on the current device."""
    n = ctypes.c_uint64(0)
    _check(load().hs_sparse_mla_workspace_size(int(H), ctypes.byref(n)))
    return int(n.value)


def _mla_args(q, kv_pool, idx, softmax_scale, out, err_flag, lse, block_table, token_req, workspace, idx_row,
              token_kvlen):
    _dev(q, "q", torch.bfloat16), _dev(kv_pool, "kv_pool", torch.uint8), _dev(idx, "idx", torch.int32)
    _dev(workspace, "workspace", torch.uint8)
    _dev(out, "out", torch.bfloat16), _dev(err_flag, "err_flag", torch.int32), _dev(lse, "lse", torch.float32)
    _dev(block_table, "block_table", torch.int32), _dev(token_req, "token_req", torch.int32)
    _dev(idx_row, "idx_row", torch.int32), _dev(token_kvlen, "token_kvlen", torch.int32)
    T, H, D = q.shape
    if D != 576 or kv_pool.shape[-1] != 656 or out.shape != (T, H, 512) or (idx_row is None and idx.shape[0] != T):
        raise HSError(1, "shape mismatch: q [T,H,576], kv_pool [R,656], idx [T,k] (or [rows,k] with idx_row), "
                         "out [T,H,512]")
    for t, n in ((idx_row, "idx_row"), (token_kvlen, "token_kvlen")):
        if t is not None and t.shape != (T,):
            raise HSError(1, "%s must be int32 [T]" % n)
    return _MlaArgs(T, H, idx.shape[1], _ptr(q), _ptr(kv_pool), kv_pool.shape[0], _ptr(idx), _ptr(block_table),
                    0 if block_table is None else block_table.shape[1], _ptr(token_req), float(softmax_scale),
                    _ptr(out), _ptr(lse), _ptr(err_flag), _ptr(workspace),
                    0 if workspace is None else workspace.numel(), _ptr(idx_row), idx.shape[0], _ptr(token_kvlen))


def hs_sparse_mla_fwd(q, kv_pool, idx, softmax_scale: float, out, err_flag, lse=None, block_table=None,
                      token_req=None, workspace=None, stream=None, idx_row=None, token_kvlen=None):
    """Sparse MLA forward: ``out`` bf16 [T, H, 512] (and ``lse`` float32 [T, H] if given). With a
    ``workspace`` (uint8 CUDA tensor of at least hs_sparse_mla_workspace_size(H) bytes) every SM
    gets an equal share of the work and split queries are merged by log-sum-exp. Shared index sets:
    ``idx_row`` (int32 [T]) names the row of ``idx`` each query reads, and ``token_kvlen`` (int32
    [T], with a block table) skips the entries a query may not see."""
    a = _mla_args(q, kv_pool, idx, softmax_scale, out, err_flag, lse, block_table, token_req, workspace, idx_row,
                  token_kvlen)
    _check(load().hs_sparse_mla_fwd(ctypes.byref(a), _stream(stream)))


def hs_sparse_mla_fwd_static(q, kv_pool, idx, softmax_scale: float, out, err_flag, lse=None, block_table=None,
                             token_req=None, stream=None, idx_row=None, token_kvlen=None):
    """hs_sparse_mla_fwd for callers that cannot allocate device memory: the split-work scratch is
    the library's own fixed device array (see include/hs.h), so no workspace is passed."""
    a = _mla_args(q, kv_pool, idx, softmax_scale, out, err_flag, lse, block_table, token_req, None, idx_row,
                  token_kvlen)
    _check(load().hs_sparse_mla_fwd_static(ctypes.byref(a), _stream(stream)))


def hs_hisparse_resolve(step: int, idx, seq_len, resident_start, block_table, host_rows, kv_pool, slot_row,
                        slot_token, slot_stamp, tok2slot, out_rows, counters, err_flag, stream=None):
    """One HiSparse resolve step. ``host_rows`` is an int64 CUDA tensor [B] of device-accessible
    pointers to each request's pinned host rows [seq_len, 656]."""
    for t, n, dt in ((idx, "idx", torch.int32), (seq_len, "seq_len", torch.int32),
                     (resident_start, "resident_start", torch.int32), (block_table, "block_table", torch.int32),
                     (host_rows, "host_rows", torch.int64), (kv_pool, "kv_pool", torch.uint8),
                     (slot_row, "slot_row", torch.int32), (slot_token, "slot_token", torch.int32),
                     (slot_stamp, "slot_stamp", torch.int32), (tok2slot, "tok2slot", torch.int32),
                     (out_rows, "out_rows", torch.int32), (counters, "counters", torch.int32),
                     (err_flag, "err_flag", torch.int32)):
        _dev(t, n, dt)
    B, k = idx.shape
    a = _ResolveArgs(B, k, slot_row.shape[1], int(step), _ptr(idx), _ptr(seq_len), _ptr(resident_start),
                     _ptr(block_table), block_table.shape[1], _ptr(host_rows), _ptr(kv_pool), kv_pool.shape[0],
                     _ptr(slot_row), _ptr(slot_token), _ptr(slot_stamp), _ptr(tok2slot), tok2slot.shape[1],
                     _ptr(out_rows), _ptr(counters), _ptr(err_flag))
    _check(load().hs_hisparse_resolve(ctypes.byref(a), _stream(stream)))


def hs_hisparse_touch_host(host_rows, seq_len, resident_start, err_flag, stream=None):
    """Read one word of every host page of each request's offloaded rows, so that the GPU's
    first-access cost for the host tier is paid here rather than inside a resolve.
    ``host_rows`` is the int64 CUDA tensor [B] of pointers that hs_hisparse_resolve takes."""
    for t, n, dt in ((host_rows, "host_rows", torch.int64), (seq_len, "seq_len", torch.int32),
                     (resident_start, "resident_start", torch.int32), (err_flag, "err_flag", torch.int32)):
        _dev(t, n, dt)
    B = host_rows.shape[0]
    if seq_len.shape[0] != B or resident_start.shape[0] != B:
        raise HSError(1, "host_rows, seq_len and resident_start must have the same length")
    _check(load().hs_hisparse_touch_host(B, _ptr(host_rows), _ptr(seq_len), _ptr(resident_start), _ptr(err_flag),
                                         _stream(stream)))


class _AppendArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("B", _i32), ("latent", _P), ("rope", _P), ("index_key", _P), ("Di", _i32),
                ("token_req", _P), ("token_pos", _P), ("block_table", _P), ("bt_stride", _i32),
                ("kv_pool", _P), ("R", _i64), ("k_cache", _P), ("k_scale", _P), ("nblk", _i64), ("err_flag", _P)]


def hs_kv_append(token_req, token_pos, block_table, err_flag, latent=None, rope=None, kv_pool=None,
                 index_key=None, k_cache=None, k_scale=None, stream=None):
    """Quantise new tokens into the paged FP8 layouts (see include/hs.h). ``latent`` / ``rope`` are
    bf16 [T, 512] / [T, 64] written into ``kv_pool`` (uint8 [R, 656]); ``index_key`` is bf16 [T, Di]
    written into ``k_cache`` (uint8 [nblk, 64, Di]) and ``k_scale`` (float32 [nblk, 64])."""
    _dev(token_req, "token_req", torch.int32), _dev(token_pos, "token_pos", torch.int32)
    _dev(block_table, "block_table", torch.int32), _dev(err_flag, "err_flag", torch.int32)
    a = _AppendArgs()
    a.T, a.B = token_req.shape[0], block_table.shape[0]
    if latent is not None:
        _dev(latent, "latent", torch.bfloat16), _dev(rope, "rope", torch.bfloat16), _dev(kv_pool, "kv_pool", torch.uint8)
        a.latent, a.rope, a.kv_pool, a.R = _ptr(latent), _ptr(rope), _ptr(kv_pool), kv_pool.shape[0]
    if index_key is not None:
        _dev(index_key, "index_key", torch.bfloat16), _dev(k_cache, "k_cache", torch.uint8)
        _dev(k_scale, "k_scale", torch.float32)
        a.index_key, a.Di, a.k_cache, a.k_scale, a.nblk = _ptr(index_key), index_key.shape[1], _ptr(k_cache), \
            _ptr(k_scale), k_cache.shape[0]
    a.token_req, a.token_pos, a.block_table, a.bt_stride = _ptr(token_req), _ptr(token_pos), _ptr(block_table), \
        block_table.shape[1]
    a.err_flag = _ptr(err_flag)
    _check(load().hs_kv_append(ctypes.byref(a), _stream(stream)))


class _OffloadArgs(ctypes.Structure):
    _fields_ = [("n", _i32), ("L", _i32), ("B", _i32), ("pools", _P), ("R", _i64), ("host_rows", _P), ("layer", _P),
                ("req", _P), ("page", _P), ("block_table", _P), ("bt_stride", _i32), ("seq_len", _P), ("err_flag", _P)]


def hs_kv_offload(pools, host_rows, layer, req, page, block_table, seq_len, err_flag, R: int, stream=None):
    """Copy complete KV pages to the host tier (see include/hs.h). ``pools`` is an int64 CUDA tensor
    [L] of device pointers to each layer's pool (uint8 [R, 656]); ``host_rows`` an int64 CUDA tensor
    [L * B] of device-accessible pointers to pinned host rows, indexed layer * B + request."""
    for t, nm, dt in ((pools, "pools", torch.int64), (host_rows, "host_rows", torch.int64), (layer, "layer", torch.int32),
                      (req, "req", torch.int32), (page, "page", torch.int32), (block_table, "block_table", torch.int32),
                      (seq_len, "seq_len", torch.int32), (err_flag, "err_flag", torch.int32)):
        _dev(t, nm, dt)
    a = _OffloadArgs()
    a.n, a.L, a.B = layer.shape[0], pools.shape[0], block_table.shape[0]
    if host_rows.shape[0] != a.L * a.B:
        raise HSError(1, "host_rows must hold L * B pointers")
    a.pools, a.R, a.host_rows = _ptr(pools), int(R), _ptr(host_rows)
    a.layer, a.req, a.page = _ptr(layer), _ptr(req), _ptr(page)
    a.block_table, a.bt_stride, a.seq_len, a.err_flag = _ptr(block_table), block_table.shape[1], _ptr(seq_len), _ptr(err_flag)
    _check(load().hs_kv_offload(ctypes.byref(a), _stream(stream)))


class _RopeArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("H2", _i32), ("rot", _i32), ("dtype", _i32), ("interleaved", _i32),
                ("inverse", _i32), ("scale", _f32), ("positions", _P), ("inv_freq", _P), ("x", _P), ("x_stride_t", _i64),
                ("x_stride_h", _i64), ("out", _P), ("out_stride_t", _i64), ("out_stride_h", _i64), ("y", _P),
                ("y_stride_t", _i64), ("y_stride_h", _i64), ("y_out", _P), ("y_out_stride_t", _i64),
                ("y_out_stride_h", _i64)]


_pack_rope = _packer(_RopeArgs)
_ROPE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ROPE_KINDS = {"plain": 0, "linear": 1, "yarn": 2}


def hs_rope_inv_freq(rot: int, base: float = 10000.0, kind: str = "plain", factor: float = 1.0, original: int = 4096,
                     beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Angles per position of each pair (float64 CPU tensor [rot / 2]) and the scale hs_rope takes; ``kind`` is
    "plain", "linear" or "yarn" (contexts ``factor`` times ``original``). Host only."""
    if kind not in _ROPE_KINDS:
        raise HSError(1, "kind must be one of %s" % ", ".join(_ROPE_KINDS))
    f, s = torch.empty(max(int(rot) // 2, 1), dtype=torch.float64), ctypes.c_float(1.0)
    _check(load().hs_rope_inv_freq(int(rot), float(base), _ROPE_KINDS[kind], float(factor), int(original), float(beta_fast),
                                   float(beta_slow), f.data_ptr(), ctypes.addressof(s)))
    return f, float(s.value)


def _rope_tensor(t, name, T, rot, dtype):
    """Address, token and head strides and heads of a [T, heads, rot] tensor whose heads are consecutive values."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not dtype or t.dim() != 3:
        raise HSError(1, "%s must be a %s CUDA tensor [T, heads, rot]" % (name, dtype))
    (n, heads, r), (a, b, c) = t.shape, t.stride()
    if n != T or r != rot or c != 1:
        raise HSError(1, "%s must be [T, heads, rot] with consecutive values in a head" % name)
    return t.data_ptr(), a, b, heads


def hs_rope(x, positions, inv_freq, out=None, y=None, y_out=None, interleaved: bool = False, scale: float = 1.0,
            inverse: bool = False, stream=None):
    """Rotary positions of ``x`` ([T, H, rot], bf16, fp16 or fp32: a slice of wider heads may be given) into ``out``
    (``x`` itself when None), and in the same launch of ``y`` ([T, H2, rot]) into ``y_out``. ``positions`` is int32 [T],
    ``inv_freq`` float64 [rot / 2] on the GPU (see hs_rope_inv_freq)."""
    dtype = x.dtype if isinstance(x, torch.Tensor) else None
    if dtype not in _ROPE_DTYPES or x.dim() != 3:
        raise HSError(1, "x must be a bf16, fp16 or fp32 CUDA tensor [T, H, rot]")
    T, _, rot = x.shape
    xp, xt, xh, H = _rope_tensor(x, "x", T, rot, dtype)
    op, ot, oh, H1 = (xp, xt, xh, H) if out is None else _rope_tensor(out, "out", T, rot, dtype)
    pos, inv = _tensor(positions, "positions", torch.int32), _tensor(inv_freq, "inv_freq", torch.float64)
    if H1 != H or positions.numel() != T or inv_freq.numel() != rot // 2:
        raise HSError(1, "shape mismatch: out [T, H, rot], positions [T], inv_freq [rot / 2]")
    yp = yt = yh = H2 = zp = zt = zh = 0
    if y is not None:
        yp, yt, yh, H2 = _rope_tensor(y, "y", T, rot, dtype)
        zp, zt, zh, H3 = (yp, yt, yh, H2) if y_out is None else _rope_tensor(y_out, "y_out", T, rot, dtype)
        if H3 != H2:
            raise HSError(1, "shape mismatch: y_out has other heads than y")
    _check(load().hs_rope(_pack_rope(T, H, H2, rot, _ROPE_DTYPES[dtype], 1 if interleaved else 0, 1 if inverse else 0, scale, pos,
                                     inv, xp, xt, xh, op, ot, oh, yp, yt, yh, zp, zt, zh), _stream(stream)))


class _PagedMlaArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("B", _i32), ("H", _i32), ("causal", _i32), ("q", _P), ("kv_pool", _P), ("R", _i64),
                ("block_table", _P), ("bt_stride", _i32), ("req_start", _P), ("seq_len", _P), ("kv_tokens", _i64),
                ("softmax_scale", _f32), ("out", _P), ("lse", _P), ("err_flag", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_uint64)]


_pack_paged_mla = _packer(_PagedMlaArgs)


def hs_paged_mla_workspace_size(T: int, B: int, H: int, kv_tokens: int) -> int:
    """Bytes of workspace hs_paged_mla_fwd needs for at most these sizes on the current device."""
    n = ctypes.c_uint64(0)
    _check(load().hs_paged_mla_workspace_size(int(T), int(B), int(H), int(kv_tokens), ctypes.byref(n)))
    return int(n.value)


def hs_paged_mla_fwd(q, kv_pool, block_table, req_start, seq_len, kv_tokens: int, softmax_scale: float, out, err_flag,
                     workspace, lse=None, causal: bool = True, stream=None):
    """Dense attention of each request's new tokens over its paged rows: ``out`` bf16 [T, H, 512] (and ``lse`` float32
    [T, H] if given). Request r's tokens are ``req_start[r] .. req_start[r + 1] - 1`` (int32 [B + 1]); its cache holds
    ``seq_len[r]`` rows (int32 [B]), theirs last; ``kv_tokens`` bounds the sum of seq_len. See include/hs.h."""
    qp, kp, bp = _tensor(q, "q", torch.bfloat16), _tensor(kv_pool, "kv_pool", torch.uint8), _tensor(block_table, "block_table", torch.int32)
    rp, sp = _tensor(req_start, "req_start", torch.int32), _tensor(seq_len, "seq_len", torch.int32)
    op, ep, wp = _tensor(out, "out", torch.bfloat16), _tensor(err_flag, "err_flag", torch.int32), _tensor(workspace, "workspace", torch.uint8)
    lp = 0 if lse is None else _tensor(lse, "lse", torch.float32)
    (T, H, D), (B, pages), (R, row) = q.shape, block_table.shape, kv_pool.shape
    if D != 576 or row != 656 or out.shape != (T, H, 512) or req_start.numel() != B + 1 or seq_len.numel() != B \
            or (lse is not None and lse.shape != (T, H)):
        raise HSError(1, "shape mismatch: q [T,H,576], kv_pool [R,656], block_table [B,pages], req_start [B+1], seq_len [B], "
                         "out [T,H,512], lse [T,H]")
    _check(load().hs_paged_mla_fwd(_pack_paged_mla(T, B, H, 1 if causal else 0, qp, kp, R, bp, pages, rp, sp, kv_tokens, softmax_scale,
                                                   op, lp, ep, wp, workspace.numel()), _stream(stream)))


class _CopyArgs(ctypes.Structure):
    _fields_ = [("n", _i32), ("L", _i32), ("Li", _i32), ("Di", _i32), ("src", _P), ("dst", _P), ("rows", _P), ("nblk", _i64),
                ("pools", _P), ("k_caches", _P), ("k_scales", _P), ("err_flag", _P)]


class _ForkArgs(ctypes.Structure):
    _fields_ = [("n", _i32), ("B", _i32), ("bt_stride", _i32), ("L", _i32), ("Li", _i32), ("Di", _i32), ("parent", _P),
                ("child", _P), ("block_table", _P), ("seq_len", _P), ("refcount", _P), ("nblk", _i64), ("src", _P), ("dst", _P),
                ("pools", _P), ("k_caches", _P), ("k_scales", _P), ("err_flag", _P)]


class _FreeArgs(ctypes.Structure):
    _fields_ = [("n", _i32), ("B", _i32), ("bt_stride", _i32), ("req", _P), ("block_table", _P), ("seq_len", _P),
                ("refcount", _P), ("nblk", _i64), ("err_flag", _P)]


class _CompactArgs(ctypes.Structure):
    _fields_ = [("B", _i32), ("bt_stride", _i32), ("L", _i32), ("Li", _i32), ("Di", _i32), ("block_table", _P),
                ("refcount", _P), ("nblk", _i64), ("table_out", _P), ("refcount_out", _P), ("src", _P), ("dst", _P),
                ("counts", _P), ("pools", _P), ("k_caches", _P), ("k_scales", _P), ("workspace", _P),
                ("workspace_bytes", ctypes.c_uint64), ("err_flag", _P)]


_pack_copy, _pack_fork, _pack_free, _pack_compact = (_packer(c) for c in (_CopyArgs, _ForkArgs, _FreeArgs, _CompactArgs))


def _layers(pools, k_caches, k_scales):
    """L, Li and the addresses of the three pointer arrays."""
    L, pp = (0, 0) if pools is None else (pools.numel(), _tensor(pools, "pools", torch.int64))
    Li, cp = (0, 0) if k_caches is None else (k_caches.numel(), _tensor(k_caches, "k_caches", torch.int64))
    Ls, sp = (0, 0) if k_scales is None else (k_scales.numel(), _tensor(k_scales, "k_scales", torch.int64))
    if Li != Ls:
        raise HSError(1, "k_caches and k_scales must have the same length")
    return L, Li, pp, cp, sp


def _int(t, name):
    return _tensor(t, name, torch.int32)


def hs_kv_copy_pages(src, dst, nblk: int, err_flag, rows=None, pools=None, k_caches=None, k_scales=None, Di: int = 128,
                     stream=None):
    """Rows 0 .. rows[i] - 1 (all 64 when ``rows`` is None) of page ``src[i]`` to page ``dst[i]`` in every layer.
    ``pools`` is an int64 CUDA tensor [L] of device pointers to the latent pools, ``k_caches`` / ``k_scales`` [Li] to the
    indexer caches and their scales."""
    n = src.numel()
    if dst.numel() != n or (rows is not None and rows.numel() != n):
        raise HSError(1, "src, dst and rows must have the same length")
    L, Li, pp, cp, sp = _layers(pools, k_caches, k_scales)
    _check(load().hs_kv_copy_pages(_pack_copy(n, L, Li, Di, _int(src, "src"), _int(dst, "dst"), 0 if rows is None else _int(rows, "rows"),
                                              nblk, pp, cp, sp, _int(err_flag, "err_flag")), _stream(stream)))


def hs_kv_fork(parent, child, block_table, seq_len, refcount, src, dst, err_flag, pools=None, k_caches=None, k_scales=None,
               Di: int = 128, stream=None):
    """Requests ``child[i]`` become copies of ``parent[i]``: complete pages are shared, the last, partial one is copied
    to the lowest free page in every layer. ``block_table`` [B, pages], ``seq_len`` [B] and ``refcount`` [nblk] are updated
    in place; ``src`` / ``dst`` (int32 [n]) receive the pages copied and taken. See include/hs.h."""
    n, (B, pages) = parent.numel(), block_table.shape
    if child.numel() != n or src.numel() != n or dst.numel() != n or seq_len.numel() != B:
        raise HSError(1, "parent, child, src and dst must have the same length, and seq_len one entry per request")
    L, Li, pp, cp, sp = _layers(pools, k_caches, k_scales)
    _check(load().hs_kv_fork(_pack_fork(n, B, pages, L, Li, Di, _int(parent, "parent"), _int(child, "child"),
                                        _int(block_table, "block_table"), _int(seq_len, "seq_len"), _int(refcount, "refcount"),
                                        refcount.numel(), _int(src, "src"), _int(dst, "dst"), pp, cp, sp,
                                        _int(err_flag, "err_flag")), _stream(stream)))


def hs_kv_free(req, block_table, seq_len, refcount, err_flag, stream=None):
    """Requests ``req[i]`` give their pages back (``refcount`` - 1 each) and become empty, in place."""
    B, pages = block_table.shape
    if seq_len.numel() != B:
        raise HSError(1, "seq_len must have one entry per request")
    _check(load().hs_kv_free(_pack_free(req.numel(), B, pages, _int(req, "req"), _int(block_table, "block_table"), _int(seq_len, "seq_len"),
                                        _int(refcount, "refcount"), refcount.numel(), _int(err_flag, "err_flag")), _stream(stream)))


def hs_kv_compact_workspace_size(nblk: int) -> int:
    """Bytes of workspace hs_kv_compact needs for a cache of nblk pages."""
    n = ctypes.c_uint64(0)
    _check(load().hs_kv_compact_workspace_size(int(nblk), ctypes.byref(n)))
    return int(n.value)


def hs_kv_compact(block_table, refcount, table_out, refcount_out, src, dst, counts, err_flag, workspace, pools=None,
                  k_caches=None, k_scales=None, Di: int = 128, stream=None):
    """Move the pages in use into the lowest ids, in every layer; ``table_out`` and ``refcount_out`` (the inputs
    themselves are allowed) receive the new state, ``src`` / ``dst`` (int32 [nblk]) the moves, ``counts`` (int32 [2])
    {pages in use, moves}. See include/hs.h."""
    (B, pages), nblk = block_table.shape, refcount.numel()
    if table_out.shape != (B, pages) or counts.numel() != 2 or refcount_out.numel() != nblk or src.numel() != nblk or dst.numel() != nblk:
        raise HSError(1, "table_out must have block_table's shape, refcount_out, src and dst one entry per page, counts two")
    L, Li, pp, cp, sp = _layers(pools, k_caches, k_scales)
    _check(load().hs_kv_compact(_pack_compact(B, pages, L, Li, Di, _int(block_table, "block_table"), _int(refcount, "refcount"), nblk,
                                              _int(table_out, "table_out"), _int(refcount_out, "refcount_out"), _int(src, "src"),
                                              _int(dst, "dst"), _int(counts, "counts"), pp, cp, sp,
                                              _tensor(workspace, "workspace", torch.uint8), workspace.numel(),
                                              _int(err_flag, "err_flag")), _stream(stream)))
