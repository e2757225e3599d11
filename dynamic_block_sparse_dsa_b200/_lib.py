"""ctypes binding of libdsa.so (the C ABI in include/dsa.h).

Only argument marshalling lives here: torch tensors are turned into device
pointers and the current CUDA stream handle; every step of the method runs
in the library's CUDA kernels.  There is no CPU fallback: if the library
cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

_lock = threading.Lock()
_lib = None
ADDRESS = {}   # entry point -> its address, once the library is loaded
on_load = []   # called once the library is loaded

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_RANGE, DSA_ERR_WORKSPACE, DSA_ERR_CUDA = range(6)
DEV_ERR_PAGE, DEV_ERR_POS, DEV_ERR_SEL, DEV_ERR_K, DEV_ERR_WAIT, DEV_ERR_VALUE = 1, 2, 4, 8, 16, 32

c_i32 = ctypes.c_int32
c_vp = ctypes.c_void_p


class KvCacheC(ctypes.Structure):
    _fields_ = [("k_pool", c_vp), ("v_pool", c_vp), ("kc_pool", c_vp), ("num_pages", c_i32),
                ("block_size", c_i32), ("num_kv_heads", c_i32), ("head_dim", c_i32), ("idx_dim", c_i32)]


class SeqsC(ctypes.Structure):
    _fields_ = [("block_table", c_vp), ("max_blocks", c_i32), ("seq_lens", c_vp), ("num_seqs", c_i32)]


class QueriesC(ctypes.Structure):
    _fields_ = [("cu_q", c_vp), ("q_pos", c_vp), ("total_q", c_i32)]


class KvCacheFp8C(ctypes.Structure):
    _fields_ = [("k_pool", c_vp), ("v_pool", c_vp), ("kc_pool", c_vp), ("k_scale", c_vp), ("v_scale", c_vp),
                ("num_pages", c_i32), ("block_size", c_i32), ("num_kv_heads", c_i32), ("head_dim", c_i32),
                ("idx_dim", c_i32)]


class RopeC(ctypes.Structure):
    _fields_ = [("inv_freq", c_vp), ("pair_axis", c_vp), ("rotary_dim", c_i32), ("layout", c_i32),
                ("num_axes", c_i32), ("scale", ctypes.c_float)]


class NewTokensC(ctypes.Structure):
    _fields_ = [("cu_new", c_vp), ("total_new", c_i32), ("k", c_vp), ("v", c_vp), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("kc", c_vp), ("pos", c_vp)]


class QueryRowsC(ctypes.Structure):
    _fields_ = [("q", c_vp), ("q_stride", ctypes.c_int64), ("num_heads", c_i32), ("pos", c_vp), ("out", c_vp)]


# The same structs as packed bytes, for the calls that take them as plain
# pointers: packing costs a fifth of filling a ctypes structure.
pack_cache = struct.Struct("@PPPiiiii").pack
pack_cache_fp8 = struct.Struct("@PPPPPiiiii").pack
pack_seqs = struct.Struct("@PiPi").pack
pack_queries = struct.Struct("@PPi").pack
pack_rope = struct.Struct("@PPiiif").pack
pack_new_tokens = struct.Struct("@PiPPqqPP").pack
pack_query_rows = struct.Struct("@PqiPP").pack


# exported symbol -> (argtypes, restype); mirrors include/dsa.h
P = ctypes.POINTER
SIGNATURES = {
    "dsa_kv_append": ([P(KvCacheC), P(SeqsC), c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp], c_i32),
    "dsa_kv_append_rope": ([c_vp] * 8, c_i32),
    "dsa_kv_append_fp8": ([c_vp] * 8, c_i32),
    "dsa_index_score": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp],
                        c_i32),
    "dsa_topk_blocks": ([P(SeqsC), P(QueriesC), c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp], c_i32),
    "dsa_index_score_i64": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_vp, c_i32, c_vp, c_vp, c_vp], c_i32),
    "dsa_index_score_fp8": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp],
                            c_i32),
    "dsa_topk_blocks_i64": ([P(SeqsC), P(QueriesC), c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp], c_i32),
    "dsa_select_blocks_workspace_size": ([c_i32], ctypes.c_size_t),
    "dsa_select_blocks": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_vp, c_i32, c_i32, c_vp, c_i32, c_vp, c_vp,
                           c_vp, ctypes.c_size_t, c_vp, c_vp], c_i32),
    "dsa_select_blocks_append": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp,
                                  c_i32, c_i32, c_vp, c_i32, c_vp, c_vp, c_vp, ctypes.c_size_t, c_vp, c_vp], c_i32),
    "dsa_sparse_attn_decode_workspace_size": ([c_i32, c_i32, c_i32, c_i32], ctypes.c_size_t),
    "dsa_sparse_attn_decode": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_i32, c_vp, c_vp, c_i32,
                                ctypes.c_float, c_vp, c_vp, c_vp, ctypes.c_size_t, c_vp, c_vp], c_i32),
    "dsa_sparse_attn_prefill": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_i32, c_vp, c_vp, c_i32,
                                 ctypes.c_float, c_vp, c_vp, c_vp, c_vp], c_i32),
    "dsa_sparse_attn_decode_noalloc": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_i32, c_vp, c_vp, c_i32,
                                        ctypes.c_float, c_vp, c_vp, c_vp, c_vp], c_i32),
    "dsa_sparse_attn_decode_fp8": ([c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_i32,
                                    ctypes.c_float, c_vp, c_vp, c_vp, ctypes.c_size_t, c_vp, c_vp], c_i32),
    "dsa_sparse_attn_prefill_fp8": ([c_vp, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_i32,
                                     ctypes.c_float, c_vp, c_vp, c_vp, c_vp], c_i32),
    "dsa_decode_fused_workspace_size": ([c_i32, c_i32, c_i32, c_i32], ctypes.c_size_t),
    "dsa_decode_fused": ([P(KvCacheC), P(SeqsC), P(QueriesC), c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_i32,
                          c_i32, c_vp, c_i32, c_vp, c_i32, ctypes.c_float, c_vp, c_vp, c_vp, c_vp, c_vp,
                          ctypes.c_size_t, c_vp, c_vp], c_i32),
    "dsa_stager_create": ([c_i32, c_vp, P(c_vp)], c_i32),
    "dsa_stager_destroy": ([c_vp], c_i32),
    "dsa_stager_begin": ([c_vp, c_i32, c_i32, c_vp, c_vp, c_vp], c_i32),
    "dsa_stager_end": ([c_vp, c_i32, c_i32, c_vp, c_vp, c_vp], c_i32),
    "dsa_stager_wait": ([c_vp, c_i32], c_i32),
    "dsa_stager_join": ([c_vp], c_i32),
    "dsa_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "dsa_version": ([], ctypes.c_int),
}


class DsaError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {msg} (status {status})")
        self.status = status


def lib_path() -> str:
    return _build.LIB


def load():
    """Load libdsa.so (building it first if it is missing or older than its
    sources and nvcc is available).  Raises if the library cannot be loaded."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if _build.is_stale():
            try:
                _build.build()
            except Exception as e:   # no toolchain here: a present library still loads
                if not os.path.exists(_build.LIB):
                    raise RuntimeError(f"libdsa.so is missing and could not be built: {e}") from e
        lib = ctypes.CDLL(_build.LIB)
        for name, (argt, rest) in SIGNATURES.items():
            f = getattr(lib, name)
            f.argtypes = argt
            f.restype = rest
            ADDRESS[name] = ctypes.cast(f, c_vp).value
        _lib = lib
    for f in on_load:
        f()
    return lib


def check(fn: str, status: int) -> None:
    if status != DSA_OK:
        msg = load().dsa_status_string(status).decode()
        raise DsaError(fn, status, msg)
