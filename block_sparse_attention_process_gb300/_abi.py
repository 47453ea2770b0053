"""ctypes mirror of include/bsa.h and the loader of libbsa.so.

Argument marshalling only: every step of the attention path runs in the
CUDA library.  If the library is missing this module raises; there is no
fallback of any kind.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
# BSA_LIBRARY_VARIANT=debug loads the range-checked build (see build.py)
LIB_PATH = os.path.join(HERE, "_lib", "libbsa_debug.so" if os.environ.get("BSA_LIBRARY_VARIANT") == "debug"
                        else "libbsa.so")

# status codes
OK, INVALID_ARG, UNSUPPORTED, CUDA, OOM, TIMEOUT, DEVICE = range(7)
# mask kinds
MASK_DENSE, MASK_CAUSAL, MASK_LOCAL, MASK_CHUNKED_CAUSAL, MASK_FULL = range(5)
ORIENT_FWD, ORIENT_DKV = 0, 1


class MaskSpec(C.Structure):
    _fields_ = [("kind", C.c_int32), ("mask_heads", C.c_int32), ("q_len", C.c_int64), ("kv_len", C.c_int64),
                ("local_left", C.c_int64), ("local_right", C.c_int64), ("chunk", C.c_int64),
                ("dense", C.c_void_p)]


class MaskOpts(C.Structure):
    _fields_ = [("block_q", C.c_int32), ("block_kv", C.c_int32), ("shrink", C.c_int32),
                ("orientation", C.c_int32)]


class MaskInfoDesc(C.Structure):
    _fields_ = [("block_mask", C.c_void_p), ("data_next", C.c_void_p), ("data_next_bytes", C.c_int32),
                ("mask_next", C.c_void_p), ("mask_next_bytes", C.c_int32),
                ("partial_mask_blocks", C.c_void_p), ("q_sequence", C.c_void_p),
                ("heads", C.c_int32), ("rows", C.c_int32), ("width", C.c_int32), ("cols", C.c_int32),
                ("num_partial", C.c_int64), ("n_empty", C.c_int64), ("n_partial", C.c_int64),
                ("n_full", C.c_int64), ("kind", C.c_int32), ("orientation", C.c_int32),
                ("shrink", C.c_int32), ("q_len", C.c_int64), ("kv_len", C.c_int64),
                ("row_len", C.c_void_p), ("row_order", C.c_void_p)]


class FwdArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("o", C.c_void_p),
                ("lse", C.c_void_p), ("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32),
                ("D", C.c_int32), ("S_q", C.c_int64), ("S_kv", C.c_int64), ("softmax_scale", C.c_float),
                ("logits_soft_cap", C.c_float), ("sinks", C.c_void_p), ("num_sinks", C.c_int32),
                ("sinks_per_kv_head", C.c_int32)]


class FwdPartialArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("o_acc", C.c_void_p),
                ("m", C.c_void_p), ("l", C.c_void_p), ("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32),
                ("D", C.c_int32), ("S_q", C.c_int64), ("S_kv_shard", C.c_int64), ("kv_offset", C.c_int64),
                ("softmax_scale", C.c_float), ("logits_soft_cap", C.c_float)]


class MergeArgs(C.Structure):
    _fields_ = [("n_shards", C.c_int32), ("o_acc", C.c_void_p), ("m", C.c_void_p), ("l", C.c_void_p),
                ("o", C.c_void_p), ("lse", C.c_void_p), ("rows", C.c_int64), ("D", C.c_int32)]


class BwdArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("v", C.c_void_p), ("o", C.c_void_p),
                ("lse", C.c_void_p), ("do_", C.c_void_p), ("dq", C.c_void_p), ("dk", C.c_void_p),
                ("dv", C.c_void_p), ("dsum", C.c_void_p), ("B", C.c_int32), ("Hq", C.c_int32),
                ("Hkv", C.c_int32), ("D", C.c_int32), ("S_q", C.c_int64), ("S_kv", C.c_int64),
                ("softmax_scale", C.c_float), ("grad_fp32", C.c_int32), ("logits_soft_cap", C.c_float),
                ("sinks", C.c_void_p), ("dsinks", C.c_void_p), ("num_sinks", C.c_int32),
                ("sinks_per_kv_head", C.c_int32)]


class KeyWeightsArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("k", C.c_void_p), ("lse", C.c_void_p), ("q_lens", C.c_void_p),
                ("weights", C.c_void_p), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t),
                ("B", C.c_int32), ("Hq", C.c_int32), ("Hkv", C.c_int32), ("D", C.c_int32), ("S_q", C.c_int64),
                ("S_kv", C.c_int64), ("softmax_scale", C.c_float), ("logits_soft_cap", C.c_float)]


class Kv4Cache(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("k_scales", C.c_void_p), ("v_codes", C.c_void_p),
                ("v_scales", C.c_void_p), ("weights", C.c_void_p), ("positions", C.c_void_p), ("B", C.c_int32),
                ("Hkv", C.c_int32), ("D", C.c_int32), ("capacity", C.c_int64)]


class Kv4AppendArgs(C.Structure):
    _fields_ = [("cache", Kv4Cache), ("k", C.c_void_p), ("v", C.c_void_p), ("k_stride", C.c_int64 * 3),
                ("v_stride", C.c_int64 * 3), ("T", C.c_int64), ("start", C.c_void_p), ("n_new", C.c_void_p),
                ("first_position", C.c_void_p), ("weights0", C.c_void_p), ("k_values", C.c_void_p),
                ("v_values", C.c_void_p)]


class Kv4FwdArgs(C.Structure):
    _fields_ = [("cache", Kv4Cache), ("q", C.c_void_p), ("o", C.c_void_p), ("lse", C.c_void_p),
                ("q_stride", C.c_int64 * 3), ("o_stride", C.c_int64 * 3), ("Hq", C.c_int32), ("T", C.c_int64),
                ("lens", C.c_void_p), ("q_lens", C.c_void_p), ("softmax_scale", C.c_float),
                ("logits_soft_cap", C.c_float), ("sinks", C.c_void_p), ("num_sinks", C.c_int32),
                ("sinks_per_kv_head", C.c_int32), ("accumulate", C.c_int32), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t)]


class Kv4EvictArgs(C.Structure):
    _fields_ = [("cache", Kv4Cache), ("out", Kv4Cache), ("lens", C.c_void_p), ("seen", C.c_void_p),
                ("keep", C.c_int64), ("recent", C.c_int64), ("new_lens", C.c_void_p), ("index", C.c_void_p),
                ("k_values", C.c_void_p), ("v_values", C.c_void_p), ("workspace", C.c_void_p),
                ("workspace_bytes", C.c_size_t)]


class PagedCache(C.Structure):
    _fields_ = [("k", C.c_void_p), ("v", C.c_void_p), ("k_stride", C.c_int64 * 3), ("v_stride", C.c_int64 * 3),
                ("bounds", C.c_void_p), ("pages", C.c_int64), ("Hkv", C.c_int32), ("D", C.c_int32), ("page", C.c_int32)]


class PagedResizeArgs(C.Structure):
    _fields_ = [("table", C.c_void_p), ("free_pages", C.c_void_p), ("used", C.c_void_p), ("lens", C.c_void_p),
                ("new_lens", C.c_void_p), ("lens_out", C.c_void_p), ("used_out", C.c_void_p), ("slots", C.c_void_p),
                ("B", C.c_int32), ("M", C.c_int64), ("T", C.c_int64), ("pages", C.c_int64), ("page", C.c_int32)]


class PagedAppendArgs(C.Structure):
    _fields_ = [("cache", PagedCache), ("k", C.c_void_p), ("v", C.c_void_p), ("src_k_stride", C.c_int64 * 3),
                ("src_v_stride", C.c_int64 * 3), ("slots", C.c_void_p), ("B", C.c_int32), ("T", C.c_int64)]


class PagedSelectArgs(C.Structure):
    _fields_ = [("cache", PagedCache), ("q", C.c_void_p), ("q_stride", C.c_int64 * 3), ("table", C.c_void_p),
                ("lens", C.c_void_p), ("q_lens", C.c_void_p), ("index", C.c_void_p), ("B", C.c_int32), ("Hq", C.c_int32),
                ("M", C.c_int64), ("T", C.c_int64), ("keep", C.c_int64), ("first", C.c_int64), ("recent", C.c_int64)]


class PagedFwdArgs(C.Structure):
    _fields_ = [("cache", PagedCache), ("q", C.c_void_p), ("o", C.c_void_p), ("lse", C.c_void_p),
                ("q_stride", C.c_int64 * 3), ("o_stride", C.c_int64 * 3), ("table", C.c_void_p), ("lens", C.c_void_p),
                ("q_lens", C.c_void_p), ("select", C.c_void_p), ("B", C.c_int32), ("Hq", C.c_int32), ("M", C.c_int64),
                ("T", C.c_int64), ("keep", C.c_int64), ("kind", C.c_int32), ("local_left", C.c_int64), ("chunk", C.c_int64),
                ("softmax_scale", C.c_float), ("logits_soft_cap", C.c_float), ("sinks", C.c_void_p), ("num_sinks", C.c_int32),
                ("sinks_per_kv_head", C.c_int32), ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t)]


# The kv4 and paged calls are made once a token, so their arguments are packed with
# struct (a third of the time a ctypes.Structure of as many fields takes): the
# cache, which every call begins with, and what follows it.
KV4_CACHE = struct.Struct("@6P3iq")
KV4_APPEND_REST = struct.Struct("@2P6qq6P")
KV4_FWD_REST = struct.Struct("@3P6qiqPPffPiiiPN")
KV4_EVICT_REST = struct.Struct("@2P2q5PN")
for _s, _rest in ((Kv4AppendArgs, KV4_APPEND_REST), (Kv4FwdArgs, KV4_FWD_REST)):
    assert KV4_CACHE.size + _rest.size == C.sizeof(_s)
PAGED_CACHE = struct.Struct("@2P6qPq3i0q")
PAGED_RESIZE = struct.Struct("@8Pi3qi0q")
PAGED_APPEND_REST = struct.Struct("@2P6qPiq")
PAGED_SELECT_REST = struct.Struct("@P3q4P2i5q")
PAGED_FWD_REST = struct.Struct("@3P6q4P2i3qi2q2fP2iPN")
assert PAGED_RESIZE.size == C.sizeof(PagedResizeArgs)
for _s, _rest in ((PagedAppendArgs, PAGED_APPEND_REST), (PagedSelectArgs, PAGED_SELECT_REST), (PagedFwdArgs, PAGED_FWD_REST)):
    assert PAGED_CACHE.size + _rest.size == C.sizeof(_s)
assert 2 * KV4_CACHE.size + KV4_EVICT_REST.size == C.sizeof(Kv4EvictArgs)


# name -> (restype, argtypes); every symbol include/bsa.h declares
SIGNATURES = {
    "bsa_mask_compile": (C.c_int, [C.POINTER(MaskSpec), C.POINTER(MaskOpts), C.c_void_p, C.POINTER(C.c_void_p)]),
    "bsa_mask_info_view": (C.c_int, [C.c_void_p, C.POINTER(MaskInfoDesc)]),
    "bsa_mask_info_destroy": (C.c_int, [C.c_void_p]),
    "bsa_fwd": (C.c_int, [C.POINTER(FwdArgs), C.c_void_p, C.c_void_p]),
    "bsa_fwd_partial": (C.c_int, [C.POINTER(FwdPartialArgs), C.c_void_p, C.c_void_p]),
    "bsa_fwd_merge": (C.c_int, [C.POINTER(MergeArgs), C.c_void_p]),
    "bsa_bwd": (C.c_int, [C.POINTER(BwdArgs), C.c_void_p, C.c_void_p, C.c_void_p]),
    "bsa_bwd_rowsum": (C.c_int, [C.POINTER(BwdArgs), C.c_void_p]),
    "bsa_bwd_noalloc": (C.c_int, [C.POINTER(BwdArgs), C.c_void_p, C.c_void_p, C.c_void_p]),
    "bsa_bwd_dkv": (C.c_int, [C.POINTER(BwdArgs), C.c_void_p, C.c_void_p]),
    "bsa_bwd_dq": (C.c_int, [C.POINTER(BwdArgs), C.c_void_p, C.c_void_p]),
    "bsa_key_weights": (C.c_int, [C.POINTER(KeyWeightsArgs), C.c_void_p, C.c_void_p]),
    "bsa_key_weights_workspace": (C.c_int, [C.POINTER(KeyWeightsArgs), C.c_void_p, C.POINTER(C.c_size_t)]),
    "bsa_kv4_append": (C.c_int, [C.c_void_p, C.c_void_p]),
    "bsa_kv4_fwd": (C.c_int, [C.c_void_p, C.c_void_p]),
    "bsa_kv4_fwd_workspace": (C.c_int, [C.c_void_p, C.POINTER(C.c_size_t)]),
    "bsa_kv4_evict": (C.c_int, [C.c_void_p, C.c_void_p]),
    "bsa_kv4_evict_workspace": (C.c_int, [C.c_void_p, C.POINTER(C.c_size_t)]),
    "bsa_paged_resize": (C.c_int, [C.c_void_p, C.c_void_p]),
    "bsa_paged_append": (C.c_int, [C.c_void_p, C.c_void_p]),
    "bsa_paged_select": (C.c_int, [C.c_void_p, C.c_void_p]),
    "bsa_paged_fwd": (C.c_int, [C.c_void_p, C.c_void_p]),
    "bsa_paged_fwd_workspace": (C.c_int, [C.c_void_p, C.POINTER(C.c_size_t)]),
    "bsa_get_device_error": (C.c_int, [C.c_void_p, C.POINTER(C.c_uint32)]),
    "bsa_set_wait_limit_ns": (C.c_int, [C.c_uint64]),
    "bsa_debug_wait_timeout": (C.c_int, [C.c_void_p]),
    "bsa_debug_selfcheck": (C.c_int, [C.c_void_p]),
    "bsa_debug_tile_schedule": (C.c_int, [C.POINTER(C.c_int32), C.POINTER(C.c_int32), C.c_int32, C.c_int32,
                                          C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32,
                                          C.POINTER(C.c_int32), C.c_int32, C.POINTER(C.c_int32)]),
    "bsa_status_string": (C.c_char_p, [C.c_int]),
    "bsa_last_error": (C.c_char_p, []),
    "bsa_version": (C.c_char_p, []),
}

_lib = None


def lib() -> C.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libbsa.so is not built ({LIB_PATH}); run __graft_entry__.build() "
                               "or python -m block_sparse_attention_process_gb300.build")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


class BsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        L = lib()
        msg = L.bsa_last_error().decode(errors="replace")
        super().__init__(f"{where}: {L.bsa_status_string(status).decode()} ({status}): {msg}")
        self.status = status


def check(status: int, where: str) -> None:
    if status != OK:
        raise BsaError(status, where)
