"""Loads libpa.so and declares the C signatures of include/pa.h (ctypes).

This module only marshals arguments; every step of the compute path runs in
the library's CUDA kernels.  Loading fails loudly when the library is
missing: there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpa.so")

PA_OK, PA_ERR_INVALID, PA_ERR_OOM, PA_ERR_CUDA, PA_ERR_UNSUPPORTED = range(5)
PA_DECODE_NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # include/pa.h
PA_KV_BF16, PA_KV_FP8_E4M3, PA_KV_INT8 = 0, 1, 2


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class DecodeOpts(ctypes.Structure):
    _fields_ = [("partition_tokens", ctypes.c_int32), ("kernel", ctypes.c_int32)]


class RopeDesc(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("max_position", ctypes.c_int32),
                ("num_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
                ("sections_in_turn", ctypes.c_int32), ("adjacent_pairs", ctypes.c_int32)]


class ScoreDesc(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("window", ctypes.c_int32), ("slopes", ctypes.c_void_p)]


class PaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class PaOOM(PaError):
    pass


STATUS_NAMES = {0: "PA_OK", 1: "PA_ERR_INVALID", 2: "PA_ERR_OOM", 3: "PA_ERR_CUDA",
                4: "PA_ERR_UNSUPPORTED"}

_lock = threading.Lock()
_lib = None
_binding = None

P = ctypes.c_void_p
I32 = ctypes.c_int32
I64 = ctypes.c_int64
PI32 = ctypes.POINTER(ctypes.c_int32)
SIZE = ctypes.c_size_t

SIGNATURES = {
    "pa_reshape_and_cache": (I32, [P, P, P, P, CacheDesc, P, I32, P, P, P]),
    "pa_decode_workspace_size": (SIZE, [I32, I32, I32, I32, I32]),
    "pa_decode_workspace_size_ex": (SIZE, [I32, I32, I32, I32, I32, I32]),
    "pa_decode": (I32, [P, P, P, P, CacheDesc, P, I32, P, I32, I32, ctypes.c_float, P, P, P,
                        SIZE, P]),
    "pa_decode_ex": (I32, [P, P, P, P, CacheDesc, P, I32, P, I32, I32, ctypes.c_float, P, P,
                           P, SIZE, ctypes.POINTER(DecodeOpts), P]),
    "pa_decode_noalloc": (I32, [P, P, P, P, CacheDesc, P, I32, P, I32, I32, ctypes.c_float, P,
                                P, P]),
    "pa_decode_noalloc_error": (I32, [P, P]),
    "pa_write_and_decode": (I32, [P, P, P, I32, P, P, P, P, CacheDesc, P, I32, P, I32, I32,
                                  ctypes.c_float, P, P, P, SIZE, P]),
    "pa_copy_blocks": (I32, [P, P, CacheDesc, P, I32, P]),
    "pa_step_prepare": (I32, [P, I32, I32, I32, P, P, I32, I32, P, P]),
    "pa_swap_blocks": (I32, [P, P, I32, P, P, I32, CacheDesc, P, I32, P]),
    "pa_varlen_workspace_size": (ctypes.c_size_t, [I32, I32, I32, I32, I32]),
    "pa_decode_multi_workspace_size": (ctypes.c_size_t, [I32, I32, I32, I32, I32, I32]),
    "pa_decode_shared_prefix_workspace_size": (ctypes.c_size_t, [I32, I32, I32, I32, I32, I32]),
    "pa_decode_shared_prefix": (I32, [P, P, P, P, CacheDesc, P, I32, P, I32, I32, I32,
                                      ctypes.c_float, P, P, P, ctypes.c_size_t, P]),
    "pa_decode_multi": (I32, [P, P, P, P, CacheDesc, P, I32, P, I32, I32, I32, ctypes.c_float,
                              P, P, P, ctypes.c_size_t, P]),
    "pa_varlen_attention": (I32, [P, P, P, P, CacheDesc, P, I32, P, P, I32, I32, I32, ctypes.c_float, P, P,
                                  P, ctypes.c_size_t, P]),
    "pa_varlen_attention_ex": (I32, [P, P, P, P, CacheDesc, P, I32, P, P, I32, I32, I32,
                                     ctypes.c_float, P, P, I32, P, ctypes.c_size_t, P]),
    "pa_rope_and_cache": (I32, [P, P, I64, I32, P, I64, P, I64, P, P, CacheDesc, P, P, P, RopeDesc,
                                I32, P, P, P]),
    "pa_summarize_blocks": (I32, [P, CacheDesc, P, I32, P, P, P]),
    "pa_select_blocks": (I32, [P, P, P, P, CacheDesc, P, I32, P, P, I32, I32, I32, I32, I32, I32,
                               P]),
    "pa_decode_selected": (I32, [P, P, P, P, CacheDesc, P, I32, P, P, P, I32, I32, I32, I32,
                                 ctypes.c_float, P, P, P]),
    "pa_norm_rope_and_cache": (I32, [P, P, I64, I32, P, I64, P, I64, P, P, CacheDesc, P, P, P,
                                     RopeDesc, P, P, ctypes.c_float, I32, P, P, P]),
    "pa_gather_cache": (I32, [P, P, P, P, CacheDesc, P, I32, P, P, P, I32, I32, P, P, P]),
    "pa_scored_workspace_size": (SIZE, [I32, I32, I32, I32]),
    "pa_decode_scored": (I32, [P, P, P, P, CacheDesc, P, I32, P, I32, I32, ctypes.c_float,
                               ScoreDesc, P, P, P, SIZE, P]),
    "pa_varlen_scored": (I32, [P, P, P, P, CacheDesc, P, I32, P, P, I32, I32, I32, ctypes.c_float,
                               ScoreDesc, P, P, P, P, SIZE, P]),
    "pa_slot_mapping": (I32, [PI32, I32, I32, I32, PI32, PI32, I32, PI32]),
    "pa_pool_create": (P, [I32]),
    "pa_pool_create_ordered": (P, [I32, PI32]),
    "pa_pool_destroy": (None, [P]),
    "pa_pool_num_blocks": (I32, [P]),
    "pa_pool_num_free": (I32, [P]),
    "pa_pool_refcount": (I32, [P, I32]),
    "pa_pool_free_order": (I32, [P, PI32, I32]),
    "pa_pool_alloc": (I32, [P, I32, PI32]),
    "pa_pool_incref": (I32, [P, PI32, I32]),
    "pa_pool_free": (I32, [P, PI32, I32]),
    "pa_pool_cow": (I32, [P, I32, PI32]),
    "pa_pool_enable_prefix_cache": (I32, [P, I32]),
    "pa_pool_alloc_prefix": (I32, [P, PI32, I32, PI32, PI32]),
    "pa_pool_register_block": (I32, [P, I32, I32, PI32]),
    "pa_pool_num_cached": (I32, [P]),
    "pa_status_string": (ctypes.c_char_p, [I32]),
    "pa_last_error": (ctypes.c_char_p, []),
    "pa_version": (ctypes.c_char_p, []),
}


def lib():
    """The loaded library (built on first use if the CUDA toolkit is here)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                from . import build as _build
                _build.build_library()
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libpa.so not found at {LIB_PATH}; run build()")
            handle = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(handle, name)
                fn.restype = res
                fn.argtypes = args
            _lib = handle
    return _lib


def binding():
    """The compiled binding of the block-sparse and scored steps' calls (_binding.so)."""
    global _binding
    if _binding is not None:
        return _binding
    lib()
    with _lock:
        if _binding is None:
            from . import build as _build
            if not _build.binding_fits():  # another torch's or Python's layouts must not be loaded
                # (libpa.so stays: the binding has to meet the one loaded above)
                _build.build_binding()
            import torch  # noqa: F401  (its libraries are what the binding links against)

            _binding = importlib.import_module("._binding", __package__)
    return _binding


def check(status: int) -> None:
    if status != PA_OK:
        msg = lib().pa_last_error().decode()
        if status == PA_ERR_OOM:
            raise PaOOM(status, msg)
        raise PaError(status, msg)
