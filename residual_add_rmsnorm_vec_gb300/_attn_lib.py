"""ctypes binding of the C ABI in include/rmsnorm_attn.h (argument marshalling
only).  The library is built next to the row norm's; a missing one raises."""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

from . import _lib
from .build import ATTN_PATH, FAST_PATH

RMSATTN_NORM = 0x1000
RMSATTN_INTERLEAVED = 0x2000
RMSATTN_POS_I64 = 0x4000
RMSATTN_OUT_FP8 = 0x8000
RMSATTN_ZERO_OUT, RMSATTN_ZERO_RESIDUAL, RMSATTN_ZERO_SCALE = 0x10000, 0x20000, 0x40000
RMSATTN_BLOCK = 16
RMSATTN_MAX_QUERIES = 32
RMSATTN_BAD_PAGE = 4  # bits of the status word
RMSATTN_WAIT_RAN_OUT = 1

EXPORTED_ATTN = ("rmsattn_qk_rope_fwd", "rmsattn_kv_append", "rmsattn_kv_attention",
                 "rmsattn_kv_attention_workspace", "rmsattn_read_status", "rmsattn_kv_prefix_attention",
                 "rmsattn_kv_prefix_attention_workspace", "rmsattn_pages_step", "rmsattn_pages_workspace",
                 "rmsattn_block_norms", "rmsattn_set_wait_limit")


class RmsattnCache(ctypes.Structure):
    """Mirror of ``rmsattn_cache``."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
                + [(n, ctypes.c_int64) for n in ("n_pages", "page_stride", "scale_stride")]
                + [(n, ctypes.c_int32) for n in ("n_kv_heads", "page_size", "head_dim", "reserved")])


_lock = threading.Lock()
_loaded = None


def attn_library_path() -> str:
    return ATTN_PATH


def load_attn() -> ctypes.CDLL:
    """Load the compiled library (raises if it has not been built)."""
    global _loaded
    if _loaded is not None:
        return _loaded
    with _lock:
        if _loaded is None:
            if not os.path.exists(ATTN_PATH):
                raise RuntimeError(f"the CUDA library {ATTN_PATH} is not built; run "
                                   "residual_add_rmsnorm_vec_gb300.build.build() first")
            # global: the marshalling module below binds to these symbols
            lib = ctypes.CDLL(ATTN_PATH, mode=ctypes.RTLD_GLOBAL)
            vp, i64, u32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_float
            cache = ctypes.POINTER(RmsattnCache)
            lib.rmsattn_qk_rope_fwd.restype = ctypes.c_int
            lib.rmsattn_qk_rope_fwd.argtypes = [vp] * 7 + [i64, vp, vp] + [i64] * 10 + [f32, f32, u32,
                                                                                       vp]
            lib.rmsattn_kv_append.restype = ctypes.c_int
            lib.rmsattn_kv_append.argtypes = [cache, vp, vp, i64, i64, vp, i64, i64, vp, vp, i64, i64,
                                              u32, vp]
            lib.rmsattn_kv_attention.restype = ctypes.c_int
            lib.rmsattn_kv_attention.argtypes = [vp, cache, vp, i64, i64, vp, vp, i64, i64, i64, i64,
                                                 i64, f32, i64, i64, vp, i64, u32, vp]
            lib.rmsattn_kv_attention_workspace.restype = i64
            lib.rmsattn_kv_attention_workspace.argtypes = [i64] * 8
            lib.rmsattn_kv_prefix_attention.restype = ctypes.c_int
            lib.rmsattn_kv_prefix_attention.argtypes = [vp, cache, vp, i64, i64, vp, vp, vp, i64, vp, i64, i64,
                                                        i64, i64, i64, f32, vp, i64, u32, vp]
            lib.rmsattn_kv_prefix_attention_workspace.restype = i64
            lib.rmsattn_kv_prefix_attention_workspace.argtypes = [i64] * 7
            lib.rmsattn_pages_step.restype = ctypes.c_int
            lib.rmsattn_pages_step.argtypes = [vp, i64, vp, vp, i64, i64, vp, vp, vp, i64, i64, i64,
                                               vp, vp, vp, vp, vp, vp, vp, vp, i64, u32, vp]
            lib.rmsattn_pages_workspace.restype = i64
            lib.rmsattn_pages_workspace.argtypes = [i64]
            lib.rmsattn_block_norms.restype = ctypes.c_int
            lib.rmsattn_block_norms.argtypes = [vp, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, i64, i64,
                                                f32, f32, f32, u32, vp]
            lib.rmsattn_set_wait_limit.restype = ctypes.c_int
            lib.rmsattn_set_wait_limit.argtypes = [i64]
            lib.rmsattn_read_status.restype = ctypes.c_int
            lib.rmsattn_read_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), ctypes.c_int]
            _loaded = lib
    return _loaded


_fast = None


def load_fast():
    """The native marshalling module (raises if it has not been built)."""
    global _fast
    if _fast is None:
        load_attn()
        if not os.path.exists(FAST_PATH):
            raise RuntimeError(f"the extension module {FAST_PATH} is not built; run "
                               "residual_add_rmsnorm_vec_gb300.build.build() first")
        import torch  # noqa: F401  (its libraries hold the module's other symbols)

        loader = importlib.machinery.ExtensionFileLoader("rmsattn_fast", FAST_PATH)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("rmsattn_fast", loader))
        loader.exec_module(mod)
        _fast = mod
    return _fast


def rmsattn_read_status(clear: bool = False) -> int:
    """Status word of the attention-path kernels on the current device (0, or the
    bits ``RMSATTN_BAD_PAGE`` and ``RMSATTN_WAIT_RAN_OUT``)."""
    v = ctypes.c_uint32(0)
    st = load_attn().rmsattn_read_status(ctypes.byref(v), int(bool(clear)))
    if st != _lib.RMSN_OK:
        raise _lib.RmsnError(st, "rmsattn_read_status")
    return int(v.value)


def rmsattn_set_wait_limit(cycles: int) -> int:
    """Testing hook: the bound of the waits inside ``kv_cache_prefix_attention``'s
    kernel on the current device (0 = the default; negative = give up once
    a barrier has been tried)."""
    return int(load_attn().rmsattn_set_wait_limit(int(cycles)))
