"""ctypes view of ``libfa_gb300.so`` (the C ABI of include/fa_gb300.h).

Argument marshalling only. The library is built in-tree by
``attention_fa2_attn_gb300.build``. If it is missing, loading fails loudly:
there is no fallback implementation.
"""

from __future__ import annotations

import ctypes
import importlib.util
import os
import re
import warnings

from . import build as _build

_HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "fa_gb300.h")

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_CUDA = 3
FA_ERR_TIMEOUT = 4
FA_ERR_BOUNDS = 5

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_ULL = ctypes.c_ulonglong
_D = ctypes.c_double

FA_DTYPE_BF16 = 0
FA_DTYPE_F32 = 1
FA_PLAN_MAX_T = 8388480
FA_TREE_MASK_MAX_T = 8192
FA_TREE_MASK_MAX_B = 65535
FA_PAGES_MAX = 4194304
FA_FORK_MAX = 65536
FA_PREFIX_MAX_GROUPS = 4096
FA_ROPE_MAX_AXES = 8
FA_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

# name -> (restype, argtypes); mirrors include/fa_gb300.h
SIGNATURES = {
    "fa_version": (_I, []),
    "fa_status_string": (ctypes.c_char_p, [_I]),
    "fa_last_cuda_error_string": (ctypes.c_char_p, []),
    "fa_fwd": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_fwd_f32": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_bwd": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P]),
    "fa_bwd_workspace_bytes": (_SZ, [_I, _I, _I]),
    "fa_fwd_kv_outer": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P]),
    "fa_fwd_kv_outer_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "fa_num_splits_heuristic": (_I, [_I, _I, _I, _I]),
    "fa_num_splits_prefill": (_I, [_I, _I, _I, _I, _I, _I]),
    "fa_decode_num_splits": (_I, [_I, _I, _I, _I, _I, _I, _I]),
    "fa_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "fa_decode_splitkv": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P]),
    "fa_decode_splitkv_static": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P]),
    "fa_lse_merge": (_I, [_P, _P, _P, _P, _I, _I, _I, _P]),
    "fa_decode_paged": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ, _P],
    ),
    "fa_paged_plan": (_I, [_P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "fa_tree_mask": (_I, [_P, _P, _P, _P, _P, _I, _I, _P]),
    "fa_rope_inv_freq": (_I, [_P, ctypes.POINTER(_F), _I, _D, _I, _D, _D, _D, _D]),
    "fa_rope": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_rope_bwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_rope_append_paged": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P],
    ),
    "fa_rope_axes": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_rope_axes_bwd": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P]),
    "fa_rope_axes_append_paged": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P],
    ),
    "fa_pages_fork": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "fa_pages_copy": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P]),
    "fa_pages_free": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "fa_pages_compact": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "fa_tree_decode_paged": (
        _I,
        [_P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _SZ, _P],
    ),
    "fa_tree_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "fa_prefix_decode_paged": (
        _I,
        [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _I, _P, _SZ, _P],
    ),
    "fa_prefix_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "fa_get_last_device_error": (_I, [_P, ctypes.POINTER(_I)]),
    "fa_set_wait_timeout_ns": (None, [_ULL]),
    "fa_get_wait_timeouts": (None, [ctypes.POINTER(_ULL), ctypes.POINTER(_ULL)]),
    "fa_selftest_wait_timeout": (_I, [_ULL, _P]),
}

_lib = None


def header_symbols() -> list[str]:
    """Names of every function the public header declares."""
    text = open(_HEADER).read()
    return sorted(set(re.findall(r"^FA_API\s+[\w\s\*]*?\b(fa_\w+)\s*\(", text, flags=re.M)))


def lib(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load (building first if needed) the CUDA library and bind its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB_PATH
    if build_if_missing and _build.needs_build():
        _build.build()
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is missing; build it with attention_fa2_attn_gb300.build.build()")
    l = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        f = getattr(l, name)
        f.restype = res
        f.argtypes = args
    _lib = l
    return l


_fast_calls = None


class _NoFastCalls:
    """In the place of an extension module that is not there: every call is left to the checks in Python."""

    def __getattr__(self, name):
        return lambda *args: None


def fast():
    """The extension module ``_fast`` (the step calls from Python objects to the library),
    loaded after the library it is linked to."""
    global _fast_calls
    if _fast_calls is None:
        lib()
        try:
            spec = importlib.util.spec_from_file_location("_fast", _build.fast_path())
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
        except (ImportError, OSError) as e:
            warnings.warn(f"no extension module, step calls cost about 15 us more on the host: {e}", RuntimeWarning,
                          stacklevel=3)
            module = _NoFastCalls()
        _fast_calls = module
    return _fast_calls


class FAError(RuntimeError):
    def __init__(self, status: int, where: str):
        l = lib()
        msg = l.fa_status_string(status).decode()
        if status == FA_ERR_CUDA:
            msg += ": " + l.fa_last_cuda_error_string().decode()
        super().__init__(f"{where}: {msg}")
        self.status = status


def check(status: int, where: str) -> None:
    if status != FA_OK:
        raise FAError(status, where)
