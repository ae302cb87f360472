"""ctypes loader for librmsnorm_gb300.so (the C ABI of include/rmsnorm.h).

Loading needs no GPU (the CUDA runtime is linked statically and only reaches
the driver on the first CUDA call), so symbol checks run anywhere.  If the
library has not been built, every entry point raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

from .build import LIB_PATH, binding_path

# Names exported by the library, in header order.
EXPORTS = (
    "rmsnorm_fwd",
    "rmsnorm_vjp",
    "rmsnorm_fused_vjp",
    "rmsnorm_fwd_ex",
    "rmsnorm_vjp_ex",
    "rmsnorm_block_fwd",
    "rmsnorm_block_vjp",
    "rmsnorm_block_vjp_ws",
    "rmsnorm_block_vjp_workspace_size",
    "rmsnorm_fwd_q8",
    "rmsnorm_gated_silu",
    "rmsnorm_rope_kv_append",
    "rmsnorm_rope",
    "rmsnorm_rope_axes",
    "rmsnorm_rope_kv_append_ex",
    "rmsnorm_kv_append",
    "rmsnorm_kv_read",
    "rmsnorm_rope_frequencies",
    "rmsnorm_kv_release",
    "rmsnorm_kv_plan",
    "rmsnorm_vjp_workspace_size",
    "rmsnorm_vjp_ws",
    "rmsnorm_vjp_noalloc",
    "rmsnorm_status_string",
    "rmsnorm_last_cuda_error",
    "rmsnorm_device_status",
    "rmsnorm_debug_inject",
    "rmsnorm_debug_fail_allocs",
    "rmsnorm_debug_claim_counters",
    "rmsnorm_describe_dispatch",
)

STATUS = {
    0: "RMSNORM_OK",
    1: "RMSNORM_ERR_INVALID_ARG",
    2: "RMSNORM_ERR_UNSUPPORTED",
    3: "RMSNORM_ERR_CUDA",
    4: "RMSNORM_ERR_NO_MEMORY",
    5: "RMSNORM_ERR_TIMEOUT",
}
DEVSTATUS_WAIT_TIMEOUT = 1
DEVSTATUS_BAD_INDEX = 2
ROPE_SCALING = {None: 0, "linear": 1, "ntk": 2, "yarn": 3, "llama3": 4}
ROPE_MAX_AXES = 4
MAX_D = 1 << 24
VJP_NOALLOC_MAX_BYTES = 16 << 20

_vp = ctypes.c_void_p
_f = ctypes.c_float
_d = ctypes.c_double
_i64 = ctypes.c_int64
_i = ctypes.c_int

_lock = threading.Lock()
_lib = None


class RmsnormError(RuntimeError):
    """A non-zero status returned by the C library."""

    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        name = STATUS.get(status, "status %d" % status)
        msg = "%s failed: %s" % (fn, name)
        if detail:
            msg += " (" + detail + ")"
        super().__init__(msg)


def _bind(lib: ctypes.CDLL) -> ctypes.CDLL:
    lib.rmsnorm_fwd.argtypes = [_vp, _vp, _vp, _f, _f, _vp, _vp, _i64, _i64, _i, _vp]
    lib.rmsnorm_fwd.restype = _i
    lib.rmsnorm_vjp.argtypes = [_vp, _vp, _vp, _f, _f, _vp, _vp, _i64, _i64, _i, _vp]
    lib.rmsnorm_vjp.restype = _i
    lib.rmsnorm_fused_vjp.argtypes = [_vp, _vp, _vp, _vp, _f, _f, _vp, _vp, _i64, _i64, _i, _vp]
    lib.rmsnorm_fused_vjp.restype = _i
    lib.rmsnorm_fwd_ex.argtypes = [_vp, _i64, _vp, _i64, _vp, _f, _f, _vp, _i64, _vp, _i64, _vp,
                                   _i64, _i64, _i, _vp]
    lib.rmsnorm_fwd_ex.restype = _i
    lib.rmsnorm_vjp_ex.argtypes = [_vp, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _f, _f, _vp, _i64,
                                   _vp, _i64, _i64, _i, _vp]
    lib.rmsnorm_vjp_ex.restype = _i
    lib.rmsnorm_block_fwd.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _f, _f, _f,
                                      _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i, _vp]
    lib.rmsnorm_block_fwd.restype = _i
    lib.rmsnorm_block_vjp.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _f, _vp, _i64,
                                      _vp, _i64, _vp, _f, _f, _vp, _i64, _vp, _i64, _vp, _vp, _vp,
                                      _i64, _i64, _i, _vp]
    lib.rmsnorm_block_vjp.restype = _i
    lib.rmsnorm_block_vjp_ws.argtypes = lib.rmsnorm_block_vjp.argtypes[:-1] + [_vp, ctypes.c_size_t, _vp]
    lib.rmsnorm_block_vjp_ws.restype = _i
    lib.rmsnorm_block_vjp_workspace_size.argtypes = [_i64, _i64, _i]
    lib.rmsnorm_block_vjp_workspace_size.restype = ctypes.c_size_t
    lib.rmsnorm_gated_silu.argtypes = [_vp, _vp, _i64, _i64, _i, _vp]
    lib.rmsnorm_gated_silu.restype = _i
    lib.rmsnorm_rope_kv_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _f,
                                           _i, _i64, _i64, _i64, _i64, _i64, _i, _vp]
    lib.rmsnorm_rope_kv_append.restype = _i
    lib.rmsnorm_rope.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _i, _i, _i64,
                                 _i64, _i64, _i64, _i64, _i64, _i, _vp]
    lib.rmsnorm_rope.restype = _i
    lib.rmsnorm_rope_kv_append_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _vp, _vp, _vp, _vp, _f, _i, _i64, _i64, _i64, _i64,
                                              _i64, _i64, _i, _vp]
    lib.rmsnorm_rope_kv_append_ex.restype = _i
    lib.rmsnorm_rope_axes.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _f, _i,
                                      _i, _i64, _i64, _i64, _i64, _i64, _i64, _i, _vp]
    lib.rmsnorm_rope_axes.restype = _i
    lib.rmsnorm_kv_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _vp, _vp, _f, _i, _i64, _i64, _i64, _i64,
                                      _i64, _i64, _i, _i, _vp]
    lib.rmsnorm_kv_append.restype = _i
    lib.rmsnorm_kv_read.argtypes = [_vp] * 13 + [_i64, _i64, _i64, _i64, _i, _i, _vp]
    lib.rmsnorm_kv_read.restype = _i
    lib.rmsnorm_fwd_q8.argtypes = [_vp, _i64, _vp, _i64, _vp, _f, _f, _vp, _i64, _vp, _i64, _vp, _i64, _i64,
                                   _i64, _i, _vp]
    lib.rmsnorm_fwd_q8.restype = _i
    lib.rmsnorm_rope_frequencies.argtypes = [_i, _i64, _d, _d, _d, _d, _d, _vp,
                                             ctypes.POINTER(ctypes.c_float)]
    lib.rmsnorm_rope_frequencies.restype = _i
    lib.rmsnorm_kv_release.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i64,
                                       _vp]
    lib.rmsnorm_kv_release.restype = _i
    lib.rmsnorm_kv_plan.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _i64, _i64, _vp]
    lib.rmsnorm_kv_plan.restype = _i
    lib.rmsnorm_vjp_workspace_size.argtypes = [_i64, _i64, _i]
    lib.rmsnorm_vjp_workspace_size.restype = ctypes.c_size_t
    lib.rmsnorm_vjp_ws.argtypes = [_vp, _vp, _vp, _f, _f, _vp, _vp, _i64, _i64, _i, _vp,
                                   ctypes.c_size_t, _vp]
    lib.rmsnorm_vjp_ws.restype = _i
    lib.rmsnorm_vjp_noalloc.argtypes = [_vp, _vp, _vp, _f, _f, _vp, _vp, _i64, _i64, _i, _vp]
    lib.rmsnorm_vjp_noalloc.restype = _i
    lib.rmsnorm_status_string.argtypes = [_i]
    lib.rmsnorm_status_string.restype = ctypes.c_char_p
    lib.rmsnorm_last_cuda_error.argtypes = []
    lib.rmsnorm_last_cuda_error.restype = _i
    lib.rmsnorm_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), _i]
    lib.rmsnorm_device_status.restype = _i
    lib.rmsnorm_debug_inject.argtypes = [_i64, _i64]
    lib.rmsnorm_debug_inject.restype = _i
    lib.rmsnorm_debug_fail_allocs.argtypes = [_i]
    lib.rmsnorm_debug_fail_allocs.restype = _i
    lib.rmsnorm_debug_claim_counters.argtypes = [_i]
    lib.rmsnorm_debug_claim_counters.restype = _i
    lib.rmsnorm_describe_dispatch.argtypes = [_i, _i64, _i64, _i, _i, _i]
    lib.rmsnorm_describe_dispatch.restype = ctypes.c_char_p
    return lib


def lib() -> ctypes.CDLL:
    """The loaded C library.  Raises if it was never built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        "%s is missing: build it with `python -m rmsnorm_fwd_bwd_add_gb300.build` "
                        "(nvcc, sm_103a); there is no CPU fallback" % LIB_PATH)
                _lib = _bind(ctypes.CDLL(LIB_PATH))
    return _lib


_BOUND = ("rmsnorm_block_fwd", "rmsnorm_block_vjp_ws", "rmsnorm_block_vjp_workspace_size", "rmsnorm_rope", "rmsnorm_rope_kv_append_ex",
          "rmsnorm_rope_axes", "rmsnorm_kv_append", "rmsnorm_kv_read", "rmsnorm_fwd_q8", "rmsnorm_kv_release", "rmsnorm_kv_plan")
_binding = None


def binding():
    """The native marshalling module (csrc/binding.cpp), bound to the library.
    Raises if it was never built."""
    global _binding
    if _binding is None:
        c = lib()
        with _lock:
            if _binding is None:
                path = binding_path()
                if not os.path.exists(path):
                    raise RuntimeError(
                        "%s is missing: build it with `python -m rmsnorm_fwd_bwd_add_gb300.build`" % path)
                loader = importlib.machinery.ExtensionFileLoader("_binding", path)
                mod = importlib.util.module_from_spec(
                    importlib.util.spec_from_loader("_binding", loader))
                loader.exec_module(mod)
                mod.bind(check, {n: ctypes.cast(getattr(c, n), ctypes.c_void_p).value for n in _BOUND})
                _binding = mod
    return _binding


def check(fn: str, status: int) -> None:
    if status != 0:
        detail = ""
        if status == 3:
            detail = "cudaError %d" % lib().rmsnorm_last_cuda_error()
        raise RmsnormError(fn, status, detail)
