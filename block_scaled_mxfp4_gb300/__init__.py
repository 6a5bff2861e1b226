"""Python binding of the GB300 block-scaled MXFP4 GEMM C ABI (include/mxfp4_gemm.h).

    D[M,N] (bf16) = alpha * A[M,K] (mxfp4) * B[N,K]^T (mxfp4) + beta * C[M,N]

The functions named like the C entry points marshal arguments only (torch
tensors or raw integer pointers -> void*, the current torch stream by
default); every step of the computation runs in the library's CUDA kernels.
There is no CPU fallback: if the compiled library is missing, loading fails.
``gemm`` is a convenience wrapper that allocates D and the workspace with
torch and calls ``mxfp4_gemm``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import warnings
from typing import Optional

__all__ = [
    "Mxfp4Error", "lib", "library_path", "header_functions",
    "mxfp4_gemm", "mxfp4_gemm_ex", "mxfp4_gemm_prepacked", "mxfp4_gemm_noalloc",
    "mxfp4_gemm_host", "MXFP4_FLAG_B_STATIC",
    "mxfp4_scale_relayout", "mxfp4_scale_relayout2", "mxfp4_quantize",
    "mxfp4_plan_gemm", "mxfp4_gemm_workspace_size", "mxfp4_gemm_prepacked_workspace_size",
    "mxfp4_scale_relayout_size", "mxfp4_gemm_host_arena_size", "mxfp4_device_status",
    "mxfp4_wait_timeout_probe", "mxfp4_set_wait_limit",
    "mxfp4_strerror", "mxfp4_version",
    "mxfp8_gemm", "mxfp8_gemm_prepacked", "mxfp8_plan_gemm", "mxfp8_gemm_workspace_size",
    "mxfp8_gemm_prepacked_workspace_size", "mxfp8_quantize", "mxfp8_gemm_host",
    "mxfp8_gemm_host_arena_size", "nvfp4_gemm", "nvfp4_gemm_workspace_size",
    "MXFP8_E4M3", "MXFP8_E5M2", "MXFP6_E2M3", "MXFP6_E3M2", "MXFP4_E2M1_PADDED",
    "mxfp4_moe_route", "mxfp4_moe_route_workspace_size", "mxfp4_group_scale_size",
    "mxfp4_group_quantize", "mxfp8_group_quantize", "mxfp4_grouped_gemm", "mxfp8_grouped_gemm",
    "mxfp4_grouped_swiglu", "mxfp8_grouped_swiglu", "mxfp4_grouped_workspace_size",
    "mxfp4_moe_combine", "mxfp4_moe_ffn", "mxfp4_moe_ffn_workspace_size",
    "MXFP4_LOGITS_BF16", "MXFP4_LOGITS_FP32", "MXFP4_GATE_TOPK", "MXFP4_GATE_ALL",
    "MXFP4_GATE_SIGMOID", "relaid_expert_scales", "moe_block",
    "gemm", "Plan",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
HEADER = os.path.join(_ROOT, "include", "mxfp4_gemm.h")
_LIB_NAME = "libmxfp4_gb300.so"

MXFP4_OK = 0
MXFP4_FLAG_B_STATIC = 1
MXFP8_E4M3, MXFP8_E5M2, MXFP6_E2M3, MXFP6_E3M2, MXFP4_E2M1_PADDED = 0, 1, 3, 4, 5
MXFP4_LOGITS_BF16, MXFP4_LOGITS_FP32 = 0, 1
MXFP4_GATE_TOPK, MXFP4_GATE_ALL, MXFP4_GATE_SIGMOID = 0, 1, 2
STATUS_NAMES = {0: "MXFP4_OK", -1: "MXFP4_ERR_INVALID_ARG", -2: "MXFP4_ERR_UNSUPPORTED_SHAPE",
                -3: "MXFP4_ERR_MISALIGNED", -4: "MXFP4_ERR_WORKSPACE", -5: "MXFP4_ERR_CUDA",
                -6: "MXFP4_ERR_TIMEOUT", -7: "MXFP4_ERR_ARCH"}


class Mxfp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} ({status})")


def library_path() -> str:
    return os.path.join(_PKG, _LIB_NAME)


class Plan(ctypes.Structure):
    _fields_ = [("swap_ab", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("tile_k", ctypes.c_int), ("stages", ctypes.c_int), ("split_k", ctypes.c_int),
                ("k_tiles_per_split", ctypes.c_int), ("grid_x", ctypes.c_int),
                ("grid_y", ctypes.c_int), ("grid_z", ctypes.c_int),
                ("workspace_bytes", ctypes.c_size_t), ("relayout_pass", ctypes.c_int),
                ("pair", ctypes.c_int), ("ctas", ctypes.c_int), ("waves", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


_lib = None


def lib() -> ctypes.CDLL:
    """Load the compiled library (build it first with block_scaled_mxfp4_gb300.build)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is missing: the CUDA library must be built "
                              "(python -m block_scaled_mxfp4_gb300.build); there is no fallback")
        L = ctypes.CDLL(path)
        vp, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                 ctypes.c_float, ctypes.c_size_t)
        sigs = {
            "mxfp4_plan_gemm": (i32, [i32, i32, i32, i32, i32, ctypes.POINTER(Plan)]),
            "mxfp4_gemm_workspace_size": (sz, [i32, i32, i32, i32]),
            "mxfp4_gemm_prepacked_workspace_size": (sz, [i32, i32, i32, i32]),
            "mxfp4_scale_relayout_size": (sz, [i32, i32]),
            "mxfp4_gemm_host_arena_size": (sz, [i32, i32, i32, i32, i32]),
            "mxfp4_scale_relayout": (i32, [vp, vp, i32, i32, i64, vp]),
            "mxfp4_scale_relayout2": (i32, [vp, vp, i32, i64, vp, vp, i32, i64, i32, vp]),
            "mxfp4_quantize": (i32, [vp, i64, vp, i64, vp, i64, i32, i32, vp]),
            "mxfp4_gemm": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                 f32, f32, i32, i32, i32, i32, vp, sz, vp]),
            "mxfp4_gemm_ex": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                    f32, f32, i32, i32, i32, i32, ctypes.c_uint, vp, sz, vp]),
            "mxfp8_gemm": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                 i32, i32, f32, f32, i32, i32, i32, i32, vp, sz, vp]),
            "mxfp8_gemm_prepacked": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp, i32, i32,
                                           f32, f32, i32, i32, i32, i32, vp, sz, vp]),
            "mxfp8_gemm_prepacked_workspace_size": (sz, [i32, i32, i32, i32]),
            "mxfp8_plan_gemm": (i32, [i32, i32, i32, i32, i32, ctypes.POINTER(Plan)]),
            "mxfp8_quantize": (i32, [vp, i64, vp, i64, vp, i64, i32, i32, i32, vp]),
            "mxfp8_gemm_workspace_size": (sz, [i32, i32, i32, i32]),
            "nvfp4_gemm": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                 f32, f32, i32, i32, i32, vp, sz, vp]),
            "nvfp4_gemm_workspace_size": (sz, [i32, i32, i32]),
            "mxfp4_gemm_prepacked": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, vp, vp,
                                           f32, f32, i32, i32, i32, i32, vp, sz, vp]),
            "mxfp4_gemm_noalloc": (i32, [vp, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                         f32, f32, i32, i32, i32, i32, vp]),
            "mxfp4_gemm_host": (i32, [vp, vp, vp, vp, vp, vp, f32, f32, i32, i32, i32, i32,
                                      vp, sz, vp]),
            "mxfp8_gemm_host": (i32, [vp, vp, vp, vp, vp, vp, i32, i32, f32, f32, i32, i32, i32,
                                      i32, vp, sz, vp]),
            "mxfp8_gemm_host_arena_size": (sz, [i32, i32, i32, i32, i32]),
            "mxfp4_moe_route": (i32, [vp, vp, vp, vp, vp, vp, i64, i32, vp, i32, i32, i32, i32, f32,
                                      vp, sz, vp]),
            "mxfp4_moe_route_workspace_size": (sz, [i32, i32]),
            "mxfp4_group_scale_size": (sz, [i32, i32, i32]),
            "mxfp4_group_quantize": (i32, [vp, i64, vp, vp, i64, i32, i32, vp, vp, i32, vp, i32, i32,
                                           vp]),
            "mxfp8_group_quantize": (i32, [vp, i64, vp, vp, i64, i32, i32, vp, vp, i32, vp, i32, i32,
                                           i32, vp]),
            "mxfp4_grouped_gemm": (i32, [vp, i64, vp, i64, vp, vp, i64, i64, vp, vp, i32, i32, i32,
                                         i32, f32, vp, sz, vp]),
            "mxfp8_grouped_gemm": (i32, [vp, i64, vp, i64, vp, vp, i64, i64, vp, vp, i32, i32, i32,
                                         i32, i32, i32, f32, vp, sz, vp]),
            "mxfp4_grouped_swiglu": (i32, [vp, i64, vp, vp, i64, vp, vp, i64, i64, vp, vp, i32, i32,
                                           i32, i32, f32, vp, sz, vp]),
            "mxfp8_grouped_swiglu": (i32, [vp, i64, vp, vp, i64, vp, vp, i64, i64, vp, vp, i32, i32,
                                           i32, i32, i32, i32, i32, f32, vp, sz, vp]),
            "mxfp4_grouped_workspace_size": (sz, [i32, i32, i32, i32]),
            "mxfp4_moe_combine": (i32, [vp, i64, vp, i64, vp, i64, i32, vp, vp, i32, vp, i64, vp, vp,
                                        f32, f32, f32, i32, i32, vp]),
            "mxfp4_moe_ffn": (i32, [vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, i32, i32, i32, i32,
                                    i32, vp, i64, vp, vp, i64, vp, vp, i64, vp, vp, f32, f32, f32,
                                    vp, sz, vp]),
            "mxfp4_moe_ffn_workspace_size": (sz, [i32, i32, i32, i32, i32]),
            "mxfp4_device_status": (i32, [ctypes.POINTER(ctypes.c_int), i32]),
            "mxfp4_wait_timeout_probe": (i32, [ctypes.c_longlong, vp]),
            "mxfp4_set_wait_limit": (None, [ctypes.c_longlong]),
            "mxfp4_strerror": (ctypes.c_char_p, [i32]),
            "mxfp4_version": (i32, []),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _bind_entries(L)
        _lib = L
    return _lib


def _raise(status, where):
    raise Mxfp4Error(status, where)


_python_entries = {}        # what _bind_entries replaced


def _entry_module():
    """The extension module built for this interpreter, by its full path: one
    built for another would be found by its name alone."""
    import importlib.util
    from .build import BINDING_LIB
    spec = importlib.util.spec_from_file_location(__name__ + "._entry", BINDING_LIB)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _bind_entries(L):
    """Replace the calls of a decoding step by the extension module's, which
    take the same arguments, by place or by name, and marshal them in C."""
    try:
        entry = _entry_module()
    except ImportError as e:
        warnings.warn(f"the Python binding's fast path cannot be loaded ({e}): the expert-layer "
                      "calls are marshalled in Python, some 2 us slower each")
        return
    names = [n for n in dir(entry) if n.startswith("mxfp")]
    entry.bind({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names}, _p,
               _current_stream, _raise)
    for n in names:
        _python_entries[n] = globals()[n]
        globals()[n] = getattr(entry, n)


def header_functions(path: str = HEADER):
    """Names of the functions declared in the public header."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(mxfp4_\w+)\s*\(", text)))


def _p(x) -> Optional[int]:
    """Tensor / integer / None -> raw pointer value."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    try:
        return x.data_ptr()
    except AttributeError:
        pass
    if hasattr(x, "ctypes"):                      # numpy array
        return x.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(x)}")


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_raw_stream = None


def _current_stream() -> int:
    """torch's current stream of the current device, as a handle."""
    global _raw_stream
    import torch
    if _raw_stream is None:
        # The handle alone where torch offers it: no Stream object per call.
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda device: torch.cuda.current_stream(device).cuda_stream)
    return _raw_stream(torch.cuda.current_device())


def _check(status: int, where: str) -> int:
    if status != MXFP4_OK:
        raise Mxfp4Error(status, where)
    return status


def mxfp4_plan_gemm(M, N, K, split_k=0, num_sms=0) -> Plan:
    plan = Plan()
    _check(lib().mxfp4_plan_gemm(M, N, K, split_k, num_sms, ctypes.byref(plan)), "mxfp4_plan_gemm")
    return plan


def mxfp4_gemm_workspace_size(M, N, K, split_k=0) -> int:
    return lib().mxfp4_gemm_workspace_size(M, N, K, split_k)


def mxfp4_gemm_prepacked_workspace_size(M, N, K, split_k=0) -> int:
    return lib().mxfp4_gemm_prepacked_workspace_size(M, N, K, split_k)


def mxfp4_scale_relayout_size(rows, K) -> int:
    return lib().mxfp4_scale_relayout_size(rows, K)


def mxfp4_gemm_host_arena_size(M, N, K, split_k=0, with_c=False) -> int:
    return lib().mxfp4_gemm_host_arena_size(M, N, K, split_k, int(bool(with_c)))


def mxfp4_scale_relayout(dst, src, rows, K, ld_src, stream=None):
    return _check(lib().mxfp4_scale_relayout(_p(dst), _p(src), rows, K, ld_src, _stream(stream)),
                  "mxfp4_scale_relayout")


def mxfp4_scale_relayout2(dst_a, src_a, rows_a, ld_a, dst_b, src_b, rows_b, ld_b, K, stream=None):
    return _check(lib().mxfp4_scale_relayout2(_p(dst_a), _p(src_a), rows_a, ld_a, _p(dst_b),
                                              _p(src_b), rows_b, ld_b, K, _stream(stream)),
                  "mxfp4_scale_relayout2")


def mxfp4_quantize(Q, ldq, S, lds, X, ldx, rows, K, stream=None):
    return _check(lib().mxfp4_quantize(_p(Q), ldq, _p(S), lds, _p(X), ldx, rows, K,
                                       _stream(stream)), "mxfp4_quantize")


def mxfp4_gemm(D, ldd, C, ldc, A, lda, B, ldb, scaleA, ld_sa, scaleB, ld_sb, alpha, beta,
               M, N, K, split_k, workspace, workspace_bytes, stream=None):
    return _check(lib().mxfp4_gemm(_p(D), ldd, _p(C), ldc, _p(A), lda, _p(B), ldb, _p(scaleA),
                                   ld_sa, _p(scaleB), ld_sb, alpha, beta, M, N, K, split_k,
                                   _p(workspace), workspace_bytes, _stream(stream)), "mxfp4_gemm")


def mxfp4_gemm_ex(D, ldd, C, ldc, A, lda, B, ldb, scaleA, ld_sa, scaleB, ld_sb, alpha, beta,
                  M, N, K, split_k, flags, workspace, workspace_bytes, stream=None):
    """mxfp4_gemm with flags (MXFP4_FLAG_B_STATIC: the work before this call
    on the stream does not write B or scaleB, so B may be loaded early)."""
    return _check(lib().mxfp4_gemm_ex(_p(D), ldd, _p(C), ldc, _p(A), lda, _p(B), ldb, _p(scaleA),
                                      ld_sa, _p(scaleB), ld_sb, alpha, beta, M, N, K, split_k,
                                      flags, _p(workspace), workspace_bytes, _stream(stream)),
                  "mxfp4_gemm_ex")


def mxfp8_gemm(D, ldd, C, ldc, A, lda, B, ldb, scaleA, ld_sa, scaleB, ld_sb, fmt_a, fmt_b,
               alpha, beta, M, N, K, split_k, workspace, workspace_bytes, stream=None):
    """MXFP8 / MXFP6 GEMM (A, B: one byte per element, lda / ldb in elements)."""
    return _check(lib().mxfp8_gemm(_p(D), ldd, _p(C), ldc, _p(A), lda, _p(B), ldb, _p(scaleA),
                                   ld_sa, _p(scaleB), ld_sb, fmt_a, fmt_b, alpha, beta, M, N, K,
                                   split_k, _p(workspace), workspace_bytes, _stream(stream)),
                  "mxfp8_gemm")


def mxfp8_gemm_prepacked(D, ldd, C, ldc, A, lda, B, ldb, scaleA_relaid, scaleB_relaid, fmt_a,
                         fmt_b, alpha, beta, M, N, K, split_k, workspace, workspace_bytes,
                         stream=None):
    """MXFP8 GEMM on scales relaid by mxfp4_scale_relayout (with this K)."""
    return _check(lib().mxfp8_gemm_prepacked(_p(D), ldd, _p(C), ldc, _p(A), lda, _p(B), ldb,
                                             _p(scaleA_relaid), _p(scaleB_relaid), fmt_a, fmt_b,
                                             alpha, beta, M, N, K, split_k, _p(workspace),
                                             workspace_bytes, _stream(stream)),
                  "mxfp8_gemm_prepacked")


def nvfp4_gemm(D, ldd, C, ldc, A, lda, B, ldb, scaleA, ld_sa, scaleB, ld_sb, alpha, beta, M, N,
               K, workspace, workspace_bytes, stream=None):
    """NVFP4 GEMM: packed E2M1 A, B; one UE4M3 scale per 16 K (ld_sa, ld_sb >= K/16)."""
    return _check(lib().nvfp4_gemm(_p(D), ldd, _p(C), ldc, _p(A), lda, _p(B), ldb, _p(scaleA),
                                   ld_sa, _p(scaleB), ld_sb, alpha, beta, M, N, K,
                                   _p(workspace), workspace_bytes, _stream(stream)),
                  "nvfp4_gemm")


def nvfp4_gemm_workspace_size(M, N, K) -> int:
    return lib().nvfp4_gemm_workspace_size(M, N, K)


def mxfp8_quantize(Q, ldq, S, lds, X, ldx, rows, K, fmt, stream=None):
    """bf16 rows -> E4M3 / E5M2 codes (one per byte) + E8M0 scales."""
    return _check(lib().mxfp8_quantize(_p(Q), ldq, _p(S), lds, _p(X), ldx, rows, K, fmt,
                                       _stream(stream)), "mxfp8_quantize")


def mxfp8_gemm_prepacked_workspace_size(M, N, K, split_k=0) -> int:
    return lib().mxfp8_gemm_prepacked_workspace_size(M, N, K, split_k)


def mxfp8_plan_gemm(M, N, K, split_k=0, num_sms=0) -> Plan:
    plan = Plan()
    _check(lib().mxfp8_plan_gemm(M, N, K, split_k, num_sms, ctypes.byref(plan)), "mxfp8_plan_gemm")
    return plan


def mxfp8_gemm_workspace_size(M, N, K, split_k=0) -> int:
    return lib().mxfp8_gemm_workspace_size(M, N, K, split_k)


def mxfp4_gemm_noalloc(D, ldd, C, ldc, A, lda, B, ldb, scaleA, ld_sa, scaleB, ld_sb, alpha,
                       beta, M, N, K, split_k, stream=None):
    """mxfp4_gemm without a workspace argument, for callers that cannot
    allocate device memory: scratch comes from a fixed array in the library's
    device image (MXFP4_NOALLOC_SCRATCH_BYTES).  Calls that overlap on the GPU
    share that array and must be serialised by the caller."""
    return _check(lib().mxfp4_gemm_noalloc(_p(D), ldd, _p(C), ldc, _p(A), lda, _p(B), ldb,
                                           _p(scaleA), ld_sa, _p(scaleB), ld_sb, alpha, beta,
                                           M, N, K, split_k, _stream(stream)),
                  "mxfp4_gemm_noalloc")


def mxfp4_gemm_prepacked(D, ldd, C, ldc, A, lda, B, ldb, scaleA_relaid, scaleB_relaid, alpha,
                         beta, M, N, K, split_k, workspace, workspace_bytes, stream=None):
    return _check(lib().mxfp4_gemm_prepacked(_p(D), ldd, _p(C), ldc, _p(A), lda, _p(B), ldb,
                                             _p(scaleA_relaid), _p(scaleB_relaid), alpha, beta,
                                             M, N, K, split_k, _p(workspace), workspace_bytes,
                                             _stream(stream)), "mxfp4_gemm_prepacked")


def mxfp8_gemm_host(D_host, C_host, A_host, B_host, scaleA_host, scaleB_host, fmt_a, fmt_b,
                    alpha, beta, M, N, K, split_k, device_arena, arena_bytes, stream=None):
    """mxfp4_gemm_host for the byte forms of mxfp8_gemm (host arrays in and out)."""
    return _check(lib().mxfp8_gemm_host(_p(D_host), _p(C_host), _p(A_host), _p(B_host),
                                        _p(scaleA_host), _p(scaleB_host), fmt_a, fmt_b, alpha,
                                        beta, M, N, K, split_k, _p(device_arena), arena_bytes,
                                        _stream(stream)), "mxfp8_gemm_host")


def mxfp8_gemm_host_arena_size(M, N, K, split_k=0, with_c=False) -> int:
    return lib().mxfp8_gemm_host_arena_size(M, N, K, split_k, int(bool(with_c)))


def mxfp4_gemm_host(D_host, C_host, A_host, B_host, scaleA_host, scaleB_host, alpha, beta,
                    M, N, K, split_k, device_arena, arena_bytes, stream=None):
    return _check(lib().mxfp4_gemm_host(_p(D_host), _p(C_host), _p(A_host), _p(B_host),
                                        _p(scaleA_host), _p(scaleB_host), alpha, beta, M, N, K,
                                        split_k, _p(device_arena), arena_bytes, _stream(stream)),
                  "mxfp4_gemm_host")


def mxfp4_device_status(reset=False) -> int:
    st = ctypes.c_int(0)
    _check(lib().mxfp4_device_status(ctypes.byref(st), int(bool(reset))), "mxfp4_device_status")
    return st.value


def mxfp4_wait_timeout_probe(limit_cycles, stream=None):
    return _check(lib().mxfp4_wait_timeout_probe(limit_cycles, _stream(stream)),
                  "mxfp4_wait_timeout_probe")


def mxfp4_set_wait_limit(cycles):
    lib().mxfp4_set_wait_limit(cycles)


def mxfp4_strerror(status) -> str:
    return lib().mxfp4_strerror(status).decode()


def mxfp4_version() -> int:
    return lib().mxfp4_version()


def mxfp4_moe_route_workspace_size(T, E) -> int:
    return lib().mxfp4_moe_route_workspace_size(T, E)


def mxfp4_group_scale_size(rows, groups, K) -> int:
    return lib().mxfp4_group_scale_size(rows, groups, K)


def mxfp4_grouped_workspace_size(rows, groups, N, K) -> int:
    return lib().mxfp4_grouped_workspace_size(rows, groups, N, K)


def mxfp4_moe_ffn_workspace_size(T, E, k, K, F) -> int:
    return lib().mxfp4_moe_ffn_workspace_size(T, E, k, K, F)


def mxfp4_moe_route(ids, gates, offsets, row_token, slot_row, logits, ldl, logits_type, token_mask,
                    T, E, k, gate_mode, gate_scale, workspace, workspace_bytes, stream=None):
    """The k largest logits per token, their gates, and the rows' grouping by expert."""
    return _check(lib().mxfp4_moe_route(_p(ids), _p(gates), _p(offsets), _p(row_token),
                                        _p(slot_row), _p(logits), ldl, logits_type,
                                        _p(token_mask), T, E, k, gate_mode, gate_scale,
                                        _p(workspace), workspace_bytes, _stream(stream)),
                  "mxfp4_moe_route")


def mxfp4_group_quantize(Q, ldq, S, X, ldx, T, K, slot_row, ids, k, offsets, groups, rows,
                         stream=None):
    """bf16 rows -> packed E2M1 rows at their places in the grouping, grouped scales."""
    return _check(lib().mxfp4_group_quantize(_p(Q), ldq, _p(S), _p(X), ldx, T, K, _p(slot_row),
                                             _p(ids), k, _p(offsets), groups, rows,
                                             _stream(stream)), "mxfp4_group_quantize")


def mxfp8_group_quantize(Q, ldq, S, X, ldx, T, K, slot_row, ids, k, offsets, groups, rows, fmt,
                         stream=None):
    """mxfp4_group_quantize into E4M3 / E5M2 codes, one per byte."""
    return _check(lib().mxfp8_group_quantize(_p(Q), ldq, _p(S), _p(X), ldx, T, K, _p(slot_row),
                                             _p(ids), k, _p(offsets), groups, rows, fmt,
                                             _stream(stream)), "mxfp8_group_quantize")


def mxfp4_grouped_gemm(D, ldd, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, N, K,
                       alpha, workspace, workspace_bytes, stream=None):
    """D[r] = alpha * A[r] . B[e]^T for every row r of group e (bf16 out)."""
    return _check(lib().mxfp4_grouped_gemm(_p(D), ldd, _p(A), lda, _p(SA), _p(B), ldb, stride_b,
                                           _p(SB), _p(offsets), groups, rows, N, K, alpha,
                                           _p(workspace), workspace_bytes, _stream(stream)),
                  "mxfp4_grouped_gemm")


def mxfp8_grouped_gemm(D, ldd, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, N, K,
                       fmt_a, fmt_b, alpha, workspace, workspace_bytes, stream=None):
    """mxfp4_grouped_gemm on the byte formats of mxfp8_gemm."""
    return _check(lib().mxfp8_grouped_gemm(_p(D), ldd, _p(A), lda, _p(SA), _p(B), ldb, stride_b,
                                           _p(SB), _p(offsets), groups, rows, N, K, fmt_a, fmt_b,
                                           alpha, _p(workspace), workspace_bytes,
                                           _stream(stream)), "mxfp8_grouped_gemm")


def mxfp4_grouped_swiglu(H, ldh, SH, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, F, K,
                         alpha, workspace, workspace_bytes, stream=None):
    """H = quantise(silu(A . Bgate^T) * (A . Bup^T)) per group, packed E2M1."""
    return _check(lib().mxfp4_grouped_swiglu(_p(H), ldh, _p(SH), _p(A), lda, _p(SA), _p(B), ldb,
                                             stride_b, _p(SB), _p(offsets), groups, rows, F, K,
                                             alpha, _p(workspace), workspace_bytes,
                                             _stream(stream)), "mxfp4_grouped_swiglu")


def mxfp8_grouped_swiglu(H, ldh, SH, A, lda, SA, B, ldb, stride_b, SB, offsets, groups, rows, F, K,
                         fmt_a, fmt_b, fmt_h, alpha, workspace, workspace_bytes, stream=None):
    """mxfp4_grouped_swiglu on byte formats, into E4M3 / E5M2 codes."""
    return _check(lib().mxfp8_grouped_swiglu(_p(H), ldh, _p(SH), _p(A), lda, _p(SA), _p(B), ldb,
                                             stride_b, _p(SB), _p(offsets), groups, rows, F, K,
                                             fmt_a, fmt_b, fmt_h, alpha, _p(workspace),
                                             workspace_bytes, _stream(stream)),
                  "mxfp8_grouped_swiglu")


def mxfp4_moe_combine(H, ldh, Nrm, ldn, Y, ldy, rows, slot_row, gates, k, resid, ldr, w_post,
                      w_pre, res_scale, out_scale, eps, T, N, stream=None):
    """Gated sum of a token's rows, its norm, the residual stream and the next block's norm."""
    return _check(lib().mxfp4_moe_combine(_p(H), ldh, _p(Nrm), ldn, _p(Y), ldy, rows, _p(slot_row),
                                          _p(gates), k, _p(resid), ldr, _p(w_post), _p(w_pre),
                                          res_scale, out_scale, eps, T, N, _stream(stream)),
                  "mxfp4_moe_combine")


def mxfp4_moe_ffn(H, ldh, Nrm, ldn, X, ldx, ids, gates, offsets, slot_row, T, E, k, K, F, B1, ldb1,
                  SB1, B2, ldb2, SB2, resid, ldr, w_post, w_pre, res_scale, out_scale, eps,
                  workspace, workspace_bytes, stream=None):
    """A routed feed-forward block on MXFP4 weights: quantise, both products, join."""
    return _check(lib().mxfp4_moe_ffn(_p(H), ldh, _p(Nrm), ldn, _p(X), ldx, _p(ids), _p(gates),
                                      _p(offsets), _p(slot_row), T, E, k, K, F, _p(B1), ldb1,
                                      _p(SB1), _p(B2), ldb2, _p(SB2), _p(resid), ldr, _p(w_post),
                                      _p(w_pre), res_scale, out_scale, eps, _p(workspace),
                                      workspace_bytes, _stream(stream)), "mxfp4_moe_ffn")


def _on_stream(stream, inputs, outputs):
    """A context with `stream` (an object, a handle, or None for the current one)
    as torch's current stream, so that what the body allocates, copies and drops
    belongs to it.  `inputs` are marked as used on it, and what the body puts
    into the list `outputs` as used on the caller's stream too.  Order between
    the two streams is the caller's, as for every entry point."""
    import torch
    if stream is None or _stream(stream) == torch.cuda.current_stream().cuda_stream:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return _other_stream(stream, inputs, outputs)


@contextlib.contextmanager
def _other_stream(stream, inputs, outputs):
    import torch
    caller = torch.cuda.current_stream()
    try:
        with torch.cuda.stream(stream):
            yield
    finally:
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
        for t in outputs:
            t.record_stream(caller)


def _refuse(what, error=ValueError):
    raise error(f"{what} expected")


def relaid_expert_scales(S, K, stream=None):
    """Row-major weight scales [..., rows, K / 32] -> one relaid buffer per
    matrix [..., mxfp4_scale_relayout_size(rows, K)], laid out once for the
    grouped products."""
    import torch
    if S.dim() < 2 or S.shape[-1] * 32 != K:
        _refuse(f"relaid_expert_scales: S [..., rows, {K} / 32]")
    if S.element_size() != 1:
        _refuse("relaid_expert_scales: S one byte per scale", TypeError)
    if not S.is_cuda:
        _refuse("relaid_expert_scales: S on the GPU")
    rows = S.shape[-2]
    size = mxfp4_scale_relayout_size(rows, K)
    made = []
    with _on_stream(stream, [S], made):
        flat = S.reshape(-1, rows, K // 32).contiguous()
        out = torch.empty((flat.shape[0], size), dtype=torch.uint8, device=S.device)
        made.append(out)
        for i in range(flat.shape[0]):
            mxfp4_scale_relayout(out[i], flat[i], rows, K, K // 32)
    return out.reshape(*S.shape[:-2], size)


def _check_block(x, logits, resid, w1, s1, w2, s2, w_pre, w_post, token_mask):
    """The entries below take pointers; this is where types and layouts are seen."""
    import torch
    if x.dim() != 2 or w1.dim() != 4 or w1.shape[1] != 2:
        _refuse("moe_block: x [T, K], w1 [E, 2, F, K / 2]")
    (T, K), (E, _, F, _) = x.shape, w1.shape
    bf16, one_gpu = (torch.bfloat16,), x.is_cuda
    for name, t, shape, types in (
            ("x", x, (T, K), bf16), ("resid", resid, (T, K), bf16),
            ("logits", logits, (T, E), (torch.bfloat16, torch.float32)),
            ("w_pre", w_pre, (K,), bf16), ("w_post", w_post, (K,), bf16),
            ("token_mask", token_mask, (T,), (torch.uint8, torch.bool, torch.int8))):
        if t is None and name in ("w_pre", "w_post", "token_mask"):
            continue
        if t.dtype not in types:
            _refuse(f"moe_block: {name} of type {' or '.join(map(str, types))}", TypeError)
        if t.shape != shape:
            _refuse(f"moe_block: {name} of shape {shape}")
        if t.stride(-1) != 1 and shape[-1] != 1 and t.numel():
            _refuse(f"moe_block: {name} with neighbouring elements side by side")
        one_gpu = one_gpu and t.device == x.device
    size1, size2 = mxfp4_scale_relayout_size(F, K), mxfp4_scale_relayout_size(K, F)
    for name, t, size, shape in (("w1", w1, E * F * K, (E, 2, F, K // 2)),
                                 ("w2", w2, E * K * F // 2, (E, K, F // 2)),
                                 ("s1", s1, 2 * E * size1, None), ("s2", s2, E * size2, None)):
        if t.element_size() != 1:
            _refuse(f"moe_block: {name} of bytes", TypeError)
        if t.numel() != size or (shape and t.shape != shape) or not t.is_contiguous():
            _refuse(f"moe_block: {name} contiguous, " +
                    (f"of shape {shape}" if shape else f"{size} bytes from relaid_expert_scales"))
        one_gpu = one_gpu and t.device == x.device
    if not one_gpu:
        _refuse("moe_block: everything on one GPU")


def moe_block(x, logits, resid, w1, s1, w2, s2, k, w_pre=None, w_post=None, token_mask=None,
              gate_mode=MXFP4_GATE_TOPK, res_scale=1.0, out_scale=1.0, eps=1e-6, stream=None):
    """A mixture-of-experts block on MXFP4 weights, from the router's logits on.

    x bf16 [T, K] (the block's normed input), logits bf16 / fp32 [T, E], resid
    bf16 [T, K], w1 uint8 [E, 2, F, K / 2], w2 uint8 [E, K, F / 2], s1 and s2
    from relaid_expert_scales.  Returns (h, n): the residual stream after the
    block and its norm, bf16 [T, K].  On another `stream` than the current one
    the block's own memory belongs to that stream; the caller orders the two.
    Rows of x, logits and resid may be apart; other types or layouts raise
    TypeError or ValueError.
    """
    import torch
    _check_block(x, logits, resid, w1, s1, w2, s2, w_pre, w_post, token_mask)
    T, K = x.shape
    E, F = w1.shape[0], w1.shape[2]
    need = max(mxfp4_moe_route_workspace_size(T, E), mxfp4_moe_ffn_workspace_size(T, E, k, K, F))
    kind = MXFP4_LOGITS_FP32 if logits.dtype == torch.float32 else MXFP4_LOGITS_BF16
    ld = lambda t: t.stride(0) if T > 1 else t.shape[1]    # (a lone row's stride can be anything)
    made = []
    with _on_stream(stream, [x, logits, resid, w1, s1, w2, s2, w_pre, w_post, token_mask], made):
        # ids, gates, row_token and slot_row [T, k] of 4 bytes, offsets [E + 1]: one array.
        tables = torch.empty(4 * T * k + E + 1, dtype=torch.int32, device=x.device)
        ids, gates, row_token, slot_row, offsets = (tables.data_ptr() + 4 * T * k * i
                                                    for i in range(5))
        h = torch.empty((T, K), dtype=torch.bfloat16, device=x.device)
        n = torch.empty_like(h)
        made += [h, n]
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
        mxfp4_moe_route(ids, gates, offsets, row_token, slot_row, logits, ld(logits), kind,
                        token_mask, T, E, k, gate_mode, 1.0, ws, ws.numel())
        mxfp4_moe_ffn(h, K, n, K, x, ld(x), ids, gates, offsets, slot_row, T, E, k, K, F, w1, K,
                      s1, w2, F, s2, resid, ld(resid), w_post, w_pre, float(res_scale),
                      float(out_scale), float(eps), ws, ws.numel())
    return h, n


def gemm(A, B, SA, SB, alpha=1.0, beta=0.0, C=None, split_k=0, out=None, workspace=None,
         stream=None):
    """D = alpha * A . B^T + beta * C on device tensors.

    A [M, K/2], B [N, K/2] uint8 (packed E2M1), SA [M, K/32], SB [N, K/32]
    uint8 (E8M0), C [M, N] bfloat16 or None.  Returns D [M, N] bfloat16.
    """
    import torch
    M, N, K = A.shape[0], B.shape[0], A.shape[1] * 2
    need = mxfp4_gemm_workspace_size(M, N, K, split_k)
    made = []
    with _on_stream(stream, [A, B, SA, SB, C, out, workspace], made):
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
            made.append(out)
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=A.device)
        mxfp4_gemm(out, out.stride(0), C, 0 if C is None else C.stride(0), A, A.stride(0) * 2,
                   B, B.stride(0) * 2, SA, SA.stride(0), SB, SB.stride(0), float(alpha),
                   float(beta), M, N, K, split_k, workspace, workspace.numel())
    return out
