"""Python binding of libq4gemv.so, the GB300 int4 weight-streaming GEMV library.

The functions here carry the C ABI's names (include/q4gemv.h) and only
marshal arguments: torch tensors (or raw integer device addresses) become
pointers, sizes are read off the tensors when not given, and the current
torch CUDA stream is passed unless another is named.  (The mixture-of-experts
calls and those for several continuations of one prompt take tensors only,
whose types and shapes they check; a program with raw addresses calls the C ABI
through lib().)  Every step of the
computation runs in the library's CUDA kernels; there is no fallback of any
kind -- if the shared library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

__all__ = [
    "Q4Error", "lib", "library_path", "exported_names",
    "q4gemv_pack_info", "q4gemv_run", "q4gemv_fused_run", "q4gemv_grouped_run", "q4_0_gemv_run", "q8_0_gemv_run",
    "q4gemm_run", "q4gemv_run_ex", "q4gemv_fused_run_ex", "q4gemv_grouped_run_ex", "q4gemm_run_ex",
    "f32gemv_run",
    "q4gemv_status_string", "q4gemv_last_cuda_error",
    "q4_dequant_f32_run", "q4_dequant_bf16_run", "vec4_read_probe_run",
    "q4gemv_device_status", "q4gemm_set_wait_timeout_ns", "q4gemv_set_overlapped_launch",
    "q4gemv_bounds_violations", "q4gemv_grouped_split",
    "q4moe_route_run", "q4moe_route_workspace", "q4moe_gemm_run", "q4moe_gemm_workspace",
    "q4_block_norm_run", "q4moe_block_run", "q4moe_block_workspace",
    "q4_rope_append_run", "q4_rope_frequencies", "q4_prefix_attn_run", "q4_prefix_attn_workspace",
    "q4_beam_step_run", "q4_beam_step_workspace", "q4_beam_reorder_run",
    "Q4_F16", "Q4_ROPE_HALF", "Q4_ROPE_INTERLEAVED", "Q4_ROPE_PLAIN", "Q4_ROPE_LINEAR", "Q4_ROPE_BANDS",
    "Q4_F32", "Q4_BF16", "Q4_ROUTE_SOFTMAX", "Q4_ROUTE_SIGMOID", "Q4_ROUTE_SCORE_BIAS",
    "Q4_OK", "Q4_ERR_INVALID_ARG", "Q4_ERR_UNSUPPORTED", "Q4_ERR_MISALIGNED",
    "Q4_ERR_CUDA", "Q4_ERR_TIMEOUT", "Q4_EPILOGUE_NONE", "Q4_EPILOGUE_SWIGLU",
    "Q4_RUN_OVERLAPPED", "Q4_RUN_EXACT_X", "Q4_RUN_WAIT_TIMEOUT",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_HERE)
HEADER = os.path.join(_ROOT, "include", "q4gemv.h")

Q4_OK, Q4_ERR_INVALID_ARG, Q4_ERR_UNSUPPORTED, Q4_ERR_MISALIGNED, Q4_ERR_CUDA, Q4_ERR_TIMEOUT = range(6)
Q4_EPILOGUE_NONE, Q4_EPILOGUE_SWIGLU = 0, 1
Q4_RUN_OVERLAPPED, Q4_RUN_EXACT_X, Q4_RUN_WAIT_TIMEOUT = 0x1, 0x2, 0x4
Q4_F32, Q4_BF16, Q4_F16 = 0, 1, 2
Q4_ROUTE_SOFTMAX, Q4_ROUTE_SIGMOID, Q4_ROUTE_SCORE_BIAS = 0, 1, 0x10
Q4_ROPE_HALF, Q4_ROPE_INTERLEAVED = 0, 1
Q4_ROPE_PLAIN, Q4_ROPE_LINEAR, Q4_ROPE_BANDS = 0, 1, 2


def library_path() -> str:
    return os.path.join(_HERE, "libq4gemv.so")


class Q4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = f"{where}: {q4gemv_status_string(status)} (status {status})"
        if status == Q4_ERR_CUDA:
            msg += f" [{q4gemv_last_cuda_error()}]"
        super().__init__(msg)


class _PackInfo(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64), ("group", ctypes.c_int32),
                ("blocks_per_row", ctypes.c_int32), ("codes_row_bytes", ctypes.c_int64),
                ("codes_bytes", ctypes.c_int64), ("scales_row_bytes", ctypes.c_int64),
                ("scales_bytes", ctypes.c_int64), ("zeros_row_bytes", ctypes.c_int64),
                ("zeros_bytes", ctypes.c_int64), ("base_alignment", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class _RunOptions(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32), ("wait_timeout_ns", ctypes.c_uint64)]


class _Segment(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales_f16", ctypes.c_void_p), ("zeros_u4_or_null", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int64)]


class _BlockNorm(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("top_k", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("R", ctypes.c_int64), ("y", ctypes.c_void_p), ("pos", ctypes.c_void_p), ("weights", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("post_gamma", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("gate_stride", ctypes.c_int64), ("pre_gamma", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("out_norm", ctypes.c_void_p), ("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)]


class _MoeBlock(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "E", "top_k", "H", "inner", "group", "dtype", "score",
                                               "renormalize")] +
                [(n, ctypes.c_float) for n in ("route_scale", "residual_scale", "eps")] +
                [(n, ctypes.c_void_p) for n in ("up_codes", "up_scales_f16", "up_zeros_u4_or_null", "down_codes",
                                                "down_scales_f16", "down_zeros_u4_or_null", "logits", "bias_or_null",
                                                "token_mask_or_null", "a", "x", "post_gamma", "gate")] +
                [("gate_stride", ctypes.c_int64)] +
                [(n, ctypes.c_void_p) for n in ("pre_gamma", "ids", "route_weights", "out", "out_norm",
                                                "workspace")] +
                [("workspace_bytes", ctypes.c_int64)])


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("D", ctypes.c_int32), ("page", ctypes.c_int32), ("pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class _RopeAppend(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("T", "Hq", "dtype", "rot", "layout")] +
                [("scale", ctypes.c_float), ("eps", ctypes.c_float)] +
                [(n, ctypes.c_void_p) for n in ("q", "k", "v")] +
                [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")] +
                [(n, ctypes.c_void_p) for n in ("q_gamma", "k_gamma", "positions", "inv_freq", "slots", "q_out")] +
                [("cache", _KvCache)])


class _PrefixAttn(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("S", "Hq", "groups", "out_dtype", "max_shared_pages",
                                               "max_own_pages")] +
                [("scale", ctypes.c_float), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                 ("cache", _KvCache)] +
                [(n, ctypes.c_void_p) for n in ("group_offsets", "shared_pages", "shared_lens", "limits", "own_pages",
                                                "own_lens", "out", "lse", "workspace")] +
                [("workspace_bytes", ctypes.c_int64)])


class _BeamReorder(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("groups", "W", "max_pages", "planes", "heads", "page")] +
                [(n, ctypes.c_int64) for n in ("pages", "row_bytes", "plane_stride", "page_stride", "head_stride",
                                               "row_stride")] +
                [(n, ctypes.c_void_p) for n in ("pool", "tables", "lens", "parents", "spare", "out_tables",
                                                "out_spare")])


_lock = threading.Lock()
_lib = None
_vp, _i32, _i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64


def lib() -> ctypes.CDLL:
    """Load libq4gemv.so (built by gemm_decode_gb300.build); raises if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise OSError(f"{path} is missing: build it with "
                              "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(path)
            L.q4gemv_pack_info.argtypes = [_i64, _i64, _i32, ctypes.POINTER(_PackInfo)]
            L.q4gemv_run.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _vp]
            L.q4gemv_fused_run.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _i32, _i64, _i64,
                                           _i32, _i32, _vp]
            L.q4gemm_run.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _vp]
            _opt = ctypes.POINTER(_RunOptions)
            L.q4gemv_run_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _opt, _vp]
            L.q4gemv_fused_run_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _i32, _i64, _i64,
                                              _i32, _i32, _opt, _vp]
            L.q4gemv_grouped_run_ex.argtypes = [ctypes.POINTER(_Segment), _i32, _i64, _i32, _opt, _vp]
            L.q4gemm_run_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i32, _opt, _vp]
            L.q4_0_gemv_run.argtypes = [_vp, _vp, _vp, _i32, _i64, _i64, _vp]
            L.q8_0_gemv_run.argtypes = [_vp, _vp, _vp, _i32, _i64, _i64, _vp]
            L.q4gemv_grouped_run.argtypes = [ctypes.POINTER(_Segment), _i32, _i64, _i32, _vp]
            L.f32gemv_run.argtypes = [_vp, _vp, _vp, _i32, _i64, _i64, _vp]
            L.q4gemv_status_string.argtypes = [ctypes.c_int]
            L.q4gemv_status_string.restype = ctypes.c_char_p
            L.q4gemv_last_cuda_error.argtypes = []
            L.q4gemv_last_cuda_error.restype = ctypes.c_char_p
            L.q4_dequant_f32_run.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]
            L.q4_dequant_bf16_run.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp]
            L.vec4_read_probe_run.argtypes = [_vp, _i64, _vp, _i32, ctypes.POINTER(_i32), _vp]
            L.q4gemv_device_status.argtypes = [_vp]
            L.q4gemm_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
            L.q4gemv_set_overlapped_launch.argtypes = [ctypes.c_int]
            L.q4gemv_bounds_violations.argtypes = [_vp]
            L.q4gemv_grouped_split.argtypes = [ctypes.POINTER(_i64), _i32, _i64, _i32, _i32,
                                               ctypes.POINTER(_i32), ctypes.POINTER(_i32)]
            L.q4moe_route_workspace.argtypes = [_i32, _i32, _i32]
            L.q4moe_gemm_workspace.argtypes = [_i64, _i64, _i64, _i64, _i32, _i32]
            L.q4moe_block_workspace.argtypes = [_i32] * 6
            for f in ("q4moe_route_workspace", "q4moe_gemm_workspace", "q4moe_block_workspace"):
                getattr(L, f).restype = _i64
            L.q4moe_route_run.argtypes = [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, ctypes.c_float, _vp, _vp, _vp,
                                          _vp, _vp, _vp, _i64, _opt, _vp]
            L.q4moe_gemm_run.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _i64, _i32, _i32,
                                         _i32, _vp, _i64, _opt, _vp]
            L.q4_block_norm_run.argtypes = [ctypes.POINTER(_BlockNorm), _opt, _vp]
            L.q4moe_block_run.argtypes = [ctypes.POINTER(_MoeBlock), _opt, _vp]
            # (the structures as bytes)
            L.q4_rope_append_run.argtypes = [_vp, _opt, _vp]
            _f64 = ctypes.c_double
            L.q4_rope_frequencies.argtypes = [ctypes.POINTER(ctypes.c_float), _i32, _f64, _i32, _f64, _f64, _f64, _f64]
            L.q4_prefix_attn_workspace.argtypes = [_i32] * 5
            L.q4_prefix_attn_run.argtypes = [_vp, _opt, _vp]
            L.q4_beam_step_workspace.argtypes = [_i32, _i32, _i32, _i64]
            L.q4_beam_step_run.argtypes = [_vp, _i64, _vp, _vp, _i32, _i32, _i32, _i64, _i32, _vp, _vp, _vp, _vp, _vp,
                                           _i64, _opt, _vp]
            L.q4_beam_reorder_run.argtypes = [_vp, _opt, _vp]
            for f in ("q4_prefix_attn_workspace", "q4_beam_step_workspace"):
                getattr(L, f).restype = _i64
            for f in ("q4_rope_append_run", "q4_rope_frequencies", "q4_prefix_attn_run", "q4_beam_step_run",
                      "q4_beam_reorder_run", "q4moe_route_run", "q4moe_gemm_run", "q4_block_norm_run", "q4moe_block_run",
                      "q4gemv_pack_info", "q4gemv_run", "q4gemv_fused_run", "q4gemv_grouped_run", "q4_0_gemv_run",
                      "q8_0_gemv_run",
                      "q4gemm_run", "f32gemv_run", "q4gemv_run_ex", "q4gemv_fused_run_ex", "q4gemv_grouped_run_ex",
                      "q4gemm_run_ex",
                      "q4_dequant_f32_run", "q4_dequant_bf16_run", "vec4_read_probe_run",
                      "q4gemv_device_status", "q4gemm_set_wait_timeout_ns",
                      "q4gemv_set_overlapped_launch", "q4gemv_bounds_violations", "q4gemv_grouped_split"):
                getattr(L, f).restype = ctypes.c_int
            _lib = L
        return _lib


def exported_names():
    """Function names declared in include/q4gemv.h."""
    text = open(HEADER).read()
    return re.findall(r"^Q4_API\s+[\w\s\*]*?\b(\w+)\s*\(", text, flags=re.M)


# ------------------------------------------------------------------ marshalling

def _addr(t, name="argument", esize=0):
    """Address of an array argument: None and integer addresses pass through as given;
    a tensor must be contiguous (the library reads packed row-major arrays) and, where
    esize is set, hold elements of esize bytes.  Metadata checks only: where the memory
    lives and how large it is stay the caller's responsibility, as in the C ABI."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is required (got strides {tuple(t.stride())})")
    if esize and t.element_size() != esize:
        raise ValueError(f"{name}: {esize}-byte elements expected, got {t.dtype}")
    return t.data_ptr()


_raw_stream = None


def _current_stream():
    """The current torch CUDA stream's address (without building a Stream object where torch
    offers that: a third of the time)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        try:
            of, dev = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
            of(dev())
            _raw_stream = lambda: of(dev())  # noqa: E731
        except (AttributeError, RuntimeError):
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(st: int, where: str):
    if st != Q4_OK:
        raise Q4Error(st, where)


def q4gemv_status_string(status: int) -> str:
    return lib().q4gemv_status_string(int(status)).decode()


def q4gemv_last_cuda_error() -> str:
    return lib().q4gemv_last_cuda_error().decode()


def q4gemv_pack_info(N: int, K: int, group: int) -> dict:
    info = _PackInfo()
    _check(lib().q4gemv_pack_info(N, K, group, ctypes.byref(info)), "q4gemv_pack_info")
    return {name: getattr(info, name) for name, _ in _PackInfo._fields_ if name != "reserved"}


def _mnk_q4(codes, x, M, N, K):
    if M is None:
        M = x.shape[0]
    if N is None:
        N = codes.shape[0]
    if K is None:
        K = x.shape[1]
    return int(M), int(N), int(K)


def q4gemv_run(codes, scales_f16, zeros_u4_or_null, x, y, M=None, N=None, K=None, group=32,
               stream=None, check=True) -> int:
    M, N, K = _mnk_q4(codes, x, M, N, K)
    st = lib().q4gemv_run(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                          _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _addr(x, "x", 4),
                          _addr(y, "y", 4), M, N, K, int(group), _stream(stream))
    if check:
        _check(st, "q4gemv_run")
    return st


def q4gemv_fused_run(codes, scales_f16, zeros_u4_or_null, x, gamma, eps, y, M=None, N=None, K=None, group=32,
                     epilogue=Q4_EPILOGUE_NONE, stream=None, check=True) -> int:
    M, N, K = _mnk_q4(codes, x, M, N, K)
    st = lib().q4gemv_fused_run(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                                _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _addr(x, "x", 4),
                                _addr(gamma, "gamma", 4), float(eps), _addr(y, "y", 4), M, N, K, int(group),
                                int(epilogue), _stream(stream))
    if check:
        _check(st, "q4gemv_fused_run")
    return st


def q4gemv_grouped_run(segments, K, group=32, stream=None, check=True) -> int:
    """segments: (codes, scales_f16, zeros_or_None, x, y[, N]) per matrix, M = 1 each;
    N defaults to codes.shape[0]."""
    arr = (_Segment * max(1, len(segments)))()
    for i, sg in enumerate(segments):
        codes, scales, zeros, x, y = sg[:5]
        N = int(sg[5]) if len(sg) > 5 else int(codes.shape[0])
        arr[i] = _Segment(_addr(codes, "codes", 1), _addr(scales, "scales_f16", 2), _addr(zeros, "zeros_u4_or_null", 1),
                          _addr(x, "x", 4), _addr(y, "y", 4), N)
    st = lib().q4gemv_grouped_run(arr, len(segments), int(K), int(group), _stream(stream))
    if check:
        _check(st, "q4gemv_grouped_run")
    return st


def _options(flags, wait_timeout_ns, reserved=0):
    """Per-call options of the *_ex entry points (None: a NULL pointer, the defaults)."""
    if flags is None and wait_timeout_ns is None and not reserved:
        return None
    f = int(flags or 0)
    if wait_timeout_ns is not None:
        f |= Q4_RUN_WAIT_TIMEOUT
    o = _RunOptions(f, int(reserved), int(wait_timeout_ns or 0))
    return ctypes.byref(o)


def q4gemv_run_ex(codes, scales_f16, zeros_u4_or_null, x, y, M=None, N=None, K=None, group=32,
                  flags=None, wait_timeout_ns=None, stream=None, check=True, _reserved=0) -> int:
    """q4gemv_run with per-call options: flags (Q4_RUN_*), and wait_timeout_ns, which sets
    Q4_RUN_WAIT_TIMEOUT when given."""
    M, N, K = _mnk_q4(codes, x, M, N, K)
    st = lib().q4gemv_run_ex(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                             _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _addr(x, "x", 4),
                             _addr(y, "y", 4), M, N, K, int(group), _options(flags, wait_timeout_ns, _reserved),
                             _stream(stream))
    if check:
        _check(st, "q4gemv_run_ex")
    return st


def q4gemv_fused_run_ex(codes, scales_f16, zeros_u4_or_null, x, gamma, eps, y, M=None, N=None, K=None, group=32,
                        epilogue=Q4_EPILOGUE_NONE, flags=None, wait_timeout_ns=None, stream=None, check=True) -> int:
    M, N, K = _mnk_q4(codes, x, M, N, K)
    st = lib().q4gemv_fused_run_ex(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                                   _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _addr(x, "x", 4),
                                   _addr(gamma, "gamma", 4), float(eps), _addr(y, "y", 4), M, N, K, int(group),
                                   int(epilogue), _options(flags, wait_timeout_ns), _stream(stream))
    if check:
        _check(st, "q4gemv_fused_run_ex")
    return st


def q4gemv_grouped_run_ex(segments, K, group=32, flags=None, wait_timeout_ns=None, stream=None, check=True) -> int:
    arr = (_Segment * max(1, len(segments)))()
    for i, sg in enumerate(segments):
        codes, scales, zeros, x, y = sg[:5]
        N = int(sg[5]) if len(sg) > 5 else int(codes.shape[0])
        arr[i] = _Segment(_addr(codes, "codes", 1), _addr(scales, "scales_f16", 2), _addr(zeros, "zeros_u4_or_null", 1),
                          _addr(x, "x", 4), _addr(y, "y", 4), N)
    st = lib().q4gemv_grouped_run_ex(arr, len(segments), int(K), int(group), _options(flags, wait_timeout_ns),
                                     _stream(stream))
    if check:
        _check(st, "q4gemv_grouped_run_ex")
    return st


def q4gemm_run_ex(codes, scales_f16, zeros_u4_or_null, a_bf16, c, M=None, N=None, K=None, group=32,
                  flags=None, wait_timeout_ns=None, stream=None, check=True) -> int:
    M, N, K = _mnk_q4(codes, a_bf16, M, N, K)
    st = lib().q4gemm_run_ex(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                             _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _addr(a_bf16, "a_bf16", 2),
                             _addr(c, "c", 4), M, N, K, int(group), _options(flags, wait_timeout_ns),
                             _stream(stream))
    if check:
        _check(st, "q4gemm_run_ex")
    return st


def q4_0_gemv_run(blocks, x, y, M=None, N=None, K=None, stream=None, check=True) -> int:
    M = int(x.shape[0] if M is None else M)
    K = int(x.shape[1] if K is None else K)
    N = int(blocks.shape[0] if N is None else N)
    st = lib().q4_0_gemv_run(_addr(blocks, "blocks", 1), _addr(x, "x", 4), _addr(y, "y", 4), M, N, K,
                             _stream(stream))
    if check:
        _check(st, "q4_0_gemv_run")
    return st


def q8_0_gemv_run(blocks, x, y, M=None, N=None, K=None, stream=None, check=True) -> int:
    M = int(x.shape[0] if M is None else M)
    K = int(x.shape[1] if K is None else K)
    N = int(blocks.shape[0] if N is None else N)
    st = lib().q8_0_gemv_run(_addr(blocks, "blocks", 1), _addr(x, "x", 4), _addr(y, "y", 4), M, N, K,
                             _stream(stream))
    if check:
        _check(st, "q8_0_gemv_run")
    return st


def q4gemm_run(codes, scales_f16, zeros_u4_or_null, a_bf16, c, M=None, N=None, K=None, group=32,
               stream=None, check=True) -> int:
    M, N, K = _mnk_q4(codes, a_bf16, M, N, K)
    st = lib().q4gemm_run(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                          _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _addr(a_bf16, "a_bf16", 2),
                          _addr(c, "c", 4), M, N, K, int(group), _stream(stream))
    if check:
        _check(st, "q4gemm_run")
    return st


def f32gemv_run(W, x, y, M=None, N=None, K=None, stream=None, check=True) -> int:
    M = int(x.shape[0] if M is None else M)
    N = int(W.shape[0] if N is None else N)
    K = int(W.shape[1] if K is None else K)
    st = lib().f32gemv_run(_addr(W, "W", 4), _addr(x, "x", 4), _addr(y, "y", 4), M, N, K, _stream(stream))
    if check:
        _check(st, "f32gemv_run")
    return st


def q4_dequant_f32_run(codes, scales_f16, zeros_u4_or_null, w, N=None, K=None, group=32,
                       stream=None, check=True) -> int:
    N = int(codes.shape[0] if N is None else N)
    K = int(codes.shape[1] * 2 if K is None else K)
    st = lib().q4_dequant_f32_run(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                                  _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _addr(w, "w", 4),
                                  N, K, int(group), _stream(stream))
    if check:
        _check(st, "q4_dequant_f32_run")
    return st


def q4_dequant_bf16_run(codes, scales_f16, zeros_u4_or_null, wb, N=None, K=None, group=32,
                        stream=None, check=True) -> int:
    N = int(codes.shape[0] if N is None else N)
    K = int(codes.shape[1] * 2 if K is None else K)
    st = lib().q4_dequant_bf16_run(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                                   _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _addr(wb, "wb", 2),
                                   N, K, int(group), _stream(stream))
    if check:
        _check(st, "q4_dequant_bf16_run")
    return st


def q4gemv_device_status(stream=None) -> int:
    """Synchronise the stream; Q4_OK or Q4_ERR_TIMEOUT (clears the flag)."""
    return lib().q4gemv_device_status(_stream(stream))


def q4gemm_set_wait_timeout_ns(ns: int) -> int:
    return lib().q4gemm_set_wait_timeout_ns(int(ns))


def q4gemv_bounds_violations(stream=None) -> int:
    """Out-of-range accesses counted since the last call (bounds-checking builds), -1
    in a library built without the checks."""
    return lib().q4gemv_bounds_violations(_stream(stream) if stream is not None else None)


def q4gemv_grouped_split(Ns, K, group, grid_max):
    """Host-only test export: (grid, nblocks per matrix, first CTA per matrix) of the CTA
    split a grouped launch makes; raises Q4Error on a negated status."""
    n = len(Ns)
    arr = (_i64 * max(1, n))(*[int(v) for v in Ns])
    nb = (_i32 * max(1, n))()
    cb = (_i32 * max(1, n))()
    grid = lib().q4gemv_grouped_split(arr, n, int(K), int(group), int(grid_max), nb, cb)
    if grid < 0:
        raise Q4Error(-grid, "q4gemv_grouped_split")
    return grid, list(nb[:n]), list(cb[:n])


def q4gemv_set_overlapped_launch(enable: bool) -> int:
    """Programmatic dependent launch for later q4gemv_run calls; returns the old setting."""
    return lib().q4gemv_set_overlapped_launch(1 if enable else 0)


def vec4_read_probe_run(buf, nbytes, partial, blocks=0, stream=None, check=True):
    used = _i32(0)
    st = lib().vec4_read_probe_run(_addr(buf, "buf"), int(nbytes), _addr(partial, "partial", 4), int(blocks),
                                   ctypes.byref(used), _stream(stream))
    if check:
        _check(st, "vec4_read_probe_run")
    return used.value


# ------------------------------------------------------------ mixture of experts

class _Types:
    """The torch types of the arrays (looked up once)."""
    f32 = bf16 = i32 = f16 = u8 = None

    @classmethod
    def load(cls):
        import torch
        cls.f32, cls.bf16, cls.i32 = torch.float32, torch.bfloat16, torch.int32
        cls.f16, cls.u8 = torch.float16, torch.uint8


def _dtype(t):
    """Q4_F32 or Q4_BF16 of a tensor or a torch dtype (an integer passes through)."""
    if isinstance(t, int):
        return t
    if _Types.f32 is None:
        _Types.load()
    d = getattr(t, "dtype", t)
    if d is _Types.f32:
        return Q4_F32
    if d is _Types.bf16:
        return Q4_BF16
    raise ValueError(f"float32 or bfloat16 expected, got {d}")


def _typed(t, name, dtype):
    """Address of a contiguous tensor of the given type (None passes through)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is required (got strides {tuple(t.stride())})")
    return t.data_ptr()


def _same(t, name, dtype):
    """Address of an activation array of the call's type (None passes through)."""
    return _typed(t, name, _Types.f32 if dtype == Q4_F32 else _Types.bf16)


def _ints(t, name):
    """Address of an int32 array (None passes through)."""
    return _typed(t, name, _Types.i32)


def _floats(t, name):
    """Address of a binary32 array (None passes through)."""
    return _typed(t, name, _Types.f32)


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _workspace(n, where):
    if n < 0:
        raise Q4Error(Q4_ERR_UNSUPPORTED, where)
    return n


def q4moe_route_workspace(T, E, top_k) -> int:
    """Bytes of workspace q4moe_route_run needs."""
    return _workspace(lib().q4moe_route_workspace(int(T), int(E), int(top_k)), "q4moe_route_workspace")


def q4moe_gemm_workspace(R, Tx, N, K, E, dtype) -> int:
    """Bytes of workspace q4moe_gemm_run needs (dtype: that of x)."""
    return _workspace(lib().q4moe_gemm_workspace(int(R), int(Tx), int(N), int(K), int(E), _dtype(dtype)),
                      "q4moe_gemm_workspace")


def q4moe_block_workspace(T, E, top_k, H, inner, dtype) -> int:
    """Bytes of workspace q4moe_block_run needs."""
    return _workspace(lib().q4moe_block_workspace(int(T), int(E), int(top_k), int(H), int(inner), _dtype(dtype)),
                      "q4moe_block_workspace")


def q4moe_route_run(logits, ids, weights, offsets, rows, pos, workspace, bias=None, token_mask=None,
                    score=Q4_ROUTE_SOFTMAX, renormalize=True, scale=1.0, flags=None, stream=None, check=True) -> int:
    """The top_k experts of each token (ids [T, top_k], weights), and the rows grouped by
    expert (offsets [E + 1], rows [T * top_k], pos [T, top_k]).  bias [E] enters the choice
    only: added to the logits, or, with score=Q4_ROUTE_SIGMOID | Q4_ROUTE_SCORE_BIAS (or
    SOFTMAX), to the scores, as the balancing bias of a model trained without an auxiliary
    loss is."""
    if _Types.f32 is None:
        _Types.load()
    T, E = logits.shape
    of = ids.shape
    k = of[1]
    _need(of[0] == T and weights.shape == of and pos.shape == of and rows.numel() == T * k and
          offsets.numel() == E + 1 and (bias is None or bias.numel() == E) and
          (token_mask is None or token_mask.numel() == T), "q4moe_route_run: shapes do not agree")
    st = lib().q4moe_route_run(_floats(logits, "logits"), _floats(bias, "bias"), _addr(token_mask, "token_mask", 1),
                               T, E, k, score, 1 if renormalize else 0, scale, _ints(ids, "ids"),
                               _floats(weights, "weights"), _ints(offsets, "offsets"), _ints(rows, "rows"),
                               _ints(pos, "pos"), _addr(workspace, "workspace", 1), workspace.numel(),
                               _options(flags, None), _stream(stream))
    if check:
        _check(st, "q4moe_route_run")
    return st


def q4moe_gemm_run(codes, scales_f16, zeros_u4_or_null, x, rows, offsets, y, workspace, group=32,
                   epilogue=Q4_EPILOGUE_NONE, flags=None, wait_timeout_ns=None, stream=None, check=True) -> int:
    """y[r] = W_e x[rows[r]] over stacked experts codes [E, N, K/2] (rows None: x[r])."""
    E, N, half = codes.shape
    Tx, K = x.shape
    R = y.shape[0]
    d = _dtype(x)
    _need(K == 2 * half and y.shape[1] == (N // 2 if epilogue == Q4_EPILOGUE_SWIGLU else N) and
          scales_f16.shape == (E, N, K // group) and offsets.numel() == E + 1 and
          (zeros_u4_or_null is None or zeros_u4_or_null.shape == (E, N, (K // group + 1) // 2)) and
          (rows is None or rows.numel() == R), "q4moe_gemm_run: shapes do not agree")
    st = lib().q4moe_gemm_run(_addr(codes, "codes", 1), _addr(scales_f16, "scales_f16", 2),
                              _addr(zeros_u4_or_null, "zeros_u4_or_null", 1), _same(x, "x", d), _ints(rows, "rows"),
                              _ints(offsets, "offsets"), _same(y, "y", d), E, R, Tx, N, K, group, d,
                              epilogue, _addr(workspace, "workspace", 1), workspace.numel(),
                              _options(flags, wait_timeout_ns), _stream(stream))
    if check:
        _check(st, "q4moe_gemm_run")
    return st


def _gate_stride(gate, T, H):
    if gate is None or gate.dim() == 1:
        _need(gate is None or gate.numel() == H, "gate: [H] or [T, H] expected")
        return 0
    _need(gate.shape == (T, H), "gate: [H] or [T, H] expected")
    return H


def q4_block_norm_run(y, x, out, pos=None, weights=None, post_gamma=None, gate=None, residual_scale=1.0,
                      pre_gamma=None, out_norm=None, eps=1e-6, flags=None, stream=None, check=True) -> int:
    """out = residual_scale x + gate norm(b), out_norm = norm(out): b is the weighted sum of
    the rows pos of y, or y itself (pos None)."""
    T, H = x.shape
    k = pos.shape[1] if pos is not None else 0
    d = _dtype(x)
    _need(y.shape[1] == H and out.shape == x.shape and (out_norm is None or out_norm.shape == x.shape) and
          (pos is None or (pos.shape[0] == T and weights is not None and weights.shape == pos.shape)) and
          (post_gamma is None or post_gamma.numel() == H) and (pre_gamma is None or pre_gamma.numel() == H),
          "q4_block_norm_run: shapes do not agree")
    a = _BlockNorm(T, H, k, d, y.shape[0], _same(y, "y", d), _ints(pos, "pos"), _floats(weights, "weights"),
                   _same(x, "x", d), _floats(post_gamma, "post_gamma"), _same(gate, "gate", d),
                   _gate_stride(gate, T, H), _floats(pre_gamma, "pre_gamma"), _same(out, "out", d),
                   _same(out_norm, "out_norm", d), residual_scale, eps)
    st = lib().q4_block_norm_run(ctypes.byref(a), _options(flags, None), _stream(stream))
    if check:
        _check(st, "q4_block_norm_run")
    return st


def q4moe_block_run(up, down, logits, a, x, out, out_norm, ids, route_weights, workspace, group=32,
                    score=Q4_ROUTE_SOFTMAX, renormalize=True, route_scale=1.0, bias=None, token_mask=None,
                    post_gamma=None, gate=None, residual_scale=1.0, pre_gamma=None, eps=1e-6, flags=None,
                    wait_timeout_ns=None, stream=None, check=True) -> int:
    """A mixture-of-experts block in one call: route, gate and up, down, norms and residual.
    up: (codes [E, 2 inner, H/2], scales, zeros or None); down: (codes [E, H, inner/2], ...)."""
    T, E = logits.shape
    H = x.shape[1]
    inner = 2 * down[0].shape[2]
    k = ids.shape[1]
    d = _dtype(x)
    for (codes, scales, zeros), N, K in ((up, 2 * inner, H), (down, H, inner)):
        _need(codes.shape == (E, N, K // 2) and scales.shape == (E, N, K // group) and
              (zeros is None or zeros.shape == (E, N, (K // group + 1) // 2)),
              "q4moe_block_run: shapes of the weights do not agree")
    _need(x.shape[0] == T and a.shape == x.shape and out.shape == x.shape and
          (out_norm is None or out_norm.shape == x.shape) and ids.shape == (T, k) and
          route_weights.shape == (T, k) and (bias is None or bias.numel() == E) and
          (token_mask is None or token_mask.numel() == T) and (post_gamma is None or post_gamma.numel() == H) and
          (pre_gamma is None or pre_gamma.numel() == H), "q4moe_block_run: shapes do not agree")
    g = _MoeBlock(T, E, k, H, inner, group, d, score, 1 if renormalize else 0, route_scale,
                  residual_scale, eps, _addr(up[0], "up codes", 1), _addr(up[1], "up scales", 2),
                  _addr(up[2], "up zeros", 1), _addr(down[0], "down codes", 1), _addr(down[1], "down scales", 2),
                  _addr(down[2], "down zeros", 1), _floats(logits, "logits"), _floats(bias, "bias"),
                  _addr(token_mask, "token_mask", 1), _same(a, "a", d), _same(x, "x", d),
                  _floats(post_gamma, "post_gamma"), _same(gate, "gate", d), _gate_stride(gate, T, H),
                  _floats(pre_gamma, "pre_gamma"), _ints(ids, "ids"), _floats(route_weights, "route_weights"),
                  _same(out, "out", d), _same(out_norm, "out_norm", d), _addr(workspace, "workspace", 1),
                  workspace.numel())
    st = lib().q4moe_block_run(ctypes.byref(g), _options(flags, wait_timeout_ns), _stream(stream))
    if check:
        _check(st, "q4moe_block_run")
    return st


# ------------------------------------------------- several continuations of one prompt
#
# What these calls do on the GPU may take no longer than their arguments' way there, so the
# structures are packed in one go (a ctypes structure of 30 fields takes 1.4 us, this 0.2) and
# the checks of a call are one expression, whose parts are told apart only where it fails.

_ROPE = struct.Struct("@5i2f3P3q6P2P4i4q")
_ATTN = struct.Struct("@6if P q 2P4i4q 9P q")
_REORDER = struct.Struct("@6i6q7P")


def _on(dev, t, name, dtype):
    """Address of a contiguous tensor of the given type on device `dev` (0 for None)."""
    if t is None:
        return 0
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is required (got strides {tuple(t.stride())})")
    raise ValueError(f"{name}: a tensor on CUDA device {dev} expected, got {t.device}")


def _device(t, name):
    """The CUDA device of the call's first tensor, which has to be the current one."""
    if _Types.f32 is None:
        _Types.load()
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: a CUDA tensor expected, got {t.device}")
    if dev != _current_device():
        raise ValueError(f"{name}: on CUDA device {dev}, which is not the current one")
    return dev


_raw_device = None


def _current_device():
    """The current CUDA device's index (without torch's own wrapper where that can be left out)."""
    global _raw_device
    if _raw_device is None:
        import torch
        _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _raw_device()


def _half_dtype(t, name):
    """Q4_BF16 or Q4_F16 of a tensor."""
    if t.dtype is _Types.bf16:
        return Q4_BF16
    if t.dtype is _Types.f16:
        return Q4_F16
    raise ValueError(f"{name}: bfloat16 or float16 expected, got {t.dtype}")


def _cache(dev, k, v):
    """The paged cache of two pools [pages, kv heads, tokens of a page, features]: the fields of
    q4_kv_cache_t."""
    shape, stride = k.shape, k.stride()
    dtype = k.dtype
    if not (len(shape) == 4 and v.shape == shape and v.stride() == stride and v.dtype is dtype and
            (stride[3] == 1 or shape[3] == 1) and k.get_device() == dev and v.get_device() == dev):
        raise ValueError("k_cache, v_cache: [pages, heads, tokens of a page, features] of the same shape, strides, type "
                         "and device, with features side by side, expected")
    pages, heads, page, D = shape
    return (k.data_ptr(), v.data_ptr(), Q4_BF16 if dtype is _Types.bf16 else _half_dtype(k, "k_cache"), heads, D, page,
            pages, stride[0], stride[1], stride[2])


def _heads(dev, t, name, T, H, D, dtype):
    """(address, elements from one token to the next) of [T, H, D] with the heads of a token side by side."""
    s = t.stride()
    if not (t.shape == (T, H, D) and (s[2] == 1 or D == 1) and (s[1] == D or H == 1) and t.dtype is dtype and
            t.get_device() == dev):
        raise ValueError(f"{name}: [{T}, {H}, {D}] of {dtype} on CUDA device {dev} with the heads of a token side by side "
                         f"expected, got {tuple(t.shape)} of {t.dtype} on {t.device} with strides {tuple(s)}")
    return t.data_ptr(), s[0]


def q4_rope_append_run(q, k, v, positions, inv_freq, q_out, k_cache, v_cache, slots=None, q_gamma=None, k_gamma=None,
                       eps=1e-6, layout=Q4_ROPE_HALF, scale=1.0, flags=None, stream=None, check=True) -> int:
    """Norm and rotary positions of q [T, Hq, D] into q_out, and of k [T, Hkv, D] into the
    cache, with v, at slots [T] (None: token t at slot t; no two the same, or -1).  The heads of a token lie side by
    side; tokens may be any stride apart, so q, k and v may be parts of one product's rows.
    k and v None: queries only (k_cache, v_cache None too).  inv_freq [rot / 2] float32:
    2 len(inv_freq) features are rotated."""
    dev = _device(q, "q")
    T, Hq, D = q.shape
    dtype, t16 = q.dtype, q_out.dtype
    f32, i32 = _Types.f32, _Types.i32
    d = Q4_F32 if dtype is f32 else _dtype(q)
    qa, qs = _heads(dev, q, "q", T, Hq, D, dtype)
    if k is not None:
        _need(v is not None and k_cache is not None and v_cache is not None,
              "q4_rope_append_run: k, v and the caches come together")
        cache = _cache(dev, k_cache, v_cache)
        _need(cache[4] == D and t16 is k_cache.dtype, "q4_rope_append_run: shapes or types do not agree")
        ka, ks = _heads(dev, k, "k", T, cache[3], D, dtype)
        va, vs = _heads(dev, v, "v", T, cache[3], D, dtype)
    else:
        _need(v is None and k_cache is None and v_cache is None, "q4_rope_append_run: k, v and the caches come together")
        cache = (0, 0, _half_dtype(q_out, "q_out"), 1, D, 1, 0, 0, 0, 0)
        ka = va = ks = vs = 0
    _need(q_out.shape == (T, Hq, D) and (positions is None or positions.numel() == T) and
          (slots is None or slots.numel() == T) and (q_gamma is None or q_gamma.numel() == D) and
          (k_gamma is None or k_gamma.numel() == D), "q4_rope_append_run: shapes do not agree")
    a = _ROPE.pack(T, Hq, d, 2 * inv_freq.numel() if inv_freq is not None else 0, layout, scale, eps, qa, ka, va, qs, ks,
                   vs, _on(dev, q_gamma, "q_gamma", f32), _on(dev, k_gamma, "k_gamma", f32),
                   _on(dev, positions, "positions", i32), _on(dev, inv_freq, "inv_freq", f32),
                   _on(dev, slots, "slots", i32), _on(dev, q_out, "q_out", t16), *cache)
    st = lib().q4_rope_append_run(a, _options(flags, None), _stream(stream))
    if check:
        _check(st, "q4_rope_append_run")
    return st


def q4_rope_frequencies(rot, base=10000.0, kind=Q4_ROPE_PLAIN, factor=1.0, trained=0.0, low=1.0, high=4.0):
    """Inverse frequencies [rot / 2] (a float32 tensor on the CPU) of rot rotated features,
    stretched by `factor` for contexts longer than the `trained` tokens."""
    import torch
    out = torch.empty(max(0, int(rot)) // 2, dtype=torch.float32)
    at = ctypes.cast(out.data_ptr() if out.numel() else (ctypes.c_float * 1)(), ctypes.POINTER(ctypes.c_float))
    _check(lib().q4_rope_frequencies(at, int(rot), float(base), int(kind), float(factor), float(trained), float(low),
                                     float(high)), "q4_rope_frequencies")
    return out


def q4_prefix_attn_workspace(S, groups, Hq, Hkv, D) -> int:
    """Bytes of workspace q4_prefix_attn_run needs on the current device."""
    return _workspace(lib().q4_prefix_attn_workspace(int(S), int(groups), int(Hq), int(Hkv), int(D)),
                      "q4_prefix_attn_workspace")


def q4_prefix_attn_run(q, k_cache, v_cache, out, workspace, group_offsets=None, shared_pages=None, shared_lens=None,
                       limits=None, own_pages=None, own_lens=None, scale=None, lse=None, flags=None,
                       wait_timeout_ns=None, stream=None, check=True) -> int:
    """Attention of q [S, Hq, D] over the segment a group of queries shares (shared_lens
    [groups], shared_pages [groups, pages], queries group_offsets[g] to group_offsets[g + 1];
    limits [S]: how much of it each query sees), then each query's own (own_lens [S],
    own_pages [S, pages]).  scale None: 1 / sqrt(D).  out [S, Hq, D], lse [S, Hq] float32."""
    dev = _device(q, "q")
    S, Hq, D = q.shape
    t16, i32 = k_cache.dtype, _Types.i32
    cache = _cache(dev, k_cache, v_cache)
    groups = most_shared = most_own = 0
    if shared_lens is not None or shared_pages is not None:
        _need(shared_lens is not None and shared_pages is not None, "q4_prefix_attn_run: shared_lens and shared_pages come together")
        groups = shared_lens.numel()
        rows, most_shared = shared_pages.shape
        _need(rows == groups and (group_offsets is None or group_offsets.numel() == groups + 1),
              "q4_prefix_attn_run: shapes do not agree")
    if own_lens is not None or own_pages is not None:
        _need(own_lens is not None and own_pages is not None, "q4_prefix_attn_run: own_lens and own_pages come together")
        rows, most_own = own_pages.shape
        _need(rows == S and own_lens.numel() == S, "q4_prefix_attn_run: shapes do not agree")
    _need(cache[4] == D and out.shape == (S, Hq, D) and (limits is None or limits.numel() == S) and
          (lse is None or lse.shape == (S, Hq)), "q4_prefix_attn_run: shapes do not agree")
    qa, qs = _heads(dev, q, "q", S, Hq, D, t16)
    o = out.dtype
    out_dtype = cache[2] if o is t16 else Q4_F32 if o is _Types.f32 else _half_dtype(out, "out")
    a = _ATTN.pack(S, Hq, groups, out_dtype, most_shared, most_own, D ** -0.5 if scale is None else scale, qa, qs, *cache,
                   _on(dev, group_offsets, "group_offsets", i32), _on(dev, shared_pages, "shared_pages", i32),
                   _on(dev, shared_lens, "shared_lens", i32), _on(dev, limits, "limits", i32),
                   _on(dev, own_pages, "own_pages", i32), _on(dev, own_lens, "own_lens", i32), _on(dev, out, "out", o),
                   _on(dev, lse, "lse", _Types.f32), _on(dev, workspace, "workspace", _Types.u8), workspace.numel())
    st = lib().q4_prefix_attn_run(a, _options(flags, wait_timeout_ns), _stream(stream))
    if check:
        _check(st, "q4_prefix_attn_run")
    return st


def q4_beam_step_workspace(groups, W, K, V) -> int:
    """Bytes of workspace q4_beam_step_run needs on the current device."""
    return _workspace(lib().q4_beam_step_workspace(int(groups), int(W), int(K), int(V)), "q4_beam_step_workspace")


def q4_beam_step_run(logits, scores, tokens, parents, out_scores, workspace, finished=None, out_finished=None, eos=-1,
                     flags=None, stream=None, check=True) -> int:
    """The K best continuations of each group: tokens, parents, out_scores (and out_finished,
    uint8) [groups, K] from logits [groups * W, V] (rows may be any stride apart) and the
    beams' scores (and finished, uint8) [groups, W].  The order within a beam is that of its
    logits, then tokens; between beams that of the scores, then beams."""
    dev = _device(logits, "logits")
    rows, V = logits.shape
    groups, W = scores.shape
    of = tokens.shape
    stride = logits.stride()
    _need(rows == groups * W and len(of) == 2 and of[0] == groups and parents.shape == of and out_scores.shape == of and (finished is None or finished.shape == scores.shape) and
          (out_finished is None or out_finished.shape == of) and logits.dtype is _Types.f32 and stride[1] == 1,
          "q4_beam_step_run: shapes or types do not agree")
    i32, f32, u8 = _Types.i32, _Types.f32, _Types.u8
    st = lib().q4_beam_step_run(logits.data_ptr(), stride[0], _on(dev, scores, "scores", f32),
                                _on(dev, finished, "finished", u8), groups, W, of[1], V, eos,
                                _on(dev, tokens, "tokens", i32), _on(dev, parents, "parents", i32),
                                _on(dev, out_scores, "out_scores", f32), _on(dev, out_finished, "out_finished", u8),
                                _on(dev, workspace, "workspace", u8), workspace.numel(), _options(flags, None),
                                _stream(stream))
    if check:
        _check(st, "q4_beam_step_run")
    return st


def q4_beam_reorder_run(tables, lens, parents, spare, out_tables, out_spare, pool, flags=None, stream=None,
                        check=True) -> int:
    """Page tables [groups * W, pages] and the unfinished pages of every plane of pool
    [planes, pages, heads, tokens of a page, features] follow parents [groups, W]; lens
    [groups], spare [groups * W]."""
    dev = _device(pool, "pool")
    groups, W = parents.shape
    planes, pages, heads, page, D = pool.shape
    n, most = tables.shape
    stride = pool.stride()
    _need(n == groups * W and lens.numel() == groups and spare.numel() == n and out_spare.numel() == n and
          out_tables.shape == tables.shape and stride[4] == 1, "q4_beam_reorder_run: shapes do not agree")
    i32, e = _Types.i32, pool.element_size()
    a = _REORDER.pack(groups, W, most, planes, heads, page, pages, D * e, stride[0] * e, stride[1] * e, stride[2] * e,
                      stride[3] * e, pool.data_ptr(), _on(dev, tables, "tables", i32), _on(dev, lens, "lens", i32),
                      _on(dev, parents, "parents", i32), _on(dev, spare, "spare", i32),
                      _on(dev, out_tables, "out_tables", i32), _on(dev, out_spare, "out_spare", i32))
    st = lib().q4_beam_reorder_run(a, _options(flags, None), _stream(stream))
    if check:
        _check(st, "q4_beam_reorder_run")
    return st
