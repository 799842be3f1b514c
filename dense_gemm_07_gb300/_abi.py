"""ctypes declarations of libgemm07.so -- one Python name per C entry point.

Argument marshalling only: every function here forwards its integers and
addresses to the C symbol of the same name and returns its result.  The
library is loaded on first use; if it has not been built, or cannot be
loaded, the call raises (there is no fallback of any kind).
"""
from __future__ import annotations

import ctypes
import threading

from . import _build

_lib = None
_lock = threading.Lock()

GEMM_OK = 0
GEMM_ERR_INVALID_ARG = 1
GEMM_ERR_MISALIGNED = 2          # reserved, never returned
GEMM_ERR_UNSUPPORTED_DEVICE = 3
GEMM_ERR_LAUNCH = 4
GEMM_ERR_TIMEOUT = 5
GEMM_ERR_INTERNAL = 6
GEMM_ERR_NO_MEMORY = 7
GEMM_ERR_SCRATCH_TOO_SMALL = 8
NOALLOC_SCRATCH_BYTES = 64 << 20

PATHS = {0: "none", 1: "zero_fill", 2: "f32_simt", 3: "bf16_tma",
         4: "bf16_packed", 5: "bf16_skinny", 6: "bf16_gemv", 7: "bf16_small",
         8: "bf16_narrow"}


class GemmPlan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("split_k", ctypes.c_int32),
                ("tiles", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("pack_a", ctypes.c_int32), ("pack_b", ctypes.c_int32),
                ("dp_tiles", ctypes.c_int64), ("sk_tiles", ctypes.c_int64),
                ("sk_pairs", ctypes.c_int32), ("pairs", ctypes.c_int32)]


class GemmEpilogue(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("bias", ctypes.c_void_p), ("activation", ctypes.c_int32)]


class GemmW4(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("ld_scales", ctypes.c_int64), ("zeros", ctypes.c_void_p),
                ("ld_zeros", ctypes.c_int64), ("group", ctypes.c_int32)]


class GemmFp8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("scales", ctypes.c_void_p), ("ld_scales", ctypes.c_int64),
                ("square", ctypes.c_int32)]


class GemmFp8QuantizeArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("C", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_type", ctypes.c_int32),
                ("square", ctypes.c_int32), ("transpose", ctypes.c_int32),
                ("index", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("batch", ctypes.c_int64), ("x_step", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("ld", ctypes.c_int64),
                ("codes_step", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("ld_scales", ctypes.c_int64), ("scales_step", ctypes.c_int64)]


class GemmRouteArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("k", ctypes.c_int64),
                ("logits", ctypes.c_void_p), ("ld", ctypes.c_int64), ("type", ctypes.c_int32),
                ("score", ctypes.c_int32), ("bias", ctypes.c_void_p),
                ("groups", ctypes.c_int32), ("groups_kept", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class GemmCombineArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int64), ("k", ctypes.c_int64),
                ("R", ctypes.c_int64), ("rows", ctypes.c_void_p), ("ld_rows", ctypes.c_int64),
                ("rows_type", ctypes.c_int32), ("slot", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
                ("x_type", ctypes.c_int32)]


class GemmNormGateArgs(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_type", ctypes.c_int32),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("y_type", ctypes.c_int32),
                ("w_post", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("ld_gate", ctypes.c_int64), ("gate_mode", ctypes.c_int32),
                ("w_pre", ctypes.c_void_p), ("alpha", ctypes.c_float), ("eps", ctypes.c_float)]


class GemmNormGateGrads(ctypes.Structure):
    _fields_ = [("d_x_out", ctypes.c_void_p), ("ld_d_x_out", ctypes.c_int64),
                ("dh", ctypes.c_void_p), ("ld_dh", ctypes.c_int64), ("dh_type", ctypes.c_int32),
                ("dx", ctypes.c_void_p), ("ld_dx", ctypes.c_int64),
                ("dy", ctypes.c_void_p), ("ld_dy", ctypes.c_int64),
                ("dgate", ctypes.c_void_p), ("dw_post", ctypes.c_void_p),
                ("dw_pre", ctypes.c_void_p)]


TYPE_F32 = 0
TYPE_BF16 = 1
GATE_NONE = 0
GATE_CHANNEL = 1
GATE_ROW = 2
GATE_FULL = 3
NORM_MAX_WIDTH = 16384
ACT_NONE = 0
ACT_RELU = 1
ACT_GELU = 2


# (name, restype, argtypes)
_i64, _vp, _i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
_GEMM_ARGS = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
SIGNATURES = [
    ("gemm_f32", _i32, _GEMM_ARGS),
    ("gemm_bf16_f32acc", _i32, _GEMM_ARGS),
    ("gemm_bf16_f32acc_noalloc", _i32, _GEMM_ARGS),
    ("gemm_f32_ex", _i32, _GEMM_ARGS[:-1] + [ctypes.POINTER(GemmEpilogue), _vp]),
    ("gemm_bf16_f32acc_ex", _i32, _GEMM_ARGS[:-1] + [ctypes.POINTER(GemmEpilogue), _vp]),
    ("gemm_f32_host", _i32, _GEMM_ARGS),
    ("gemm_f32_ladder", _i32, [_i32] + _GEMM_ARGS),
    ("gemm_bf16_f32acc_host", _i32, _GEMM_ARGS),
    ("gemm_status_string", ctypes.c_char_p, [_i32]),
    ("gemm_get_device_status", _i32, [_vp]),
    ("gemm_shutdown", None, []),
    ("gemm_abi_version", _i32, []),
    ("gemm_launch_count", ctypes.c_uint64, []),
    ("gemm_debug_inject", _i32, [_i32, ctypes.c_uint64]),
    ("gemm_tile_order", _i32, [_i64, _i64, _i64, _i64,
                               ctypes.POINTER(_i64), ctypes.POINTER(_i64)]),
    ("gemm_plan_bf16", _i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                              ctypes.POINTER(GemmPlan)]),
    ("gemm_plan_f32", _i32, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                             ctypes.POINTER(GemmPlan)]),
    ("gemm_pair_units", _i64, [_i64, _i64, _i64, _i32, _i32, _i32, _vp, _i64]),
    ("gemm_set_bf16_schedule", _i32, [_i32]),
    ("gemm_set_bf16_small_limit", _i64, [_i64]),
    ("gemm_w4_packed_bytes", _i64, [_i64, _i64]),
    ("gemm_w4", _i32, [_i64, _i64, _i64, _vp, _i64, ctypes.POINTER(GemmW4), _vp, _i64,
                       ctypes.c_int32, ctypes.POINTER(GemmEpilogue), _vp]),
    ("gemm_w4_pack", _i32, [_i64, _i64, _vp, _i64, _vp, _vp]),
    ("gemm_w4_quantize", _i32, [_i64, _i64, ctypes.c_int32, _vp, _i64, ctypes.c_int32, _vp,
                                _vp, _i64, _vp, _i64, _vp]),
    ("gemm_w4_unpack", _i32, [_i64, _i64, ctypes.POINTER(GemmW4), _vp, _i64, _vp]),
    ("gemm_norm_gate", _i32, [ctypes.POINTER(GemmNormGateArgs), _vp, _i64, _vp, _i64, _vp]),
    ("gemm_norm_gate_bwd", _i32, [ctypes.POINTER(GemmNormGateArgs),
                                  ctypes.POINTER(GemmNormGateGrads), _vp]),
    ("gemm_ckpt8_bytes", _i64, [_i64, _i64]),
    ("gemm_ckpt8_pack", _i32, [_i64, _i64, _vp, _i64, ctypes.c_int32, _vp, _vp,
                               ctypes.c_int32, _vp, _i64, _vp]),
    ("gemm_ckpt8_unpack", _i32, [_i64, _i64, _vp, _vp, _vp, _i64, ctypes.c_int32, _vp]),
    ("gemm_ckpt8_act_grad", _i32, [_i64, _i64, _vp, _i64, ctypes.c_int32, _vp, _vp,
                                   ctypes.c_int32, _vp, _i64, _vp, _vp]),
    ("gemm_ckpt8_wgrad", _i32, [_i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64,
                                ctypes.c_float, _vp]),
    ("gemm_ckpt8_wgrad_units", _i64, [_i64, _i64, _i64, _i32, _i32, _vp, _i64]),
    ("gemm_fp8_quantize", _i32, [ctypes.POINTER(GemmFp8QuantizeArgs), _vp]),
    ("gemm_fp8", _i32, [_i64, _i64, _i64, ctypes.POINTER(GemmFp8), ctypes.POINTER(GemmFp8), _vp,
                        _i64, _i32, ctypes.POINTER(GemmEpilogue), _vp]),
    ("gemm_fp8_experts", _i32, [_i64, _i64, _i64, _i64, ctypes.POINTER(GemmFp8),
                                ctypes.POINTER(GemmFp8), _vp, _vp, _i64, _i32,
                                ctypes.POINTER(GemmEpilogue), _vp]),
    ("gemm_route_workspace_bytes", _i64, [_i64, _i64]),
    ("gemm_route", _i32, [ctypes.POINTER(GemmRouteArgs), _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    ("gemm_route_bwd", _i32, [ctypes.POINTER(GemmRouteArgs), _vp, _vp, _vp, _i64, _vp]),
    ("gemm_combine", _i32, [ctypes.POINTER(GemmCombineArgs), _vp, _i64, _i32, _vp]),
    ("gemm_combine_bwd", _i32, [ctypes.POINTER(GemmCombineArgs), _vp, _i64, _i32, _vp, _i64, _vp,
                                _vp]),
]


def lib(build_if_missing: bool = True) -> ctypes.CDLL:
    """The loaded library (built first if needed and allowed)."""
    global _lib
    with _lock:
        if _lib is None:
            if build_if_missing:
                path = _build.build_library()
            else:
                path = _build.LIB_PATH
            try:
                handle = ctypes.CDLL(path)
            except OSError as exc:
                raise RuntimeError(f"libgemm07.so could not be loaded from "
                                   f"{path}: {exc}") from exc
            for name, res, args in SIGNATURES:
                fn = getattr(handle, name)
                fn.restype = res
                fn.argtypes = args
            _lib = handle
    return _lib


def library_path() -> str:
    return _build.LIB_PATH


def gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream):
    return lib().gemm_f32(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_bf16_f32acc(M, N, K, A, lda, B, ldb, C, ldc, stream):
    return lib().gemm_bf16_f32acc(M, N, K, A, lda, B, ldb, C, ldc, stream)


def _epi(epilogue):
    return None if epilogue is None else ctypes.byref(epilogue)


def gemm_f32_ex(M, N, K, A, lda, B, ldb, C, ldc, epilogue, stream):
    """gemm_f32 with a fused epilogue (GemmEpilogue or None)."""
    return lib().gemm_f32_ex(M, N, K, A, lda, B, ldb, C, ldc, _epi(epilogue), stream)


def gemm_bf16_f32acc_ex(M, N, K, A, lda, B, ldb, C, ldc, epilogue, stream):
    """gemm_bf16_f32acc with a fused epilogue (GemmEpilogue or None)."""
    return lib().gemm_bf16_f32acc_ex(M, N, K, A, lda, B, ldb, C, ldc, _epi(epilogue),
                                     stream)


def gemm_bf16_f32acc_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream):
    """gemm_bf16_f32acc without any device allocation (fixed scratch)."""
    return lib().gemm_bf16_f32acc_noalloc(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_ladder(rung, M, N, K, A, lda, B, ldb, C, ldc, stream):
    """Teaching rung 0 (naive), 1 (smem-tiled) or 2 (1-D register tiles)."""
    return lib().gemm_f32_ladder(rung, M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_f32_host(M, N, K, A, lda, B, ldb, C, ldc, stream):
    return lib().gemm_f32_host(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_bf16_f32acc_host(M, N, K, A, lda, B, ldb, C, ldc, stream):
    return lib().gemm_bf16_f32acc_host(M, N, K, A, lda, B, ldb, C, ldc, stream)


def gemm_status_string(status: int) -> str:
    return lib().gemm_status_string(status).decode()


def gemm_get_device_status(stream) -> int:
    return lib().gemm_get_device_status(stream)


def gemm_shutdown() -> None:
    lib().gemm_shutdown()


def gemm_abi_version() -> int:
    return lib().gemm_abi_version()


def gemm_debug_inject(mode: int, wait_ns: int) -> int:
    """Test hook: bounded-wait limit and fault mode (see include/gemm07.h)."""
    return lib().gemm_debug_inject(mode, wait_ns)


def gemm_launch_count() -> int:
    return int(lib().gemm_launch_count())


def gemm_tile_order(tiles_m, tiles_n, group, linear):
    tm, tn = _i64(), _i64()
    s = lib().gemm_tile_order(tiles_m, tiles_n, group, linear,
                              ctypes.byref(tm), ctypes.byref(tn))
    return s, tm.value, tn.value


def _plan(fn, M, N, K, A, lda, B, ldb, C, ldc):
    p = GemmPlan()
    s = fn(M, N, K, A, lda, B, ldb, C, ldc, ctypes.byref(p))
    return s, p


def gemm_plan_bf16(M, N, K, A, lda, B, ldb, C, ldc):
    return _plan(lib().gemm_plan_bf16, M, N, K, A, lda, B, ldb, C, ldc)


def gemm_plan_f32(M, N, K, A, lda, B, ldb, C, ldc):
    return _plan(lib().gemm_plan_f32, M, N, K, A, lda, B, ldb, C, ldc)


SCHEDULE_AUTO = 0
SCHEDULE_STREAM_K = 1
SCHEDULE_COLUMN_SPLIT = 2


def gemm_set_bf16_schedule(schedule: int) -> int:
    return lib().gemm_set_bf16_schedule(schedule)


def gemm_set_bf16_small_limit(max_macs: int) -> int:
    """Largest M*N*K (M >= 2) sent to the CUDA-core small-problem path;
    0 sends every BF16 call to the tensor-core kernels.  Returns the
    previous limit."""
    return lib().gemm_set_bf16_small_limit(max_macs)


def gemm_pair_units(M, N, K, max_pairs, pair, schedule=SCHEDULE_AUTO):
    """The BF16 paired-SM kernel's work units for one pair, in order, as a
    list of (tile, k0, k1, slot, first_pair, segments, stream_k, n_off,
    width) tuples; raises on bad arguments."""
    return _units("gemm_pair_units", M, N, K, max_pairs, schedule, pair)


def gemm_ckpt8_wgrad_units(T, K, N, max_pairs, pair):
    """The weight gradient's work units for one pair, as gemm_pair_units lists
    them (slices of 128 rows of T)."""
    return _units("gemm_ckpt8_wgrad_units", T, K, N, max_pairs, pair)


def _units(name, *args):
    fn = getattr(lib(), name)
    n = fn(*args, None, 0)
    if n < 0:
        raise ValueError(f"{name}: argument out of range")
    buf = (ctypes.c_int64 * (9 * max(n, 1)))()
    n2 = fn(*args, buf, n)
    assert n2 == n
    return [tuple(buf[9 * i:9 * i + 9]) for i in range(n)]


def gemm_w4_packed_bytes(K, N):
    return lib().gemm_w4_packed_bytes(K, N)


def gemm_w4(M, N, K, A, lda, w, C, ldc, c_type, epilogue, stream):
    """w: a GemmW4; epilogue: a GemmEpilogue or None."""
    return lib().gemm_w4(M, N, K, A, lda, _epi(w), C, ldc, c_type, _epi(epilogue), stream)


def gemm_w4_pack(K, N, codes, ld, packed, stream):
    return lib().gemm_w4_pack(K, N, codes, ld, packed, stream)


def gemm_w4_quantize(K, N, group, B, ldb, b_type, packed, scales, ld_scales, zeros, ld_zeros,
                     stream):
    return lib().gemm_w4_quantize(K, N, group, B, ldb, b_type, packed, scales, ld_scales,
                                  zeros, ld_zeros, stream)


def gemm_w4_unpack(K, N, w, B, ldb, stream):
    return lib().gemm_w4_unpack(K, N, _epi(w), B, ldb, stream)


def gemm_norm_gate(args, x_out, ld_x_out, h, ldh, stream):
    """args: a GemmNormGateArgs."""
    return lib().gemm_norm_gate(_epi(args), x_out, ld_x_out, h, ldh, stream)


def gemm_norm_gate_bwd(args, grads, stream):
    """args: a GemmNormGateArgs; grads: a GemmNormGateGrads."""
    return lib().gemm_norm_gate_bwd(_epi(args), _epi(grads), stream)


def gemm_ckpt8_bytes(T, N):
    return lib().gemm_ckpt8_bytes(T, N)


def gemm_ckpt8_pack(T, N, X, ldx, x_type, q, scales, activation, act_out, ld_act, stream):
    return lib().gemm_ckpt8_pack(T, N, X, ldx, x_type, q, scales, activation, act_out, ld_act,
                                 stream)


def gemm_ckpt8_unpack(T, N, q, scales, out, ld, out_type, stream):
    return lib().gemm_ckpt8_unpack(T, N, q, scales, out, ld, out_type, stream)


def gemm_ckpt8_act_grad(T, N, G, ldg, g_type, q, scales, activation, dZ, ld_dz, dbias, stream):
    return lib().gemm_ckpt8_act_grad(T, N, G, ldg, g_type, q, scales, activation, dZ, ld_dz,
                                     dbias, stream)


def gemm_ckpt8_wgrad(T, K, N, q, scales, dY, ld_dy, dW, ldw, beta, stream):
    return lib().gemm_ckpt8_wgrad(T, K, N, q, scales, dY, ld_dy, dW, ldw, beta, stream)


def gemm_fp8_quantize(args, stream):
    """args: a GemmFp8QuantizeArgs."""
    return lib().gemm_fp8_quantize(_epi(args), stream)


def gemm_fp8(M, N, K, A, B, C, ldc, c_type, epilogue, stream):
    """A, B: GemmFp8; epilogue: a GemmEpilogue or None."""
    return lib().gemm_fp8(M, N, K, _epi(A), _epi(B), C, ldc, c_type, _epi(epilogue), stream)


def gemm_fp8_experts(E, M, N, K, A, B, offsets, C, ldc, c_type, epilogue, stream):
    return lib().gemm_fp8_experts(E, M, N, K, _epi(A), _epi(B), offsets, C, ldc, c_type,
                                  _epi(epilogue), stream)


def gemm_route_workspace_bytes(T, E):
    return lib().gemm_route_workspace_bytes(T, E)


def gemm_route(args, index, weight, slot, source, offsets, workspace, stream):
    """args: a GemmRouteArgs."""
    return lib().gemm_route(_epi(args), index, weight, slot, source, offsets, workspace, stream)


def gemm_route_bwd(args, index, d_weight, d_logits, ld_d, stream):
    """args: a GemmRouteArgs."""
    return lib().gemm_route_bwd(_epi(args), index, d_weight, d_logits, ld_d, stream)


def gemm_combine(args, out, ld_out, out_type, stream):
    """args: a GemmCombineArgs."""
    return lib().gemm_combine(_epi(args), out, ld_out, out_type, stream)


def gemm_combine_bwd(args, d_out, ld_d_out, d_out_type, d_rows, ld_d_rows, d_weight, stream):
    """args: a GemmCombineArgs."""
    return lib().gemm_combine_bwd(_epi(args), d_out, ld_d_out, d_out_type, d_rows, ld_d_rows,
                                  d_weight, stream)
