"""The operators of a transformer layer around the GEMM: 4-bit weights, norms
with gate and residual, 8-bit activation checkpoints.

Every function marshals CUDA tensors into the C entry point of its name
(declared in ``include/gemm07.h``), on ``stream`` (default: the current
stream).  Matrices have contiguous rows and any row stride; a refused argument
raises ValueError or TypeError, a status of the library GemmError.
"""
from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from . import _abi as abi
from ._errors import GemmError

_TYPES = {torch.float32: abi.TYPE_F32, torch.bfloat16: abi.TYPE_BF16}
_ACTS = {"none": abi.ACT_NONE, "relu": abi.ACT_RELU, "gelu": abi.ACT_GELU}
_FLOATS = (torch.float32, torch.bfloat16)
_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)


def _matrix(t, name, dtypes, device, shape=None):
    """Row stride of a 2-D tensor, after its checks."""
    size = t.shape
    if len(size) != 2:
        raise ValueError(f"{name} must be 2-D")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    rows, cols = size
    if shape is not None and size != shape:
        raise ValueError(f"{name} must be {shape[0]} x {shape[1]}, not {rows} x {cols}")
    r, c = t.stride()
    if c == 1 and r >= cols > 0:
        return r
    if cols > 1 and c != 1:
        raise ValueError(f"{name}: rows must be contiguous (stride(1) == 1)")
    if rows > 1 and cols > 0 and r < cols:
        raise ValueError(f"{name}: rows must not overlap (stride(0) >= columns)")
    return max(r if rows > 1 else cols, cols, 1)


def _vector(t, name, dtype, device, n):
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype or t.device != device \
            or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n} elements "
                         f"on {device}")


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _bytes16(t, name, numel, device):
    if t.dtype != torch.uint8 or t.device != device or not t.is_contiguous() \
            or t.numel() != numel:
        raise ValueError(f"{name} must be {numel} contiguous uint8 elements on {device}")
    if t.data_ptr() % 16:
        raise ValueError(f"{name} must start on a 16-byte boundary")


def _act(activation):
    act = _ACTS.get(activation)
    if act is None:
        raise ValueError(f"activation must be one of {sorted(_ACTS)}")
    return act


def _ptr(t):
    """Address of a tensor's elements (0 when it has none), None for no tensor."""
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=None)
def _entry(name):
    return getattr(abi.lib(), name)


# The handle of a device's current stream, without a Stream object around it
# (0.1 us where torch.cuda.current_stream takes 2 us).
_current_stream = torch._C._cuda_getCurrentRawStream


def _run(name, device, stream, *args):
    """Calls a C entry point with the device current and the stream last."""
    index = device.index
    handle = _current_stream(index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == index:
        s = _entry(name)(*args, handle)
    else:
        with torch.cuda.device(device):
            s = _entry(name)(*args, handle)
    if s:
        raise GemmError(s, name)


def _output(out, name, shape, dtype, device):
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
        return out, max(shape[1], 1)
    return out, _matrix(out, name, (dtype,), device, shape)


# ---------------------------------------------------------- 4-bit weights

@functools.lru_cache(maxsize=None)
def _packed_bytes(K, N):
    n = abi.gemm_w4_packed_bytes(K, N)
    if n < 0:
        raise ValueError(f"no packed matrix of {K} x {N}")
    return n


def _w4(packed, scales, zeros, group, K, device):
    """(N, GemmW4) of the weight tensors, after their checks."""
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    G, N = -(-K // group), scales.shape[-1]
    ld = _matrix(scales, "scales", _BF16, device, (G, N))
    ldz = N
    if zeros is not None:
        ldz = _matrix(zeros, "zeros", (torch.uint8,), device, (G, N))
    _bytes16(packed, "packed", _packed_bytes(K, N), device)
    return N, abi.GemmW4(_ptr(packed), _ptr(scales), ld, _ptr(zeros), max(ldz, 1), group)


def gemm_w4(A, packed, scales, zeros=None, group=128, out=None, alpha=1.0, beta=0.0,
            bias=None, activation="none", out_dtype=None, stream=None):
    """C = act(alpha * A @ W + beta * C + bias) for a bfloat16 A of a few rows and
    4-bit weights W[k, n] = (q[k, n] - z[k // group, n]) * scales[k // group, n].

    packed: from w4_pack or w4_quantize; scales: bfloat16, ceil(K / group) x N;
    zeros: uint8 of the same shape, or None (z = 8).  C is float32 (out_dtype)
    or bfloat16."""
    device = _cuda(A, "A")
    lda = _matrix(A, "A", _BF16, device)
    M, K = A.shape
    N, w = _w4(packed, scales, zeros, group, K, device)
    if beta != 0.0 and out is None:
        raise ValueError("beta != 0 reads C: pass its prior contents as `out`")
    if out_dtype is None:
        out_dtype = torch.float32 if out is None else out.dtype
    if out_dtype not in _TYPES:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    out, ldc = _output(out, "out", (M, N), out_dtype, device)
    if bias is not None:
        _vector(bias, "bias", torch.float32, device, N)
    epi = abi.GemmEpilogue(alpha, beta, _ptr(bias), _act(activation))
    _run("gemm_w4", device, stream, M, N, K, _ptr(A), lda, w, _ptr(out), ldc,
         _TYPES[out_dtype], epi)
    return out


def w4_pack(codes, stream=None):
    """4-bit codes (uint8, K x N, the low four bits of each) in the packed order
    that gemm_w4 reads."""
    device = _cuda(codes, "codes")
    ld = _matrix(codes, "codes", (torch.uint8,), device)
    K, N = codes.shape
    packed = torch.empty(_packed_bytes(K, N), dtype=torch.uint8, device=device)
    _run("gemm_w4_pack", device, stream, K, N, _ptr(codes), ld, _ptr(packed))
    return packed


def w4_quantize(B, group=128, symmetric=True, stream=None):
    """(packed, scales, zeros) of a float32 or bfloat16 matrix B (K x N), rounded to
    the nearest 4-bit codes; zeros is None when symmetric."""
    device = _cuda(B, "B")
    ldb = _matrix(B, "B", _FLOATS, device)
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    K, N = B.shape
    G = -(-K // group)
    packed = torch.empty(_packed_bytes(K, N), dtype=torch.uint8, device=device)
    scales = torch.empty((G, N), dtype=torch.bfloat16, device=device)
    zeros = None if symmetric else torch.empty((G, N), dtype=torch.uint8, device=device)
    ld = max(N, 1)
    _run("gemm_w4_quantize", device, stream, K, N, group, _ptr(B), ldb, _TYPES[B.dtype],
         _ptr(packed), _ptr(scales), ld, _ptr(zeros), ld)
    return packed, scales, zeros


def w4_unpack(packed, scales, zeros=None, group=128, K=None, stream=None):
    """The K x N bfloat16 matrix that the 4-bit weights stand for (for prompts:
    gemm_bf16_f32acc).  K defaults to all rows of the groups."""
    device = _cuda(packed, "packed")
    if scales.dim() != 2:
        raise ValueError("scales must be 2-D")
    K = scales.shape[0] * group if K is None else K
    N, w = _w4(packed, scales, zeros, group, K, device)
    out = torch.empty((K, N), dtype=torch.bfloat16, device=device)
    _run("gemm_w4_unpack", device, stream, K, N, w, _ptr(out), max(N, 1))
    return out


# ------------------------------------------------- norms, gate, residual

def _norm_args(x, y, weight_post, gate, weight_pre, residual_scale, eps):
    device = _cuda(x, "x")
    ldx = _matrix(x, "x", _FLOATS, device)
    T, D = x.shape
    if not 1 <= D <= abi.NORM_MAX_WIDTH:
        raise ValueError(f"rows must have 1 to {abi.NORM_MAX_WIDTH} elements")
    ldy, y_type = D, abi.TYPE_F32
    if y is not None:
        ldy, y_type = _matrix(y, "y", _FLOATS, device, (T, D)), _TYPES[y.dtype]
    elif weight_post is not None or gate is not None:
        raise ValueError("weight_post and gate need y")
    if weight_post is not None:
        _vector(weight_post, "weight_post", torch.float32, device, D)
    if weight_pre is not None:
        _vector(weight_pre, "weight_pre", torch.float32, device, D)
    mode, ld_gate = abi.GATE_NONE, D
    if gate is not None:
        if gate.shape == (T, D):
            mode = abi.GATE_FULL
        elif gate.shape == (T, 1):
            mode = abi.GATE_ROW
        elif gate.shape == (D,):
            mode = abi.GATE_CHANNEL
        else:
            raise ValueError("gate must be D values, T x 1 or T x D")
        if gate.dtype != torch.float32 or gate.device != device or not gate.is_contiguous():
            raise ValueError(f"gate must be contiguous float32 on {device}")
    args = abi.GemmNormGateArgs(T, D, _ptr(x), ldx, _TYPES[x.dtype], _ptr(y), ldy, y_type,
                                _ptr(weight_post), _ptr(gate), ld_gate, mode,
                                _ptr(weight_pre), residual_scale, eps)
    return device, T, D, args


def gemm_norm_gate(x, y=None, weight_post=None, gate=None, weight_pre=None,
                   residual_scale=1.0, eps=1e-6, x_out=None, h=None, stream=None):
    """(x_out, h): the residual stream after a block, and its norm for the next.

        p     = y / rms(y) * weight_post      (y itself without weight_post)
        x_out = residual_scale * x + gate * p
        h     = x_out / rms(x_out) * weight_pre

    x, y: T x D, float32 or bfloat16 each (y: a block's output, None for none).
    gate: float32, one value per channel (D), per row (T x 1) or per element
    (T x D).  x_out has x's type and may be x; h is bfloat16, or None without
    weight_pre."""
    device, T, D, args = _norm_args(x, y, weight_post, gate, weight_pre, residual_scale, eps)
    x_out, ld_o = _output(x_out, "x_out", (T, D), x.dtype, device)
    ldh = D
    if weight_pre is not None:
        h, ldh = _output(h, "h", (T, D), torch.bfloat16, device)
    elif h is not None:
        raise ValueError("h needs weight_pre")
    _run("gemm_norm_gate", device, stream, args, _ptr(x_out), ld_o, _ptr(h), ldh)
    return x_out, h


class NormGateGrads(NamedTuple):
    """Gradients of gemm_norm_gate; None for an input that was None."""
    dx: torch.Tensor
    dy: torch.Tensor | None
    dweight_post: torch.Tensor | None
    dgate: torch.Tensor | None
    dweight_pre: torch.Tensor | None


def gemm_norm_gate_bwd(x, y=None, d_x_out=None, d_h=None, weight_post=None, gate=None,
                       weight_pre=None, residual_scale=1.0, eps=1e-6, stream=None):
    """NormGateGrads of gemm_norm_gate from the gradients of its outputs.

    d_x_out (x's type) may be None; d_h (float32 or bfloat16) is needed with
    weight_pre.  dx has x's type, dy is bfloat16 (the operand of the gradient
    GEMMs), the others are float32."""
    device, T, D, args = _norm_args(x, y, weight_post, gate, weight_pre, residual_scale, eps)
    if (d_h is None) != (weight_pre is None):
        raise ValueError("d_h goes with weight_pre")
    ld_o = D if d_x_out is None else _matrix(d_x_out, "d_x_out", (x.dtype,), device, (T, D))
    ldh, h_type = D, abi.TYPE_F32
    if d_h is not None:
        ldh, h_type = _matrix(d_h, "d_h", _FLOATS, device, (T, D)), _TYPES[d_h.dtype]
    empty = functools.partial(torch.empty, device=device)
    dx = empty((T, D), dtype=x.dtype)
    dy = None if y is None else empty((T, D), dtype=torch.bfloat16)
    dw_post = None if weight_post is None else empty(D, dtype=torch.float32)
    dw_pre = None if weight_pre is None else empty(D, dtype=torch.float32)
    dgate = None if gate is None else empty(gate.shape, dtype=torch.float32)
    grads = abi.GemmNormGateGrads(_ptr(d_x_out), ld_o, _ptr(d_h), ldh, h_type, _ptr(dx), D,
                                  _ptr(dy), D, _ptr(dgate), _ptr(dw_post), _ptr(dw_pre))
    _run("gemm_norm_gate_bwd", device, stream, args, grads)
    return NormGateGrads(dx, dy, dw_post, dgate, dw_pre)


# --------------------------------------------------- 8-bit checkpoints

class Ckpt8(NamedTuple):
    """A T x N matrix kept in 8 bits (layout: gemm_ckpt8_pack in the header)."""
    q: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int


def _ckpt(kept):
    device = _cuda(kept.q, "kept.q")
    T, N = kept.rows, kept.cols
    _bytes16(kept.q, "kept.q", -(-T // 32) * 32 * N, device)
    if kept.scales.dtype != torch.uint8 or kept.scales.device != device \
            or not kept.scales.is_contiguous() or kept.scales.shape != (-(-T // 32), N):
        raise ValueError("kept.scales must be contiguous uint8, ceil(rows / 32) x cols")
    return device, T, N


def gemm_ckpt8_pack(X, activation=None, act_out=None, stream=None):
    """Keep X (T x N, float32 or bfloat16) in 8 bits: a Ckpt8.  With an activation
    ("none", "relu" or "gelu"): (Ckpt8, act(X) in bfloat16)."""
    device = _cuda(X, "X")
    ldx = _matrix(X, "X", _FLOATS, device)
    T, N = X.shape
    runs = -(-T // 32)
    q = torch.empty(runs * 32 * N, dtype=torch.uint8, device=device)
    scales = torch.empty((runs, N), dtype=torch.uint8, device=device)
    kept = Ckpt8(q, scales, T, N)
    if activation is None:
        if act_out is not None:
            raise ValueError("act_out needs an activation")
        _run("gemm_ckpt8_pack", device, stream, T, N, _ptr(X), ldx, _TYPES[X.dtype],
             _ptr(q), _ptr(scales), abi.ACT_NONE, None, max(N, 1))
        return kept
    act = _act(activation)
    act_out, ld = _output(act_out, "act_out", (T, N), torch.bfloat16, device)
    _run("gemm_ckpt8_pack", device, stream, T, N, _ptr(X), ldx, _TYPES[X.dtype],
         _ptr(q), _ptr(scales), act, _ptr(act_out), ld)
    return kept, act_out


def gemm_ckpt8_unpack(kept, dtype=torch.bfloat16, stream=None):
    """The values kept, T x N (exact in float32 and in bfloat16)."""
    device, T, N = _ckpt(kept)
    if dtype not in _TYPES:
        raise TypeError("dtype must be torch.float32 or torch.bfloat16")
    out = torch.empty((T, N), dtype=dtype, device=device)
    _run("gemm_ckpt8_unpack", device, stream, T, N, _ptr(kept.q), _ptr(kept.scales),
         _ptr(out), max(N, 1), _TYPES[dtype])
    return out


def gemm_ckpt8_act_grad(grad, kept, activation, bias_grad=True, out=None, stream=None):
    """(dZ, dbias) through an activation whose input was kept: dZ = grad *
    act'(kept), bfloat16; dbias: its float32 column sums, or None."""
    device, T, N = _ckpt(kept)
    ldg = _matrix(grad, "grad", _FLOATS, device, (T, N))
    act = _act(activation)
    out, ld = _output(out, "out", (T, N), torch.bfloat16, device)
    dbias = torch.empty(N, dtype=torch.float32, device=device) if bias_grad else None
    _run("gemm_ckpt8_act_grad", device, stream, T, N, _ptr(grad), ldg, _TYPES[grad.dtype],
         _ptr(kept.q), _ptr(kept.scales), act, _ptr(out), ld, _ptr(dbias))
    return out, dbias


def gemm_ckpt8_wgrad(kept, dY, out=None, beta=0.0, stream=None):
    """dW = (values kept)^T @ dY + beta * dW: the float32 weight gradient (K x N) of a
    layer whose input (T x K) was kept, from the bfloat16 dY (T x N)."""
    device, T, K = _ckpt(kept)
    ld = _matrix(dY, "dY", _BF16, device)
    if dY.shape[0] != T:
        raise ValueError(f"dY must have the {T} rows that were kept")
    N = dY.shape[1]
    if beta != 0.0 and out is None:
        raise ValueError("beta != 0 reads dW: pass its prior contents as `out`")
    out, ldw = _output(out, "out", (K, N), torch.float32, device)
    _run("gemm_ckpt8_wgrad", device, stream, T, K, N, _ptr(kept.q), _ptr(kept.scales),
         _ptr(dY), ld, _ptr(out), ldw, beta)
    return out
