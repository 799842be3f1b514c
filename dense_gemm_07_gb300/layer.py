"""The operators of a transformer layer around the GEMM: 4-bit weights, norms
with gate and residual, 8-bit activation checkpoints.

Every function passes CUDA tensors to the C entry point of its name (declared in
``include/gemm07.h``) through the compiled binding ``csrc/layer_binding.cpp``, on
``stream`` (default: the current stream).  Tensors that a call makes come from the
current stream's memory, as in the rest of the package: another ``stream`` has to
wait for the current one first, as it has to for the operands.  Matrices have
contiguous rows and any row stride; a refused argument raises ValueError or
TypeError, a status of the library GemmError.
"""
from __future__ import annotations

import functools
import importlib.machinery
import importlib.util
from typing import NamedTuple

import torch

from . import _build


@functools.lru_cache(maxsize=None)
def _binding():
    """The compiled binding (built first if needed); there is no other path."""
    loader = importlib.machinery.ExtensionFileLoader("layer_binding", _build.build_binding())
    spec = importlib.util.spec_from_loader("layer_binding", loader)
    module = importlib.util.module_from_spec(spec)
    loader.exec_module(module)
    return module


def _handle(stream):
    return None if stream is None else stream.cuda_stream


# ---------------------------------------------------------- 4-bit weights

def gemm_w4(A, packed, scales, zeros=None, group=128, out=None, alpha=1.0, beta=0.0,
            bias=None, activation="none", out_dtype=None, stream=None):
    """C = act(alpha * A @ W + beta * C + bias) for a bfloat16 A of a few rows and
    4-bit weights W[k, n] = (q[k, n] - z[k // group, n]) * scales[k // group, n].

    packed: from w4_pack or w4_quantize; scales: bfloat16, ceil(K / group) x N;
    zeros: uint8 of the same shape, or None (z = 8).  C is float32 (out_dtype)
    or bfloat16."""
    return _binding().w4(A, packed, scales, zeros, group, out, alpha, beta, bias, activation,
                         out_dtype, _handle(stream))


def w4_pack(codes, stream=None):
    """4-bit codes (uint8, K x N, the low four bits of each) in the packed order
    that gemm_w4 reads."""
    return _binding().w4_pack(codes, _handle(stream))


def w4_quantize(B, group=128, symmetric=True, stream=None):
    """(packed, scales, zeros) of a float32 or bfloat16 matrix B (K x N), rounded to
    the nearest 4-bit codes; zeros is None when symmetric."""
    return _binding().w4_quantize(B, group, symmetric, _handle(stream))


def w4_unpack(packed, scales, zeros=None, group=128, K=None, stream=None):
    """The K x N bfloat16 matrix that the 4-bit weights stand for (for prompts:
    gemm_bf16_f32acc).  K defaults to all rows of the groups."""
    return _binding().w4_unpack(packed, scales, zeros, group, K, _handle(stream))


# ------------------------------------------------- norms, gate, residual

def gemm_norm_gate(x, y=None, weight_post=None, gate=None, weight_pre=None,
                   residual_scale=1.0, eps=1e-6, x_out=None, h=None, stream=None):
    """(x_out, h): the residual stream after a block, and its norm for the next.

        p     = y / rms(y) * weight_post      (y itself without weight_post)
        x_out = residual_scale * x + gate * p
        h     = x_out / rms(x_out) * weight_pre

    x, y: T x D, float32 or bfloat16 each (y: a block's output, None for none).
    gate: float32, one value per channel (D), per row (T x 1; both contiguous) or
    per element (T x D).  x_out has x's type and may be x; h is bfloat16, or None without
    weight_pre."""
    return _binding().norm_gate(x, y, weight_post, gate, weight_pre, residual_scale, eps, x_out, h,
                                _handle(stream))


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
    GEMMs), the others are float32; dgate has the shape and the row stride of gate."""
    return NormGateGrads(*_binding().norm_gate_bwd(x, y, d_x_out, d_h, weight_post, gate,
                                                   weight_pre, residual_scale, eps,
                                                   _handle(stream)))


# --------------------------------------------------- 8-bit checkpoints

class Ckpt8(NamedTuple):
    """A T x N matrix kept in 8 bits (layout: gemm_ckpt8_pack in the header)."""
    q: torch.Tensor
    scales: torch.Tensor
    rows: int
    cols: int


def gemm_ckpt8_pack(X, activation=None, act_out=None, stream=None):
    """Keep X (T x N, float32 or bfloat16) in 8 bits: a Ckpt8.  With an activation
    ("none", "relu" or "gelu"): (Ckpt8, act(X) in bfloat16)."""
    q, scales, act = _binding().ckpt8_pack(X, activation, act_out, _handle(stream))
    rows, cols = X.shape
    kept = Ckpt8(q, scales, rows, cols)
    return kept if activation is None else (kept, act)


def gemm_ckpt8_unpack(kept, dtype=torch.bfloat16, stream=None):
    """The values kept, T x N (exact in float32 and in bfloat16)."""
    return _binding().ckpt8_unpack(*kept, dtype, _handle(stream))


def gemm_ckpt8_act_grad(grad, kept, activation, bias_grad=True, out=None, stream=None):
    """(dZ, dbias) through an activation whose input was kept: dZ = grad *
    act'(kept), bfloat16; dbias: its float32 column sums, or None."""
    q, scales, rows, cols = kept
    return _binding().ckpt8_act_grad(grad, q, scales, rows, cols, activation, bias_grad, out,
                                     _handle(stream))


def gemm_ckpt8_wgrad(kept, dY, out=None, beta=0.0, stream=None):
    """dW = (values kept)^T @ dY + beta * dW: the float32 weight gradient (K x N) of a
    layer whose input (T x K) was kept, from the bfloat16 dY (T x N)."""
    return _binding().ckpt8_wgrad(*kept, dY, out, beta, _handle(stream))
