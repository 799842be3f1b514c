"""Products in 8-bit floating point, and the layer of experts that is made of them:
routing, the experts' products, combining.

As in ``layer``, every function passes CUDA tensors to the C entry point of its name
(declared in ``include/gemm07.h``) through the compiled binding, on ``stream``
(default: the current stream; tensors that a call makes come from the current
stream's memory).  Matrices have contiguous rows and any row stride unless it says
otherwise; a refused argument raises ValueError or TypeError, a status of the library
GemmError.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from .layer import _binding, _handle

# ---------------------------------------------- 8-bit floating-point products


class Fp8(NamedTuple):
    """A matrix (R x K) in 8-bit floating point: codes times scales.

    codes: torch.float8_e4m3fn, rows a multiple of 16 bytes apart.
    scales: float32; a scale for each 128 values of a row is scales[k // 128, r]
    (square False), one for each 128 x 128 values scales[r // 128, k // 128].
    E matrices of weights have codes E x R x K and scales E x ... (square)."""
    codes: torch.Tensor
    scales: torch.Tensor
    square: bool = False


def gemm_fp8_quantize(X, square=False, transpose=False, index=None, stream=None):
    """X (float32 or bfloat16) in 8-bit floating point, an Fp8: a power-of-two scale
    for each 128 values of a row, or for each 128 x 128 (square), and the nearest
    codes.

    transpose: the codes are X^T's.  index (int32): the rows of X to take, in that
    order; a row of zeros where it is outside X (-1).  With square, X may be E
    matrices (E x R x K)."""
    codes, scales = _binding().fp8_quantize(X, square, transpose, index, _handle(stream))
    return Fp8(codes, scales, square)


def gemm_fp8(a, b, out=None, alpha=1.0, beta=0.0, bias=None, activation="none", out_dtype=None,
             stream=None):
    """C = act(alpha * A @ B^T + beta * C + bias) of two Fp8: a (M x K) with a scale
    for each 128 values of a row, b (N x K) likewise or with square scales.  C is
    float32 (out_dtype) or bfloat16."""
    return _binding().fp8(*a, *b, out, alpha, beta, bias, activation, out_dtype, _handle(stream))


def gemm_fp8_experts(a, b, offsets, out=None, alpha=1.0, beta=0.0, bias=None, activation="none",
                     out_dtype=None, stream=None):
    """gemm_fp8 of rows sorted by expert: rows offsets[e] .. offsets[e + 1] - 1 of a
    (an Fp8, M x K) with the e-th matrix of b (an Fp8 of E x N x K, square).

    offsets: int32, E + 1, on the device (Routing.offsets); rows outside of them are
    not written, and hold anything in an out that the call makes.  bias: float32, E x N."""
    return _binding().fp8_experts(*a, *b, offsets, out, alpha, beta, bias, activation, out_dtype,
                                  _handle(stream))


# --------------------------------------------------------------- experts

class Routing(NamedTuple):
    """Experts of T tokens, k each, and the chosen pairs sorted by expert (parts of one
    block of memory)."""
    index: torch.Tensor    # T x k int32: the experts, best first; -1: none
    weight: torch.Tensor   # T x k float32
    slot: torch.Tensor     # T x k int32: the pair's row in the sorted order; -1: none
    source: torch.Tensor   # T * k int32: the token of each row; -1 past the last
    offsets: torch.Tensor  # E + 1 int32: the first row of each expert


def gemm_route(logits, k, score="softmax", bias=None, groups=1, groups_kept=None, group_top=2,
               renormalize=True, scale=1.0, stream=None):
    """The Routing of tokens by their logits (T x E, float32 or bfloat16).

    The k experts with the largest score ("softmax" over the logits or "sigmoid" of
    each) + bias (float32, E), ties to the lowest; with groups_kept < groups only from
    the groups whose group_top best have the largest sums.  Weights are scale * score,
    over their sum when renormalize.  An expert with the logit -inf is not chosen."""
    return Routing(*_binding().route(logits, k, score, bias, groups,
                                     groups if groups_kept is None else groups_kept, group_top,
                                     renormalize, scale, _handle(stream)))


def gemm_route_bwd(logits, index, d_weight, score="softmax", renormalize=True, scale=1.0,
                   out=None, stream=None):
    """The gradient of the logits (their type) from that of Routing.weight."""
    return _binding().route_bwd(logits, index, d_weight, score, renormalize, scale, out,
                                _handle(stream))


def gemm_combine(rows, slot, weight, x=None, out=None, out_dtype=None, stream=None):
    """x + the weighted sum of each token's rows: out[t] = x[t] + sum over j of
    weight[t, j] * rows[slot[t, j]] (slot -1: no row).  out has x's type, or the rows'
    without x, unless out_dtype says otherwise."""
    return _binding().combine(rows, slot, weight, x, out, out_dtype, _handle(stream))


def gemm_combine_bwd(d_out, rows, slot, weight, d_rows=None, stream=None):
    """(d_rows, d_weight) of gemm_combine for distinct slots, as a Routing's are: a row
    that two slots name would need the sum of two gradients, and gets either of them.
    Rows that no slot names are zero in a new d_rows, which the call clears first, and
    stay as they are in one that is passed."""
    return _binding().combine_bwd(d_out, rows, slot, weight, d_rows, _handle(stream))
