"""Plain 64-bit forms of the layer operators (torch double, any device), written
from their definitions in include/gemm07.h; they import nothing of the package."""
import math

import torch

EPS32 = 2.0 ** -23


def w4_layout_decode(packed, K, N):
    """Codes (K x N) from the packed order, element by element of the definition."""
    KT = -(-K // 128)
    words = packed.cpu().view(torch.int32).to(torch.int64) & 0xFFFFFFFF
    k = torch.arange(K)[:, None]
    n = torch.arange(N)[None, :]
    word = ((n // 16) * KT + k // 128) * 256 + ((n % 16) * 4 + (k % 32) // 8) * 4 + (k % 128) // 32
    e = k % 8
    return ((words[word] >> (4 * (e // 2 + 4 * (e % 2)))) & 15).to(torch.uint8)


def w4_weights(codes, scales, zeros, group):
    g = torch.arange(codes.shape[0], device=codes.device) // group
    z = 8.0 if zeros is None else zeros.double()[g]
    return (codes.double() - z) * scales.double()[g]


def act(v, kind):
    if kind == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if kind == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0))
    return v


def act_slope(v, kind):
    if kind == "relu":
        return torch.where(v.isnan(), v, (v > 0).double())
    if kind == "gelu":
        return 0.5 * torch.erfc(-v / math.sqrt(2.0)) \
            + v * torch.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    return torch.ones_like(v)


def kept(x):
    """The values that the 8-bit checkpoint of x stands for, run by run."""
    x = x.double()
    out = torch.empty_like(x)
    for t in range(0, x.shape[0], 32):
        r = x[t:t + 32]
        top = r.abs().amax(0)
        ok = torch.isfinite(top)
        top = torch.where(ok, top, torch.ones_like(top))
        step = torch.full_like(top, 2.0 ** -126)
        for _ in range(260):  # the smallest power of two that reaches the run
            step = torch.where(top > 127.0 * step, step * 2.0, step)
        step = step.clamp(max=2.0 ** 121)  # 64 of the next step would be 2^128
        v = torch.round(r / step).clamp(-127, 127) * step
        out[t:t + 32] = torch.where(ok, v, torch.full_like(v, math.nan))
    return out


class Norm:
    """gemm_norm_gate and its gradient in 64 bits, with the magnitudes that the
    error bounds go by."""

    def __init__(self, x, y, w_post, gate, w_pre, alpha, eps):
        d = lambda t: None if t is None else t.double()  # noqa: E731
        self.x, self.y, self.w_post, self.gate, self.w_pre = map(d, (x, y, w_post, gate, w_pre))
        self.alpha, self.eps = alpha, eps
        self.g = 1.0 if gate is None else self.gate
        if y is None:
            self.r2, self.n = 1.0, torch.zeros_like(self.x)
        elif w_post is None:
            self.r2, self.n = 1.0, self.y
        else:
            self.r2 = 1.0 / torch.sqrt((self.y ** 2).mean(1, keepdim=True) + eps)
            self.n = self.y * self.r2
        self.p = self.n if w_post is None else self.n * self.w_post
        self.u = alpha * self.x + self.g * self.p
        self.u_size = (alpha * self.x).abs() + (self.g * self.p).abs()
        self.r1 = 1.0 / torch.sqrt((self.u ** 2).mean(1, keepdim=True) + eps)
        self.h = None if w_pre is None else self.u * self.r1 * self.w_pre

    def backward(self, d_x_out, dh):
        D = self.x.shape[1]
        du = torch.zeros_like(self.x) if d_x_out is None else d_x_out.double()
        size = du.abs()
        dw_pre = pre_size = None
        if dh is not None:
            dh = dh.double()
            t = dh * self.w_pre
            c = (t * self.u).sum(1, keepdim=True) / D
            du = du + self.r1 * (t - self.u * self.r1 ** 2 * c)
            size = size + self.r1 * (t.abs() + self.u_size * self.r1 ** 2
                                     * (t * self.u_size).abs().mean(1, keepdim=True))
            dw_pre = (dh * self.u * self.r1).sum(0)
            pre_size = (dh.abs() * self.u_size * self.r1).sum(0)
        out = {"dx": self.alpha * du, "dw_pre": dw_pre}
        bound = {"dx": abs(self.alpha) * size, "dw_pre": pre_size}
        if self.y is None:
            return out, bound
        dp = self.g * du
        dp_size = abs(self.g) * size if self.gate is None else self.gate.abs() * size
        if self.w_post is None:
            out["dy"], bound["dy"] = dp, dp_size
        else:
            t = dp * self.w_post
            ts = dp_size * self.w_post.abs()
            out["dy"] = self.r2 * (t - self.n * (t * self.n).mean(1, keepdim=True))
            bound["dy"] = self.r2 * (ts + self.n.abs() * (ts * self.n.abs()).mean(1, keepdim=True))
            out["dw_post"] = (dp * self.n).sum(0)
            bound["dw_post"] = (dp_size * self.n.abs()).sum(0)
        if self.gate is not None:
            dg, gs = du * self.p, size * self.p.abs()
            T = self.x.shape[0]
            if self.gate.dim() == 1:
                dg, gs = dg.sum(0), gs.sum(0)
            elif self.gate.shape == (T, 1) and D != 1:
                dg, gs = dg.sum(1, keepdim=True), gs.sum(1, keepdim=True)
            out["dgate"], bound["dgate"] = dg, gs
        return out, bound
