"""A layer of experts in 8-bit floating point, from the router to its gradients.

    out = x + sum over the chosen experts of weight * (gelu(x W1^T + b1) W2^T)

Serving (``serve_step``): the experts' rows picked and quantised in one pass, both
products with the GELU in the first one's epilogue.  Training (``train_step``): the
pre-activations kept in 8 bits, every gradient of the layer from the same operators.

    python -m dense_gemm_07_gb300.experts_example --tokens 4096 --width 4096 --hidden 2048
"""
from __future__ import annotations

import argparse

import torch

import dense_gemm_07_gb300 as g7

BF16, F32 = torch.bfloat16, torch.float32


class Experts:
    """Weights of a layer: a BF16 router, E matrices each in 8 bits (and transposed, for
    the gradients), FP32 biases; a bias for balance on the router's scores."""

    def __init__(self, width, hidden, experts, chosen, groups=1, groups_kept=1, seed=0,
                 device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale

        self.router = normal(width, experts, scale=width ** -0.5).to(BF16)
        self.router_t = self.router.t().contiguous()
        self.balance = normal(experts, scale=0.01)
        self.w1 = normal(experts, hidden, width, scale=width ** -0.5).to(BF16)
        self.w2 = normal(experts, width, hidden, scale=hidden ** -0.5).to(BF16)
        self.b1 = normal(experts, hidden, scale=0.1)
        self.w1_q, self.w1_tq = (g7.gemm_fp8_quantize(self.w1, square=True, transpose=t)
                                 for t in (False, True))
        self.w2_q, self.w2_tq = (g7.gemm_fp8_quantize(self.w2, square=True, transpose=t)
                                 for t in (False, True))
        self.chosen = chosen
        self.how = dict(score="sigmoid", renormalize=True, scale=1.5)
        self.groups = dict(groups=groups, groups_kept=groups_kept)

    def route(self, x, open_=None):
        """(logits, Routing); open_: a token per row that is False goes to no expert."""
        logits = g7.gemm_bf16_f32acc(x, self.router)
        if open_ is not None:
            logits = logits.masked_fill(~open_[:, None], float("-inf"))
        return logits, g7.gemm_route(logits, self.chosen, bias=self.balance, **self.how,
                                     **self.groups)


def serve_step(e, x, open_=None):
    """out (x's type), for tokens x (T x width, bfloat16)."""
    _, r = e.route(x, open_)
    a = g7.gemm_fp8_quantize(x, index=r.source)
    h = g7.gemm_fp8_experts(a, e.w1_q, r.offsets, bias=e.b1, activation="gelu", out_dtype=BF16)
    y = g7.gemm_fp8_experts(g7.gemm_fp8_quantize(h), e.w2_q, r.offsets, out_dtype=BF16)
    return g7.gemm_combine(y, r.slot, r.weight, x=x)


def train_step(e, x, d_out, open_=None):
    """(out, gradients of x, router, w1, b1 and w2): one forward and backward pass from
    the gradient of out (bfloat16).  Reads the experts' numbers of rows back once, for
    their weight gradients."""
    logits, r = e.route(x, open_)
    rows, (hidden, width) = r.source.numel(), e.w1.shape[1:]

    def zeros(cols, dtype):  # rows of tokens without an expert stay zero
        return torch.zeros((rows, cols), dtype=dtype, device=x.device)

    a = g7.gemm_fp8_quantize(x, index=r.source)
    z = g7.gemm_fp8_experts(a, e.w1_q, r.offsets, bias=e.b1, out=zeros(hidden, F32))
    z8, h = g7.gemm_ckpt8_pack(z, activation="gelu")
    y = g7.gemm_fp8_experts(g7.gemm_fp8_quantize(h), e.w2_q, r.offsets, out=zeros(width, BF16))
    out = g7.gemm_combine(y, r.slot, r.weight, x=x)
    del z, a

    dy, dw = g7.gemm_combine_bwd(d_out, y, r.slot, r.weight, d_rows=zeros(width, BF16))
    d_logits = g7.gemm_route_bwd(logits, r.index, dw, **e.how)
    dh = g7.gemm_fp8_experts(g7.gemm_fp8_quantize(dy), e.w2_tq, r.offsets, out=zeros(hidden, F32))
    dz, _ = g7.gemm_ckpt8_act_grad(dh, z8, "gelu", bias_grad=False)
    dxe = g7.gemm_fp8_experts(g7.gemm_fp8_quantize(dz), e.w1_tq, r.offsets, out=zeros(width, BF16))
    d_low = d_logits.to(BF16)
    dx = g7.gemm_bf16_f32acc(d_low, e.router_t) + d_out
    g7.gemm_combine(dxe, r.slot, torch.ones_like(r.weight), x=dx, out=dx)
    grads = dict(x=dx, router=g7.gemm_bf16_f32acc(x.t().contiguous(), d_low),
                 w1=torch.zeros_like(e.w1, dtype=F32), w2=torch.zeros_like(e.w2, dtype=F32),
                 b1=torch.zeros_like(e.b1))
    at = r.offsets.tolist()
    for i, (lo, hi) in enumerate(zip(at, at[1:])):
        if lo == hi:
            continue
        turned = [g7.gemm_fp8_quantize(t, transpose=True)
                  for t in (dz[lo:hi], x[r.source[lo:hi].long()], dy[lo:hi], h[lo:hi])]
        g7.gemm_fp8(turned[0], turned[1], out=grads["w1"][i])
        g7.gemm_fp8(turned[2], turned[3], out=grads["w2"][i])
        grads["b1"][i] = dz[lo:hi].sum(0, dtype=F32)
    return out, grads


def _time(f, n=20):
    for _ in range(3):
        f()
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    for _ in range(n):
        f()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / n


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--chosen", type=int, default=4)
    a = p.parse_args(argv)
    e = Experts(a.width, a.hidden, a.experts, a.chosen)
    x = torch.randn((a.tokens, a.width), device="cuda").to(BF16)
    d = torch.randn_like(x)
    train, serve = _time(lambda: train_step(e, x, d), 5), _time(lambda: serve_step(e, x))
    few = _time(lambda: serve_step(e, x[:16]))
    print(f"train step, {a.tokens} tokens, {a.experts} experts of {a.width} x {a.hidden}, "
          f"{a.chosen} a token: {train:.3f} ms")
    print(f"serve step, {a.tokens} tokens: {serve:.3f} ms; 16 tokens: {few * 1e3:.1f} us")
    status = g7.gemm_get_device_status()
    if status:
        raise g7.GemmError(status, "experts_example")


if __name__ == "__main__":
    main()
