"""The layer operators together, as a residual MLP block uses them.

    x_out = scale * x + gate * norm(gelu(norm(x) W1 + b1) W2)

Training (``train_step``): the GEMMs on BF16 tensor cores, the inputs of both and
the pre-activations kept in 8 bits, every gradient of the block from them.
Serving (``decode_step``): the same block for a few rows with 4-bit weights.

    python -m dense_gemm_07_gb300.layer_example --tokens 2048 --width 4096 --hidden 11008
"""
from __future__ import annotations

import argparse

import torch

import dense_gemm_07_gb300 as g7


class Block:
    """Weights of one block: BF16 matrices (and their transposes, for the
    gradients), FP32 vectors, 4-bit copies of the matrices for serving."""

    def __init__(self, width, hidden, seed=0, device="cuda", group=128):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale

        self.w1 = normal(width, hidden, scale=width ** -0.5).to(torch.bfloat16)
        self.w2 = normal(hidden, width, scale=hidden ** -0.5).to(torch.bfloat16)
        self.b1 = normal(hidden, scale=0.1)
        self.pre = 1.0 + normal(width, scale=0.1)       # norm before this block
        self.post = 1.0 + normal(width, scale=0.1)      # norm after it
        self.gate = 0.5 + normal(width, scale=0.1)      # one gate value per channel
        self.next_pre = 1.0 + normal(width, scale=0.1)  # norm before the next block
        self.scale = 0.9
        self.w1_t, self.w2_t = self.w1.t().contiguous(), self.w2.t().contiguous()
        self.group = group
        self.w1_q = g7.w4_quantize(self.w1, group=group, symmetric=False)
        self.w2_q = g7.w4_quantize(self.w2, group=group, symmetric=False)


def train_step(b, x, d_x_out, d_h):
    """(x_out, h, gradients): one forward and backward pass over the tokens of x,
    from the gradients of the two outputs.  What is kept between the passes besides
    x and y is in 8 bits."""
    _, h = g7.gemm_norm_gate(x, weight_pre=b.pre)
    h8 = g7.gemm_ckpt8_pack(h)
    z = g7.gemm_bf16_f32acc_ex(h, b.w1, bias=b.b1)
    z8, a = g7.gemm_ckpt8_pack(z, activation="gelu")
    a8 = g7.gemm_ckpt8_pack(a)
    y = g7.gemm_bf16_f32acc(a, b.w2)
    del h, z, a
    args = dict(weight_post=b.post, gate=b.gate, weight_pre=b.next_pre, residual_scale=b.scale)
    x_out, h_next = g7.gemm_norm_gate(x, y, **args)

    d = g7.gemm_norm_gate_bwd(x, y, d_x_out, d_h, **args)
    dw2 = g7.gemm_ckpt8_wgrad(a8, d.dy)
    da = g7.gemm_bf16_f32acc(d.dy, b.w2_t)
    dz, db1 = g7.gemm_ckpt8_act_grad(da, z8, "gelu")
    dw1 = g7.gemm_ckpt8_wgrad(h8, dz)
    dh = g7.gemm_bf16_f32acc(dz, b.w1_t)
    # the norm before the block, with the residual's gradient added
    d0 = g7.gemm_norm_gate_bwd(x, None, d.dx, dh, weight_pre=b.pre)
    grads = dict(x=d0.dx, w1=dw1, b1=db1, w2=dw2, pre=d0.dweight_pre, post=d.dweight_post,
                 gate=d.dgate, next_pre=d.dweight_pre)
    return x_out, h_next, grads


def decode_step(b, x, h):
    """(x_out, h): the block for a few rows, from the residual stream and its norm."""
    (p1, s1, z1), (p2, s2, z2) = b.w1_q, b.w2_q
    a = g7.gemm_w4(h, p1, s1, zeros=z1, group=b.group, bias=b.b1, activation="gelu",
                   out_dtype=torch.bfloat16)
    y = g7.gemm_w4(a, p2, s2, zeros=z2, group=b.group)
    return g7.gemm_norm_gate(x, y, weight_post=b.post, gate=b.gate, weight_pre=b.next_pre,
                             residual_scale=b.scale)


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
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=11008)
    a = p.parse_args(argv)
    b = Block(a.width, a.hidden)
    x = torch.randn((a.tokens, a.width), device="cuda").to(torch.bfloat16)
    dx, dh = torch.randn_like(x), torch.randn((a.tokens, a.width), device="cuda")
    one = x[:1]
    _, h = g7.gemm_norm_gate(one, weight_pre=b.pre)
    train, decode = _time(lambda: train_step(b, x, dx, dh)), _time(lambda: decode_step(b, one, h))
    flops = 12.0 * a.tokens * a.width * a.hidden
    print(f"train step, {a.tokens} tokens, {a.width} x {a.hidden}: {train:.3f} ms "
          f"({flops / train / 1e9:.0f} TFLOP/s in its six matrix products)")
    print(f"decode step, 1 token: {decode * 1e3:.1f} us")
    status = g7.gemm_get_device_status()
    if status:
        raise g7.GemmError(status, "layer_example")


if __name__ == "__main__":
    main()
