"""Timed cases of the operators that stand beside the dense GEMM in a
transformer layer:

  w4          products of a few rows with a 4-bit weight matrix (group scales)
  norm        RMS norms after and before a block, fused with the block's gate
              and the scaled residual; norm_bwd is the gradient
  ckpt_act    pre-activations kept in 8 bits, and the activation's gradient
              and the bias gradient computed from them
  ckpt_wgrad  a layer's input kept in 8 bits, and the weight gradient from it

`run` computes a case with the package's kernels where `own` is true, and in
elementary torch operations in 32 bits where it is false; `exact` gives the
same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}
SIZE = {"f32": 4, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # one token through a square projection: the latency of a decode step
        dict(name="w4 1x4096x4096", op="w4", M=1, K=4096, N=4096, group=128,
             zeros=False, act="none", bias=False, out="f32"),
        # a few sequences, ragged in every size, small groups with zero points,
        # and a whole MLP epilogue
        dict(name="w4 5x3001x1000", op="w4", M=5, K=3001, N=1000, group=32,
             zeros=True, act="gelu", bias=True, out="bf16"),
        # sixteen sequences, a weight matrix larger than L2
        dict(name="w4 16x8192x32768", op="w4", M=16, K=8192, N=32768, group=64,
             zeros=True, act="none", bias=False, out="f32"),
        # one token between two blocks
        dict(name="norm 1x4096", op="norm", T=1, D=4096, x="bf16", y="f32", gate="channel"),
        # an odd prompt, FP32 residual stream, a gate computed for every element
        dict(name="norm 2047x4096", op="norm", T=2047, D=4096, x="f32", y="f32", gate="full"),
        # training, a width that no vector divides, one gate value per token
        dict(name="norm_bwd 1000x3001", op="norm_bwd", T=1000, D=3001, x="f32", y="f32",
             gate="row"),
        # training, a long batch, BF16 residual stream
        dict(name="norm_bwd 8192x4096", op="norm_bwd", T=8192, D=4096, x="bf16", y="f32",
             gate="channel"),
        # a small ragged layer with ReLU
        dict(name="ckpt_act 127x1000", op="ckpt_act", T=127, N=1000, act="relu", z="bf16",
             g="bf16"),
        # the wide layer of an MLP with GELU
        dict(name="ckpt_act 2048x11008", op="ckpt_act", T=2048, N=11008, act="gelu", z="f32",
             g="f32"),
        # a small layer: few tiles, latency
        dict(name="ckpt_wgrad 127x127x1000", op="ckpt_wgrad", T=127, K=127, N=1000, x="bf16"),
        # odd everywhere: rows of dY that no 16 bytes divide
        dict(name="ckpt_wgrad 3001x1000x3001", op="ckpt_wgrad", T=3001, K=1000, N=3001,
             x="f32"),
        # the wide layer of an MLP over a long batch
        dict(name="ckpt_wgrad 4096x4096x11008", op="ckpt_wgrad", T=4096, K=4096, N=11008,
             x="bf16"),
    ]


def _size(rng, lo, hi):
    """Log-uniform over [lo, hi], half of the time rounded to a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 128:
        v = v // 64 * 64
    v = min(max(v, lo), hi)
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["w4", "norm", "norm_bwd", "ckpt_act", "ckpt_wgrad"])
    if op == "w4":
        K = _size(rng, 64, 16384)
        return dict(op=op, M=rng.randint(1, 16), K=K,
                    N=_size(rng, 64, min(32768, 8192 * 32768 // K)),
                    group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu"]), bias=rng.random() < 0.5,
                    out=rng.choice(["f32", "bf16"]))
    if op in ("norm", "norm_bwd"):
        D = _size(rng, 64, 8192)
        return dict(op=op, T=_size(rng, 1, min(8192, 8192 * 4096 // D)), D=D,
                    x=rng.choice(["f32", "bf16"]), y=rng.choice(["f32", "bf16"]),
                    gate=rng.choice(["none", "channel", "row", "full"]))
    if op == "ckpt_act":
        N = _size(rng, 64, 11008)
        return dict(op=op, T=_size(rng, 1, min(8192, 2048 * 11008 // N)), N=N,
                    act=rng.choice(["relu", "gelu"]), z=rng.choice(["f32", "bf16"]),
                    g=rng.choice(["f32", "bf16"]))
    return dict(op=op, T=_size(rng, 16, 4096), K=_size(rng, 64, 4096),
                N=_size(rng, 64, 11008), x=rng.choice(["f32", "bf16"]))


def work(case):
    c, op = case, case["op"]
    if op == "w4":
        M, K, N = c["M"], c["K"], c["N"]
        groups = -(-K // c["group"])
        w = K * N // 2 + groups * N * (3 if c["zeros"] else 2)
        return dict(bytes=w + 2 * M * K + SIZE[c["out"]] * M * N + (4 * N if c["bias"] else 0),
                    flops=2 * M * K * N)
    if op in ("norm", "norm_bwd"):
        T, D, x, y = c["T"], c["D"], SIZE[c["x"]], SIZE[c["y"]]
        gate = {"none": 0, "channel": 4 * D, "row": 4 * T, "full": 4 * T * D}[c["gate"]]
        if op == "norm":
            return dict(bytes=T * D * (2 * x + y + 2) + 8 * D + gate, flops=10 * T * D)
        # x, dx_out and dx; y and dh; dy in BF16
        return dict(bytes=T * D * (3 * x + 2 * y + 2) + 16 * D + 2 * gate, flops=30 * T * D)
    if op == "ckpt_act":
        n = c["T"] * c["N"]
        # z and the gradient in, the activations and dz out, 8.25 bits kept and read
        kept = n + -(-c["T"] // 32) * c["N"]
        return dict(bytes=n * (SIZE[c["z"]] + SIZE[c["g"]] + 4) + 2 * kept + 4 * c["N"],
                    flops=40 * n)
    T, K, N = c["T"], c["K"], c["N"]
    kept = T * K + -(-T // 32) * K
    return dict(bytes=T * K * SIZE[c["x"]] + 2 * kept + 2 * T * N + 4 * K * N,
                flops=2 * T * K * N)


# ---------------------------------------------------------------- inputs

def _inputs(case, seed, dev):
    """The case's data, from the seed alone."""
    c, op = case, case["op"]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=F32, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    s = dict(case)
    if op == "w4":
        M, K, N, grp = c["M"], c["K"], c["N"], c["group"]
        G = -(-K // grp)
        s["a"] = normal(M, K, dtype=BF16)
        s["codes"] = torch.randint(0, 16, (K, N), generator=g, device=dev, dtype=torch.uint8)
        s["scales"] = ((torch.rand((G, N), generator=g, device=dev) + 0.5)
                       * (0.2 / math.sqrt(K))).to(BF16)
        s["zero"] = torch.randint(4, 13, (G, N), generator=g, device=dev, dtype=torch.uint8) \
            if c["zeros"] else None
        s["bias_v"] = normal(N, scale=0.1) if c["bias"] else None
    elif op in ("norm", "norm_bwd"):
        T, D = c["T"], c["D"]
        # rows of unlike sizes, as a residual stream has them
        rows = torch.exp(torch.randn((T, 1), generator=g, device=dev) * 0.5)
        s["xs"] = (normal(T, D) * rows).to(DTYPES[c["x"]])
        s["ys"] = (normal(T, D) * rows.flip(0) * 3.0).to(DTYPES[c["y"]])
        s["w_post"] = 1.0 + normal(D, scale=0.1)
        s["w_pre"] = 1.0 + normal(D, scale=0.1)
        shape = {"none": None, "channel": (D,), "row": (T, 1), "full": (T, D)}[c["gate"]]
        s["gates"] = None if shape is None else torch.rand(shape, generator=g, device=dev) + 0.25
        s["scale"] = 0.875
        if op == "norm_bwd":
            s["dx_out"] = normal(T, D, dtype=DTYPES[c["x"]])
            s["dh"] = normal(T, D, dtype=DTYPES[c["y"]])
    elif op == "ckpt_act":
        s["zs"] = normal(c["T"], c["N"], scale=1.5, dtype=DTYPES[c["z"]])
        s["gs"] = normal(c["T"], c["N"], dtype=DTYPES[c["g"]])
    else:
        T, K, N = c["T"], c["K"], c["N"]
        # channels of unlike sizes, a few of them large and some without a value
        ch = torch.exp(torch.randn((1, K), generator=g, device=dev))
        ch = ch * (torch.rand((1, K), generator=g, device=dev) > 0.03)
        s["xs"] = (normal(T, K) * ch).to(DTYPES[c["x"]])
        s["dy"] = normal(T, N, dtype=BF16)
    return s


def _w4_layout(codes):
    """4-bit codes (K x N) in the order that `gemm_w4` reads: tiles of 16 columns
    by 128 rows of 1 KB; in a tile word (half, column, quarter, block) holds rows
    32 * block + 8 * quarter .. + 7 of column 8 * half + column, the even rows in
    its low 16 bits and the odd ones in its high 16 bits."""
    K, N = codes.shape
    kt, nt = -(-K // 128), -(-N // 16)
    c = torch.nn.functional.pad(codes, (0, nt * 16 - N, 0, kt * 128 - K))
    c = c.view(kt, 4, 4, 4, 2, nt, 2, 8)       # k tile, block, quarter, pair, odd, n tile, half, col
    c = c.permute(5, 0, 6, 7, 2, 1, 4, 3)      # nt kt half col quarter block odd pair
    c = c.reshape(-1, 2)                       # low nibble first
    return (c[:, 0] | (c[:, 1] << 4)).view(nt, kt, 1024)


def prepare(case, seed):
    s = _inputs(case, seed, "cuda")
    if case["op"] == "w4":
        s["packed"] = _w4_layout(s["codes"])
    return s


# ------------------------------------------------------------ plain forms

def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return v * 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v


def _act_slope(v, act):
    if act == "relu":
        return (v > 0).to(v.dtype)
    return 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5))) \
        + v * torch.exp(v * v * -0.5) * (1.0 / math.sqrt(2.0 * math.pi))


def _kept(x):
    """What the 8-bit checkpoint of x (T x K) stands for: in each run of 32 rows of
    a column, whole multiples (-127..127) of the smallest power of two (at least
    2^-126) that reaches the run's largest magnitude; NaN where a run holds a value
    that is not finite."""
    T, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, 0, 0, -T % 32)).view(-1, 32, K)
    top = v.abs().amax(1, keepdim=True)
    m, e = torch.frexp(top)
    e = (e.to(torch.int32) - 7 + (m > 127.0 / 128.0).to(torch.int32)).clamp(min=-126)
    e = torch.where(torch.isfinite(top), e, torch.zeros_like(e))
    # powers of two from their bits: 2^e, -126 <= e <= 121
    up, down = ((127 + e) << 23).view(F32), ((127 - e) << 23).view(F32)
    v = torch.round(v * down) * up
    v = torch.where(torch.isfinite(top), v, torch.full_like(v, math.nan))
    return v.view(-1, K)[:T]


def _plain(s):
    op = s["op"]
    if op == "w4":
        grp, K = s["group"], s["K"]
        sc = s["scales"].float().repeat_interleave(grp, 0)[:K]
        z = 8.0 if s["zero"] is None else s["zero"].float().repeat_interleave(grp, 0)[:K]
        v = torch.matmul(s["a"].float(), (s["codes"].float() - z) * sc)
        if s["bias_v"] is not None:
            v = v + s["bias_v"]
        return _act(v, s["act"]).to(DTYPES[s["out"]])
    if op in ("norm", "norm_bwd"):
        x, y, a = s["xs"].float(), s["ys"].float(), s["scale"]
        g = s["gates"]
        r2 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        n = y * r2
        p = n * s["w_post"]
        u = a * x + (p if g is None else g * p)
        r1 = torch.rsqrt((u * u).mean(1, keepdim=True) + EPS)
        if op == "norm":
            return {"x_out": u.to(s["xs"].dtype), "h": (u * r1 * s["w_pre"]).to(BF16)}
        dh = s["dh"].float()
        dn = dh * s["w_pre"]
        du = s["dx_out"].float() + r1 * (dn - u * (r1 * r1 * (dn * u).mean(1, keepdim=True)))
        dp = du if g is None else g * du
        dm = dp * s["w_post"]
        out = {"dx": (a * du).to(s["xs"].dtype),
               "dy": (r2 * (dm - n * (dm * n).mean(1, keepdim=True))).to(BF16),
               "dw_post": (dp * n).sum(0), "dw_pre": (dh * u * r1).sum(0)}
        if g is not None:
            dg = du * p
            out["dgate"] = {"channel": lambda: dg.sum(0), "row": lambda: dg.sum(1, keepdim=True),
                            "full": lambda: dg}[s["gate"]]()
        return out
    if op == "ckpt_act":
        z = s["zs"].float()
        dz = s["gs"].float() * _act_slope(_kept(z), s["act"])
        return {"act": _act(z, s["act"]).to(BF16), "dz": dz.to(BF16), "dbias": dz.sum(0)}
    return torch.matmul(_kept(s["xs"]).t(), s["dy"].float())


def run(state):
    s = state
    if not own:
        return _plain(s)
    import dense_gemm_07_gb300 as g7
    op = s["op"]
    if op == "w4":
        return g7.gemm_w4(s["a"], s["packed"], s["scales"], zeros=s["zero"], group=s["group"],
                          bias=s["bias_v"], activation=s["act"], out_dtype=DTYPES[s["out"]])
    if op == "norm":
        x_out, h = g7.gemm_norm_gate(s["xs"], s["ys"], weight_post=s["w_post"], gate=s["gates"],
                                     weight_pre=s["w_pre"], residual_scale=s["scale"], eps=EPS)
        return {"x_out": x_out, "h": h}
    if op == "norm_bwd":
        d = g7.gemm_norm_gate_bwd(s["xs"], s["ys"], s["dx_out"], s["dh"],
                                  weight_post=s["w_post"], gate=s["gates"],
                                  weight_pre=s["w_pre"], residual_scale=s["scale"], eps=EPS)
        out = {"dx": d.dx, "dy": d.dy, "dw_post": d.dweight_post, "dw_pre": d.dweight_pre}
        if s["gates"] is not None:
            out["dgate"] = d.dgate
        return out
    if op == "ckpt_act":
        kept, act = g7.gemm_ckpt8_pack(s["zs"], activation=s["act"])
        dz, dbias = g7.gemm_ckpt8_act_grad(s["gs"], kept, activation=s["act"])
        return {"act": act, "dz": dz, "dbias": dbias}
    kept = g7.gemm_ckpt8_pack(s["xs"])
    return g7.gemm_ckpt8_wgrad(kept, s["dy"])


# ---------------------------------------------------------------- 64 bits

def _kept64(x):
    """The checkpoint's values, run by run from the definition."""
    x = x.double()
    T, K = x.shape
    out = torch.empty_like(x)
    for t in range(0, T, 32):
        run_ = x[t:t + 32]
        top = run_.abs().max(0).values
        e = torch.ceil(torch.log2(top / 127.0)).clamp(min=-126.0).to(torch.int64)
        step = ((1023 + e) << 52).view(torch.float64)
        # log2 may fall on the wrong side of a whole number: settle it exactly
        step = torch.where(top / step > 127.0, step * 2, step)
        lower = (step * 0.5).clamp(min=2.0 ** -126)
        step = torch.where(top / lower <= 127.0, lower, step)
        out[t:t + 32] = torch.round(run_ / step) * step
    return out


def exact(case, seed):
    s = _inputs(case, seed, "cuda")
    op = s["op"]
    rt2 = math.sqrt(2.0)

    def cdf(v):
        return 0.5 * torch.erfc(-v / rt2)

    def act64(v, act):
        return v if act == "none" else v.clamp(min=0.0) if act == "relu" else v * cdf(v)

    if op == "w4":
        K, grp = s["K"], s["group"]
        at = torch.arange(K, device="cuda") // grp
        acc = torch.zeros((s["M"], s["N"]), dtype=torch.float64, device="cuda")
        for k in range(0, K, 2048):
            r = at[k:k + 2048]
            zero = 8.0 if s["zero"] is None else s["zero"][r].double()
            w = (s["codes"][k:k + 2048].double() - zero) * s["scales"][r].double()
            acc += s["a"][:, k:k + 2048].double() @ w
        if s["bias_v"] is not None:
            acc += s["bias_v"].double()
        return act64(acc, s["act"])
    if op in ("norm", "norm_bwd"):
        D = s["D"]
        x, y = s["xs"].double(), s["ys"].double()
        w2, w1, a = s["w_post"].double(), s["w_pre"].double(), s["scale"]
        g = 1.0 if s["gates"] is None else s["gates"].double()
        rms_y = ((y ** 2).sum(1, keepdim=True) / D + EPS).sqrt()
        p = y / rms_y * w2
        u = a * x + g * p
        rms_u = ((u ** 2).sum(1, keepdim=True) / D + EPS).sqrt()
        if op == "norm":
            return {"x_out": u, "h": u / rms_u * w1}
        dh = s["dh"].double()
        uh = u / rms_u
        t = dh * w1
        du = s["dx_out"].double() + (t - uh * (t * uh).sum(1, keepdim=True) / D) / rms_u
        yh = y / rms_y
        t2 = du * g * w2
        out = {"dx": a * du, "dy": (t2 - yh * (t2 * yh).sum(1, keepdim=True) / D) / rms_y,
               "dw_post": (du * g * yh).sum(0), "dw_pre": (dh * uh).sum(0)}
        if s["gates"] is not None:
            dg = du * p
            out["dgate"] = dg.sum(0) if s["gate"] == "channel" else \
                dg.sum(1, keepdim=True) if s["gate"] == "row" else dg
        return out
    if op == "ckpt_act":
        z, k = s["zs"].double(), _kept64(s["zs"])
        if s["act"] == "relu":
            slope = torch.where(k > 0, 1.0, 0.0).double()
        else:
            slope = cdf(k) + k * torch.exp(-0.5 * k ** 2) / math.sqrt(2.0 * math.pi)
        dz = s["gs"].double() * slope
        return {"act": act64(z, s["act"]), "dz": dz, "dbias": dz.sum(0)}
    return _kept64(s["xs"]).t() @ s["dy"].double()
