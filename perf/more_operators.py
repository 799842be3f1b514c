"""Timed cases of the operators of a layer of experts, and of the 8-bit products
that it and the dense layers use:

  quantize   a matrix in 8-bit floating point, a scale for each 128 values of a
             row; the rows picked by an index, or the matrix transposed
  fp8        products of two such matrices, the second one also with a scale for
             each 128 x 128 values (weights)
  experts    products of rows sorted by expert with the expert's weights
  route      tokens to experts: scores, choice, weights, and the sorted order;
             route_bwd is the gradient of the weights
  combine    the experts' rows back to their tokens; combine_bwd is the gradient

`run` computes a case with the package's kernels where `own` is true, and in
elementary torch operations where it is false (in 32 bits; the choice of experts,
which is a comparison of nearly equal numbers, in 64); `exact` gives the same
outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
DTYPES = {"f32": F32, "bf16": BF16}
SIZE = {"f32": 4, "bf16": 2}
B = 128  # values that share a scale


def listed():
    return [
        # activations for a weight gradient: the transposed matrix, ragged both ways
        dict(name="quantize 127x1000 transposed", op="quantize", T=127, C=1000, rows=0, x="bf16",
             transpose=True),
        # the tokens of a long batch, each copied to its four experts' rows
        dict(name="quantize 16384 of 4096x4096", op="quantize", T=4096, C=4096, rows=16384,
             x="bf16", transpose=False),
        # one token through a square projection: the latency of a decode step
        dict(name="fp8 1x4096x4096", op="fp8", M=1, K=4096, N=4096, square=True, bias=False,
             act="none", out="bf16"),
        # a weight gradient: both factors with a scale for each 128 values of a row, odd sizes
        dict(name="fp8 1000x3001x1000 rows", op="fp8", M=1000, K=3001, N=1000, square=False,
             bias=False, act="none", out="f32"),
        # the wide layer of an MLP over a long batch, with its epilogue
        dict(name="fp8 4096x4096x11008", op="fp8", M=4096, K=4096, N=11008, square=True,
             bias=True, act="gelu", out="bf16"),
        # a decode step of sixteen sequences, two experts each: reading weights
        dict(name="experts 32x4096x4096 of 8", op="experts", R=32, K=4096, N=4096, E=8, bias=False,
             act="none", out="bf16"),
        # training or a long prompt: many experts, unlike numbers of rows
        dict(name="experts 16384x4096x2048 of 64", op="experts", R=16384, K=4096, N=2048, E=64,
             bias=True, act="relu", out="bf16"),
        # a decode step's router
        dict(name="route 1x64", op="route", T=1, E=64, k=4, score="softmax", bias=False, groups=1,
             kept=1, group_top=1, renorm=True, x="f32", pad=0),
        # a long batch, experts in groups, a bias that balances them, some padding behind it
        dict(name="route 16384x256", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True,
             groups=8, kept=4, group_top=2, renorm=True, x="f32", pad=100),
        # training: the gradient through the weights, odd sizes
        dict(name="route_bwd 8191x257", op="route_bwd", T=8191, E=257, k=6, score="softmax",
             bias=False, groups=1, kept=1, group_top=1, renorm=True, x="bf16", pad=0),
        # an odd prompt, rows that no vector divides, added to the residual stream
        dict(name="combine 1000x3001", op="combine", T=1000, D=3001, k=5, E=60, rows="bf16",
             x=True, out="f32", pad=17),
        # training, a long batch
        dict(name="combine_bwd 4096x4096", op="combine_bwd", T=4096, D=4096, k=8, E=256,
             rows="bf16", x=False, out="bf16", pad=0),
    ]


def _size(rng, lo, hi):
    """Log-uniform over [lo, hi], half of the time rounded to a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 128:
        v = v // 64 * 64
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["quantize", "fp8", "fp8", "experts", "experts", "route", "route_bwd",
                     "combine", "combine_bwd"])
    if op == "quantize":
        C = _size(rng, 64, 11008)
        T = _size(rng, 1, min(8192, 4096 * 4096 // C))
        kind = rng.choice(["plain", "index", "transpose"])
        return dict(op=op, T=T, C=C, rows=_size(rng, 1, 4 * T) if kind == "index" else 0,
                    x=rng.choice(["f32", "bf16"]), transpose=kind == "transpose")
    if op == "fp8":
        return dict(op=op, M=_size(rng, 1, 4096), K=_size(rng, 64, 4096), N=_size(rng, 64, 11008),
                    square=rng.random() < 0.6, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu"]), out=rng.choice(["f32", "bf16"]))
    if op == "experts":
        E = _size(rng, 2, 64)
        K, N = _size(rng, 64, 4096), _size(rng, 64, 2048)
        return dict(op=op, R=_size(rng, 1, 16384), K=K, N=N, E=E, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "relu", "gelu"]), out=rng.choice(["f32", "bf16"]))
    if op in ("route", "route_bwd"):
        groups = rng.choice([1, 1, 2, 4, 8])
        each = _size(rng, max(2, 8 // groups), 512 // groups)
        kept = rng.randint(1, groups)
        return dict(op=op, T=_size(rng, 1, 16384), E=groups * each,
                    k=rng.randint(1, min(12, kept * each)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, kept=kept, group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.7, x=rng.choice(["f32", "bf16"]),
                    pad=rng.choice([0, 0, 1, 7]))
    E = _size(rng, 8, 256)
    D = _size(rng, 64, 8192)
    k = rng.randint(1, 8)
    return dict(op=op, T=_size(rng, 1, min(8192, 4096 * 4096 * 8 // (D * k))), D=D, k=k, E=E,
                rows=rng.choice(["f32", "bf16"]), x=rng.random() < 0.5,
                out=rng.choice(["f32", "bf16"]), pad=rng.choice([0, 0, 1, 7]))


def work(case):
    c, op = case, case["op"]
    if op == "quantize":
        T, C, R = c["T"], c["C"], c["rows"]
        if R:  # rows that are picked are read once each
            return dict(bytes=min(T, R) * C * SIZE[c["x"]] + R * C + R * (-(-C // B) + 1) * 4,
                        flops=2 * R * C)
        runs = -(-T // B) * C if c["transpose"] else -(-C // B) * T
        return dict(bytes=T * C * (SIZE[c["x"]] + 1) + 4 * runs, flops=2 * T * C)
    if op == "fp8":
        M, K, N = c["M"], c["K"], c["N"]
        KB = -(-K // B)
        scales = 4 * KB * (M + (-(-N // B) if c["square"] else N))
        return dict(bytes=M * K + N * K + scales + SIZE[c["out"]] * M * N
                    + (4 * N if c["bias"] else 0), flops=2 * M * N * K)
    if op == "experts":
        R, K, N, E = c["R"], c["K"], c["N"], min(c["E"], c["R"])
        KB = -(-K // B)
        return dict(bytes=R * K + E * N * K + 4 * KB * (R + E * -(-N // B))
                    + SIZE[c["out"]] * R * N + (4 * E * N if c["bias"] else 0), flops=2 * R * N * K)
    if op in ("route", "route_bwd"):
        T, E, k = c["T"], c["E"], c["k"]
        if op == "route":
            return dict(bytes=T * E * SIZE[c["x"]] + 16 * T * k + 4 * (E + 1)
                        + (4 * E if c["bias"] else 0), flops=10 * T * E)
        return dict(bytes=2 * T * E * SIZE[c["x"]] + 8 * T * k, flops=10 * T * E)
    T, D, k = c["T"], c["D"], c["k"]
    rows = T * k * D * SIZE[c["rows"]]
    if op == "combine":
        return dict(bytes=rows + 8 * T * k + T * D * SIZE[c["out"]] * (2 if c["x"] else 1),
                    flops=2 * T * k * D)
    return dict(bytes=2 * rows + 12 * T * k + T * D * SIZE[c["out"]], flops=3 * T * k * D)


# ---------------------------------------------------------------- inputs

def _codes(values, scales):
    """8-bit codes (rows on 16 bytes) of values over scales that reach them."""
    r, c = values.shape[-2:]
    buf = torch.zeros((*values.shape[:-1], -(-c // B) * B), dtype=F8, device=values.device)
    buf[..., :c] = (values / scales).clamp(-448, 448).to(F8)
    return buf[..., :c]


def _row_scaled(v):
    """(codes, scales): a scale for each 128 values of a row, scales[k // 128, row]."""
    r, c = v.shape
    top = torch.nn.functional.pad(v, (0, -c % B)).view(r, -1, B).abs().amax(2)
    s = (top / 448.0).clamp(min=1e-12)
    return _codes(v, s.repeat_interleave(B, 1)[:, :c]), s.t().contiguous()


def _square_scaled(v):
    """(codes, scales): a scale for each 128 x 128 values, scales[..., row // 128, k // 128]."""
    r, c = v.shape[-2:]
    p = torch.nn.functional.pad(v, (0, -c % B, 0, -r % B))
    p = p.view(*v.shape[:-2], -(-r // B), B, -(-c // B), B)
    s = (p.abs().amax((-3, -1)) / 448.0).clamp(min=1e-12)
    full = s.repeat_interleave(B, -2).repeat_interleave(B, -1)[..., :r, :c]
    return _codes(v, full), s


def _sorted(index, E):
    """(slot, source, offsets) of chosen experts (T x k; -1: none): rows sorted by
    expert, then by token, then by choice."""
    T, k = index.shape
    key = torch.where(index < 0, E, index).reshape(-1).to(torch.int64)
    order = torch.sort(key, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=index.device)
    offsets[1:] = (key[:, None] == torch.arange(E, device=index.device)).sum(0).cumsum(0)
    at = torch.arange(T * k, device=index.device)
    slot = torch.empty_like(at)
    slot[order] = at
    slot = torch.where(key == E, -1, slot).view(T, k)
    source = torch.where(at < offsets[E], order // k, -1)
    i32 = torch.int32
    return slot.to(i32), source.to(i32), offsets.to(i32)


def _inputs(case, seed, dev):
    """The case's data, from the seed alone."""
    c, op = case, case["op"]
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=F32, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    s = dict(case)
    if op == "quantize":
        # columns of unlike sizes, as activations have them
        s["xs"] = (normal(c["T"], c["C"]) * torch.exp(normal(c["C"], scale=0.7))).to(DTYPES[c["x"]])
        s["index"] = torch.randint(0, c["T"], (c["rows"],), generator=g, device=dev,
                                   dtype=torch.int32) if c["rows"] else None
    elif op in ("fp8", "experts"):
        rows, K, N = c["M"] if op == "fp8" else c["R"], c["K"], c["N"]
        # activations: rows and channels of unlike sizes
        a = normal(rows, K) * torch.exp(normal(rows, 1, scale=0.5)) * torch.exp(normal(K, scale=0.5))
        s["a"], s["a_scales"] = _row_scaled(a)
        if op == "fp8":
            w = normal(N, K, scale=K ** -0.5)
            s["b"], s["b_scales"] = _square_scaled(w) if c["square"] else _row_scaled(w)
            s["bias_v"] = normal(N, scale=0.1) if c["bias"] else None
        else:
            E = c["E"]
            s["b"], s["b_scales"] = _square_scaled(normal(E, N, K, scale=K ** -0.5))
            s["bias_v"] = normal(E, N, scale=0.1) if c["bias"] else None
            # experts that are chosen more and less often
            p = torch.exp(normal(E, scale=0.5))
            of = torch.multinomial(p, rows, replacement=True, generator=g)
            n = (of[:, None] == torch.arange(E, device=dev)).sum(0)
            s["offsets"] = torch.nn.functional.pad(n.cumsum(0), (1, 0)).to(torch.int32)
            s["most"] = int(n.max())
    elif op in ("route", "route_bwd"):
        T, E = c["T"], c["E"]
        s["logits"] = (normal(T, E, scale=1.5) + normal(E, scale=0.3)).to(DTYPES[c["x"]])
        if op == "route" and c["pad"] < T:  # tokens behind the last sequence go to no expert
            s["logits"][T - c["pad"]:] = -math.inf
        s["bias_v"] = normal(E, scale=0.05) if c["bias"] else None
        if op == "route_bwd":
            # the experts that a forward pass chose
            pick = torch.rand((T, E), generator=g, device=dev) + s["logits"].float() * 0.1
            s["index"] = pick.topk(c["k"], 1).indices.to(torch.int32)
            s["d_weight"] = normal(T, c["k"])
    else:
        T, D, k, E = c["T"], c["D"], c["k"], c["E"]
        index = torch.rand((T, E), generator=g, device=dev).topk(k, 1).indices
        if c["pad"] < T:
            index[T - c["pad"]:] = -1
        s["slot"], _, _ = _sorted(index, E)
        s["rows_v"] = normal(T * k, D, dtype=DTYPES[c["rows"]])
        w = torch.rand((T, k), generator=g, device=dev) + 0.1
        s["weight"] = w / w.sum(1, keepdim=True)
        if op == "combine":
            s["xs"] = normal(T, D, dtype=DTYPES[c["out"]]) if c["x"] else None
        else:
            s["d_out"] = normal(T, D, dtype=DTYPES[c["out"]])
            s["d_rows"] = torch.zeros_like(s["rows_v"])  # rows of no token stay as they are
    return s


def prepare(case, seed):
    return _inputs(case, seed, "cuda")


# ------------------------------------------------------------ plain forms

def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == "gelu":
        return v * 0.5 * (1.0 + torch.erf(v * math.sqrt(0.5)))
    return v


def _quantize(v):
    """(codes, scales) of each 128 values of a row: the scale is the smallest power of
    two (at least 2^-126) that brings them to 448 at most."""
    r, c = v.shape
    p = torch.nn.functional.pad(v.float(), (0, -c % B)).view(r, -1, B)
    top = p.abs().amax(2)
    m, e = torch.frexp(top)
    e = (e.to(torch.int32) - 9 + (m > 448.0 / 512.0).to(torch.int32)).clamp(min=-126)
    up, down = ((127 + e) << 23).view(F32), ((127 - e) << 23).view(F32)
    return (p * down[..., None]).to(F8).view(r, -1)[:, :c], up.t()


def _values(codes, scales, square):
    r, c = codes.shape[-2:]
    if square:
        full = scales.repeat_interleave(B, -2).repeat_interleave(B, -1)[..., :r, :c]
    else:
        full = scales.t().repeat_interleave(B, 1)[:, :c]
    return codes.float() * full


def _choose(s):
    """Index of the experts of each token (-1: none), from 64-bit scores."""
    l, E, k, G = s["logits"].double(), s["E"], s["k"], s["groups"]
    open_ = l > -math.inf
    p = torch.softmax(l, 1) if s["score"] == "softmax" else torch.sigmoid(l)
    v = p if s["bias_v"] is None else p + s["bias_v"].double()
    v = torch.where(open_, v, -math.inf)
    if s["kept"] < G:
        best = v.view(-1, G, E // G).sort(dim=2, descending=True).values[:, :, :s["group_top"]]
        top = best[:, :, 0] + torch.where(best > -math.inf, best, 0.0)[:, :, 1:].sum(2)
        order = top.sort(dim=1, descending=True, stable=True).indices[:, :s["kept"]]
        keep = torch.zeros_like(top, dtype=torch.bool).scatter_(1, order, True)
        v = torch.where(keep.repeat_interleave(E // G, 1), v, -math.inf)
    best, index = v.sort(dim=1, descending=True, stable=True)
    return torch.where(best > -math.inf, index, -1)[:, :k]


def _plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["xs"]
        if s["index"] is not None:
            x = x[s["index"].to(torch.int64)]
        codes, scales = _quantize(x.t() if s["transpose"] else x)
        return {"codes": codes, "scales": scales}
    if op == "fp8":
        v = _values(s["a"], s["a_scales"], False) @ _values(s["b"], s["b_scales"], s["square"]).t()
        if s["bias_v"] is not None:
            v = v + s["bias_v"]
        return _act(v, s["act"]).to(DTYPES[s["out"]])
    if op == "experts":
        a, first, n = _values(s["a"], s["a_scales"], False), s["offsets"][:-1], s["offsets"].diff()
        at = torch.arange(s["most"], device=a.device)
        row = first[:, None] + torch.minimum(at[None], (n[:, None] - 1).clamp(min=0))
        row = row.clamp(max=s["R"] - 1).to(torch.int64)
        v = torch.bmm(a[row], _values(s["b"], s["b_scales"], True).transpose(1, 2))
        if s["bias_v"] is not None:
            v = v + s["bias_v"][:, None]
        r = torch.arange(s["R"], device=a.device)
        e = torch.searchsorted(s["offsets"].to(torch.int64), r, right=True) - 1
        return _act(v[e, r - first[e]], s["act"]).to(DTYPES[s["out"]])
    if op == "route":
        index = _choose(s)
        l = s["logits"].double()
        # (a token of no expert has a row of zeros)
        p = torch.softmax(l, 1).nan_to_num(0.0) if s["score"] == "softmax" else torch.sigmoid(l)
        w = torch.where(index < 0, 0.0, p.gather(1, index.clamp(min=0)))
        if s["renorm"]:
            t = w.sum(1, keepdim=True)
            w = torch.where(t > 0, w / t, 0.0)
        slot, source, offsets = _sorted(index, s["E"])
        return {"index": index.to(torch.int32), "weight": (w * 2.5).to(F32), "slot": slot,
                "source": source, "offsets": offsets}
    if op == "route_bwd":
        l, i, d = s["logits"].float(), s["index"].to(torch.int64), s["d_weight"] * 2.5
        p = torch.softmax(l, 1) if s["score"] == "softmax" else torch.sigmoid(l)
        q = p.gather(1, i)
        if s["renorm"]:
            t = q.sum(1, keepdim=True)
            d = (d - (d * q).sum(1, keepdim=True) / t) / t
        dp = torch.zeros_like(l).scatter_(1, i, d)
        if s["score"] == "softmax":
            return (p * (dp - (d * q).sum(1, keepdim=True))).to(s["logits"].dtype)
        return (dp * p * (1.0 - p)).to(s["logits"].dtype)
    slot, w = s["slot"].to(torch.int64), s["weight"]
    used = slot >= 0
    if op == "combine":
        v = s["rows_v"].float()[slot.clamp(min=0)] * torch.where(used, w, 0.0)[..., None]
        v = v.sum(1)
        if s["xs"] is not None:
            v = v + s["xs"].float()
        return v.to(DTYPES[s["out"]])
    d = s["d_out"].float()[:, None]
    d_rows = s["d_rows"].clone()
    d_rows[slot[used]] = (d * w[..., None])[used].to(d_rows.dtype)
    dw = (s["rows_v"].float()[slot.clamp(min=0)] * d).sum(2)
    return {"d_rows": d_rows, "d_weight": torch.where(used, dw, 0.0)}


def run(state):
    s = state
    if not own:
        return _plain(s)
    import dense_gemm_07_gb300 as g7
    op = s["op"]
    if op == "quantize":
        q = g7.gemm_fp8_quantize(s["xs"], index=s["index"], transpose=s["transpose"])
        return {"codes": q.codes, "scales": q.scales}
    if op == "fp8":
        return g7.gemm_fp8(g7.Fp8(s["a"], s["a_scales"]),
                           g7.Fp8(s["b"], s["b_scales"], square=s["square"]), bias=s["bias_v"],
                           activation=s["act"], out_dtype=DTYPES[s["out"]])
    if op == "experts":
        return g7.gemm_fp8_experts(g7.Fp8(s["a"], s["a_scales"]),
                                   g7.Fp8(s["b"], s["b_scales"], square=True), s["offsets"],
                                   bias=s["bias_v"], activation=s["act"],
                                   out_dtype=DTYPES[s["out"]])
    if op == "route":
        r = g7.gemm_route(s["logits"], s["k"], score=s["score"], bias=s["bias_v"],
                          groups=s["groups"], groups_kept=s["kept"], group_top=s["group_top"],
                          renormalize=s["renorm"], scale=2.5)
        return {"index": r.index, "weight": r.weight, "slot": r.slot, "source": r.source,
                "offsets": r.offsets}
    if op == "route_bwd":
        return g7.gemm_route_bwd(s["logits"], s["index"], s["d_weight"], score=s["score"],
                                 renormalize=s["renorm"], scale=2.5)
    if op == "combine":
        return g7.gemm_combine(s["rows_v"], s["slot"], s["weight"], x=s["xs"],
                               out_dtype=DTYPES[s["out"]])
    d_rows, d_weight = g7.gemm_combine_bwd(s["d_out"], s["rows_v"], s["slot"], s["weight"],
                                           d_rows=s["d_rows"])
    return {"d_rows": d_rows, "d_weight": d_weight}


# ---------------------------------------------------------------- 64 bits

def _values64(codes, scales, square):
    """Code times scale, block by block of the definition."""
    out = codes.double()
    for k in range(0, out.shape[-1], B):
        part = out[..., k:k + B]
        if square:
            for r in range(0, out.shape[-2], B):
                part[..., r:r + B, :] *= scales[..., r // B, k // B].double()[..., None, None]
        else:
            part *= scales[k // B].double()[:, None]
    return out


def _round8(v):
    """The nearest 8-bit floating-point number (4 exponent, 3 mantissa bits; ties to even)."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6)
    step = torch.exp2(e - 3.0)
    return torch.round(v / step) * step


def exact(case, seed):
    s = _inputs(case, seed, "cuda")
    op = s["op"]

    def act64(v, act):
        if act == "relu":
            return v.clamp(min=0.0)
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0)) if act == "gelu" else v

    if op == "quantize":
        x = s["xs"].double()
        if s["index"] is not None:
            x = x.index_select(0, s["index"].to(torch.int64))
        x = x.t() if s["transpose"] else x
        codes, scales = torch.empty_like(x), []
        for k in range(0, x.shape[1], B):
            top = x[:, k:k + B].abs().amax(1)
            scale = torch.exp2(torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0))
            # log2 may fall on the wrong side of a whole number: settle it exactly
            scale = torch.where(top > 448.0 * scale, scale * 2.0, scale)
            lower = (scale * 0.5).clamp(min=2.0 ** -126)
            scale = torch.where(top <= 448.0 * lower, lower, scale)
            codes[:, k:k + B] = _round8(x[:, k:k + B] / scale[:, None])
            scales.append(scale)
        return {"codes": codes, "scales": torch.stack(scales)}
    if op == "fp8":
        v = _values64(s["a"], s["a_scales"], False) @ _values64(s["b"], s["b_scales"], s["square"]).t()
        return act64(v if s["bias_v"] is None else v + s["bias_v"].double(), s["act"])
    if op == "experts":
        a, at = _values64(s["a"], s["a_scales"], False), s["offsets"].tolist()
        out = torch.empty((s["R"], s["N"]), dtype=torch.float64, device="cuda")
        for e in range(s["E"]):
            r = slice(at[e], at[e + 1])
            out[r] = a[r] @ _values64(s["b"][e], s["b_scales"][e], True).t()
            if s["bias_v"] is not None:
                out[r] += s["bias_v"][e].double()
        return act64(out, s["act"])
    if op == "route":
        l = s["logits"].double().cpu().numpy()
        T, E = l.shape
        G, k = s["groups"], s["k"]
        with np.errstate(all="ignore"):
            if s["score"] == "softmax":
                p = np.exp(l - l.max(1, keepdims=True))
                p = np.nan_to_num(p / p.sum(1, keepdims=True))
            else:
                p = 1.0 / (1.0 + np.exp(-l))
        v = p + (0.0 if s["bias_v"] is None else s["bias_v"].double().cpu().numpy())
        v[np.isneginf(l)] = -np.inf
        group = np.sort(v.reshape(T, G, E // G), axis=2)[:, :, ::-1]
        best = group[:, :, 0].copy()
        if s["group_top"] == 2:
            best += np.where(np.isneginf(group[:, :, 1]), 0.0, group[:, :, 1])
        worse = np.argsort(-best, axis=1, kind="stable")[:, s["kept"]:]
        shut = np.zeros((T, G), dtype=bool)
        np.put_along_axis(shut, worse, True, 1)
        v[np.repeat(shut, E // G, axis=1)] = -np.inf
        index = np.argsort(-v, axis=1, kind="stable")[:, :k]
        none = np.isneginf(np.take_along_axis(v, index, 1))
        w = np.where(none, 0.0, np.take_along_axis(p, index, 1))
        if s["renorm"]:
            w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
        index = np.where(none, -1, index)
        rows = [(e, t, j) for t, r in enumerate(index.tolist()) for j, e in enumerate(r) if e >= 0]
        rows.sort()
        slot, source = np.full((T, k), -1), np.full(T * k, -1)
        for n, (_, t, j) in enumerate(rows):
            slot[t, j], source[n] = n, t
        offsets = np.concatenate([[0], np.cumsum(np.bincount([r[0] for r in rows], minlength=E))])
        return {"index": index, "weight": 2.5 * w, "slot": slot, "source": source,
                "offsets": offsets}
    if op == "route_bwd":
        # the slope of each weight with respect to each logit, written out
        l, i, d = s["logits"].double(), s["index"].to(torch.int64), 2.5 * s["d_weight"].double()
        picked = torch.zeros_like(l).scatter_(1, i, 1.0)
        dd = torch.zeros_like(l).scatter_(1, i, d)
        if s["score"] == "softmax":
            e = torch.exp(l - l.amax(1, keepdim=True))
            if s["renorm"]:  # a softmax over the chosen ones
                e = e * picked
            p = e / e.sum(1, keepdim=True)
            return p * (dd - (dd * p).sum(1, keepdim=True))
        p = 1.0 / (1.0 + torch.exp(-l))
        if s["renorm"]:
            t = (p * picked).sum(1, keepdim=True)
            dd = picked * (dd / t - (dd * p).sum(1, keepdim=True) / t ** 2)
        return dd * p / (1.0 + torch.exp(l))
    w, slot = s["weight"].double(), s["slot"].to(torch.int64)
    rows = s["rows_v"].double()
    if op == "combine":
        out = torch.zeros((s["T"], s["D"]), dtype=torch.float64, device="cuda")
        if s["xs"] is not None:
            out += s["xs"].double()
        for j in range(s["k"]):
            on = slot[:, j] >= 0
            out[on] += w[on, j, None] * rows[slot[on, j]]
        return out
    d = s["d_out"].double()
    d_rows, d_weight = torch.zeros_like(rows), torch.zeros_like(w)
    for j in range(s["k"]):
        on = slot[:, j] >= 0
        d_rows[slot[on, j]] = w[on, j, None] * d[on]
        d_weight[on, j] = (rows[slot[on, j]] * d[on]).sum(1)
    return {"d_rows": d_rows, "d_weight": d_weight}
