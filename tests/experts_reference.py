"""Plain 64-bit forms of the 8-bit floating-point products and of a layer of experts
(torch double, any device), written from their definitions in include/gemm07.h; they
import nothing of the package."""
import math

import torch

BLOCK = 128


def e4m3_numbers():
    """The finite non-negative E4M3 numbers, by code."""
    out = []
    for code in range(127):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


def nearest_code(v):
    """Codes (uint8) of the nearest E4M3 numbers, ties to the even code; |v| <= 448."""
    table = e4m3_numbers().to(v.device)
    mag = v.abs().contiguous()
    hi = torch.searchsorted(table, mag).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = mag - table[lo], table[hi] - mag
    pick = torch.where(below < above, lo, torch.where(above < below, hi,
                                                      torch.where(lo % 2 == 0, lo, hi)))
    return pick + 128 * (torch.signbit(v)).to(pick.dtype)


def block_scale(top):
    """The smallest power of two (at least 2^-126) that brings `top` to 448 at most."""
    s = torch.full_like(top, 2.0 ** -126)
    for _ in range(260):
        s = torch.where(top > 448.0 * s, s * 2.0, s)
    return s


def quantize(x, square=False):
    """(codes uint8, scales) of x (R x K); codes of non-finite blocks are 0x7F."""
    x = x.double()
    R, K = x.shape
    codes = torch.zeros((R, K), dtype=torch.int64, device=x.device)
    KB, RB = -(-K // BLOCK), -(-R // BLOCK)
    scales = torch.zeros((RB, KB) if square else (KB, R), dtype=torch.float64, device=x.device)
    step = BLOCK if square else 1
    for k in range(0, K, BLOCK):
        if square:
            for r in range(0, R, step):
                part = x[r:r + step, k:k + BLOCK]
                if bool(torch.isfinite(part).all()):
                    s = block_scale(part.abs().max())
                    codes[r:r + step, k:k + BLOCK] = nearest_code(part / s)
                else:
                    s = torch.ones((), dtype=torch.float64)
                    codes[r:r + step, k:k + BLOCK] = 127
                scales[r // BLOCK, k // BLOCK] = s
        else:
            part = x[:, k:k + BLOCK]
            fine = torch.isfinite(part).all(1)
            s = torch.where(fine, block_scale(torch.where(fine, part.abs().amax(1), 1.0)), 1.0)
            q = nearest_code(torch.where(fine[:, None], part / s[:, None], 0.0))
            codes[:, k:k + BLOCK] = torch.where(fine[:, None], q, 127)
            scales[k // BLOCK] = s
    return codes.to(torch.uint8), scales


def values(codes, scales, square):
    """What codes and scales stand for (R x K, or E x R x K with square)."""
    v = codes.double()
    R, K = v.shape[-2:]
    s = scales.double()
    if square:
        return v * s.repeat_interleave(BLOCK, -2).repeat_interleave(BLOCK, -1)[..., :R, :K]
    return v * s.t().repeat_interleave(BLOCK, 1)[:, :K]


def route(logits, k, score="softmax", bias=None, groups=1, groups_kept=None, group_top=2,
          renormalize=True, scale=1.0):
    """(index, weight, slot, source, offsets), token by token of the definition."""
    kept = groups if groups_kept is None else groups_kept
    l = logits.double().cpu()
    T, E = l.shape
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double().cpu()
    index = torch.full((T, k), -1, dtype=torch.int32)
    weight = torch.zeros((T, k), dtype=torch.float64)
    inf = math.inf
    for t in range(T):
        row = l[t]
        if bool(row.isnan().any()) or (score == "softmax" and float(row.max()) == inf):
            weight[t] = math.nan
            continue
        if float(row.max()) == -inf:
            continue
        s = torch.softmax(row, 0) if score == "softmax" else torch.sigmoid(row)
        v = (s + b).tolist()
        order = row.tolist() if bias is None else v  # without a bias the logits decide
        open_ = [e for e in range(E) if float(row[e]) > -inf and v[e] > -inf]
        if kept < groups:
            size = E // groups
            sums = []
            for g in range(groups):
                best = sorted((v[e] for e in open_ if e // size == g), reverse=True)[:group_top]
                sums.append(sum(best) if best else -inf)
            chosen = sorted(range(groups), key=lambda g: (-sums[g], g))[:kept]
            open_ = [e for e in open_ if e // size in chosen]
        picks = sorted(open_, key=lambda e: (-order[e], e))[:k]
        w = s[picks]
        if renormalize:
            total = float(w.sum())
            w = w / total if total > 0 else w * 0
        index[t, :len(picks)] = torch.tensor(picks, dtype=torch.int32)
        weight[t, :len(picks)] = w * scale
    slot, source, offsets = sort_pairs(index, E)
    return index, weight, slot, source, offsets


def sort_pairs(index, E):
    T, k = index.shape
    pairs = sorted((e, t, j) for t, r in enumerate(index.tolist()) for j, e in enumerate(r) if e >= 0)
    slot = torch.full((T, k), -1, dtype=torch.int32)
    source = torch.full((T * k,), -1, dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32)
    for n, (e, t, j) in enumerate(pairs):
        slot[t, j] = n
        source[n] = t
        offsets[e + 1:] += 1
    return slot, source, offsets


def route_weights(logits, index, score, renormalize, scale):
    """The weights as a differentiable function of the logits (index >= 0)."""
    s = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    w = s.gather(1, index)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    return scale * w


def route_grad(logits, index, d_weight, score, renormalize, scale):
    """(d_logits, the magnitudes that its error goes by), from the formula."""
    l, d = logits.double(), d_weight.double() * scale
    T, E = l.shape
    on = (index >= 0) & (index < E)
    at = torch.where(on, index, 0).to(torch.int64)
    d = torch.where(on, d, 0.0)
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    q = torch.where(on, s.gather(1, at), 0.0)
    if renormalize:
        total = q.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        ds = (d - (d * q).sum(1, keepdim=True) / total) / total
        size = (d.abs() + (d * q).abs().sum(1, keepdim=True) / total) / total
    else:
        ds, size = d, d.abs()
    ds, size = torch.where(on, ds, 0.0), torch.where(on, size, 0.0)
    full = torch.zeros_like(l).scatter_add_(1, at, ds)
    mag = torch.zeros_like(l).scatter_add_(1, at, size)
    if score == "sigmoid":
        return full * s * (1 - s), mag * s * (1 - s)
    rest = (ds * q).sum(1, keepdim=True), (size * q).sum(1, keepdim=True)
    return s * (full - rest[0]), s * (mag + rest[1])


def combine(rows, slot, weight, x=None):
    """(out, the magnitudes that its error goes by)."""
    R = rows.shape[0]
    on = (slot >= 0) & (slot < R)
    at = torch.where(on, slot, 0).to(torch.int64)
    w = weight.double()
    if R:
        part = torch.where(on[..., None], rows.double()[at], 0.0) * w[..., None]
    else:
        part = torch.zeros((*slot.shape, rows.shape[1]), dtype=torch.float64,
                           device=rows.device) * w[..., None]
    out, size = part.sum(1), part.abs().sum(1)
    if x is not None:
        out, size = out + x.double(), size + x.double().abs()
    return out, size


def combine_grad(d_out, rows, slot, weight, d_rows):
    """(d_rows, d_weight, magnitudes of d_weight); d_rows: what was there before."""
    R = rows.shape[0]
    d_rows = d_rows.double().clone()
    on = (slot >= 0) & (slot < R)
    d = d_out.double()[:, None]
    at = torch.where(on, slot, 0).to(torch.int64)
    d_rows[slot[on].to(torch.int64)] = (d * weight.double()[..., None])[on]
    part = torch.where(on[..., None], rows.double()[at], 0.0) * d
    return d_rows, part.sum(2), part.abs().sum(2)
