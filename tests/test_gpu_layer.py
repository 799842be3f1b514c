"""The layer operators (4-bit weights, gated norms, 8-bit checkpoints) against
their plain 64-bit forms, at the sizes, strides, types and values where they can
go wrong.

Tolerances.  EPS32 = 2^-23 is one unit of FP32, the loss of one truncated or
rounded operation relative to the magnitudes it adds; BF16 outputs add half a
unit of BF16, 2^-9 of the value (2^-8 allowed).
"""
import itertools

import pytest
import torch

import dense_gemm_07_gb300 as g7
from dense_gemm_07_gb300 import _abi
from layer_reference import (EPS32, Norm, act, act_slope, kept, w4_layout_decode, w4_weights)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
ROUND = {F32: EPS32, BF16: 2.0 ** -8}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _strided(t, extra):
    """The same values in rows `extra` elements further apart, off by one element
    when extra is odd; the gaps hold NaN."""
    r, c = t.shape
    fill = float("nan") if t.is_floating_point() else 255
    buf = torch.full((r * (c + extra) + extra + 1,), fill, dtype=t.dtype, device=t.device)
    v = buf[extra % 2:][: r * (c + extra)].view(r, c + extra)[:, :c]
    v.copy_(t)
    return v


def _close(got, want, tol, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
        f"{float(((got - want).abs() / tol.clamp(min=1e-300)).nan_to_num(9e9).max()):.3g} of the bound")


# ---------------------------------------------------------------- 4-bit weights

def _w4_case(seed, M, K, N, group, zeros):
    g = _gen(seed)
    G = -(-K // group)
    a = _randn(g, M, K, dtype=BF16)
    codes = torch.randint(0, 16, (K, N), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand((G, N), generator=g, device="cuda") + 0.1).to(BF16)
    z = torch.randint(0, 16, (G, N), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return a, codes, scales, z


def _w4_tol(a, w, K, group, out):
    """A group's tensor-core sum loses at most one unit in each of its group / 16
    steps (two products each) and one per product group inside a step; the scaled
    sums of the groups and of at most 64 partial sums add one each."""
    steps = group // 16 * 4 + -(-K // group) + 64
    return steps * EPS32 * (a.double().abs() @ w.abs()) + ROUND[out.dtype] * 2 * out.double().abs() \
        + 1e-30


W4_SHAPES = [(1, 1, 1), (1, 128, 16), (1, 4096, 4096), (2, 127, 17), (3, 129, 15), (7, 3001, 1000),
             (8, 512, 100), (9, 640, 33), (16, 1024, 2048), (16, 130, 260), (17, 300, 40),
             (40, 257, 129), (5, 11008, 512), (16, 8192, 64), (4, 32, 5000)]


@pytest.mark.parametrize("M,K,N", W4_SHAPES)
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
def test_w4(M, K, N, group, zeros):
    a, codes, scales, z = _w4_case(M * 7 + K, M, K, N, group, zeros)
    packed = g7.w4_pack(codes)
    assert torch.equal(w4_layout_decode(packed, K, N), codes.cpu())
    w = w4_weights(codes, scales, z, group)
    out = g7.gemm_w4(a, packed, scales, zeros=z, group=group)
    _close(out, a.double() @ w, _w4_tol(a, w, K, group, out), "product")
    again = g7.gemm_w4(a, packed, scales, zeros=z, group=group)
    assert torch.equal(out, again)


@pytest.mark.parametrize("M,K,N", [(1, 515, 77), (6, 1031, 130), (16, 384, 256)])
@pytest.mark.parametrize("act_kind", ["none", "relu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_w4_epilogue_and_strides(M, K, N, act_kind, dtype):
    group = 64
    a, codes, scales, z = _w4_case(5, M, K, N, group, True)
    g = _gen(6)
    bias, old = _randn(g, N), _randn(g, M, N, dtype=dtype)
    out = _strided(old, 3)
    w = w4_weights(codes, scales, z, group)
    got = g7.gemm_w4(_strided(a, 5), g7.w4_pack(_strided(codes, 7)), _strided(scales, 1),
                     zeros=_strided(z, 9), group=group, out=out, alpha=0.5, beta=-2.0, bias=bias,
                     activation=act_kind)
    v = 0.5 * (a.double() @ w) - 2.0 * old.double() + bias.double()
    tol = 0.5 * _w4_tol(a, w, K, group, torch.zeros((), dtype=F32)) \
        + 4 * EPS32 * (2 * old.double().abs() + bias.double().abs() + v.abs())
    want = act(v, act_kind)
    _close(got, want, 1.13 * tol + 4 * EPS32 * v.abs() + ROUND[dtype] * want.abs(), act_kind)


def test_w4_guard_band_and_dirty_padding():
    """Codes past K and N may hold anything; nothing outside C is written."""
    M, K, N = 3, 200, 21
    a, codes, scales, z = _w4_case(1, M, K, N, 32, True)
    packed = g7.w4_pack(codes)
    clean = g7.gemm_w4(a, packed, scales, zeros=z, group=32)
    full = torch.randint(0, 256, packed.shape, dtype=torch.uint8, device="cuda")
    big = torch.randint(0, 16, (256, 32), dtype=torch.uint8, device="cuda")
    big[:K, :N] = codes
    full = g7.w4_pack(big)
    assert full.shape == packed.shape and not torch.equal(full, packed)
    guard = torch.full((M + 2, N + 8), 7.0, device="cuda")
    out = guard[1:M + 1, 4:4 + N]
    g7.gemm_w4(a, full, scales, zeros=z, group=32, out=out)
    assert torch.equal(out, clean)
    guard[1:M + 1, 4:4 + N] = 7.0
    assert bool((guard == 7.0).all())


def test_w4_non_finite_values_stay_in_their_rows_and_columns():
    M, K, N = 4, 300, 50
    a, codes, scales, z = _w4_case(2, M, K, N, 64, False)
    a[1, 7] = float("nan")
    a[2, 299] = float("inf")
    scales[1, 9] = float("nan")
    out = g7.gemm_w4(a, g7.w4_pack(codes), scales, group=64)
    assert bool(out[1].isnan().all()) and bool(out[:, 9].isnan().all())
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[1:3] = False
    rest[:, 9] = False
    assert bool(out[rest].isfinite().all())
    assert not bool(out[2].isfinite().any())


def test_w4_empty_sizes():
    scales = torch.empty((0, 5), dtype=BF16, device="cuda")
    packed = g7.w4_pack(torch.empty((0, 5), dtype=torch.uint8, device="cuda"))
    bias = torch.arange(5.0, device="cuda") - 2
    out = g7.gemm_w4(torch.empty((3, 0), dtype=BF16, device="cuda"), packed, scales, bias=bias,
                     activation="relu")
    assert torch.equal(out, bias.clamp(min=0).expand(3, 5))
    a, codes, scales, _ = _w4_case(3, 2, 64, 8, 64, False)
    assert g7.gemm_w4(a[:0], g7.w4_pack(codes), scales, group=64).shape == (0, 8)


@pytest.mark.parametrize("K,N,group", [(1, 1, 32), (128, 16, 128), (300, 45, 32), (1000, 129, 64)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("symmetric", [True, False])
def test_w4_quantize_and_unpack(K, N, group, dtype, symmetric):
    b = _randn(_gen(K), K, N, dtype=dtype)
    b[:, 0] = 0.0
    packed, scales, zeros = g7.w4_quantize(_strided(b, 3), group=group, symmetric=symmetric)
    codes = w4_layout_decode(packed, K, N).cuda()
    w = w4_weights(codes, scales, zeros, group)
    got = g7.w4_unpack(packed, scales, zeros, group=group, K=K)
    assert torch.equal(got, w.to(BF16))
    # the nearest code is at most half a step off; the scale's rounding to BF16
    # (2^-9) moves the ends of the range by 15 codes * 2^-9, and a zero point
    # rounded to a whole code can clip up to half a step more
    step = scales.double()[torch.arange(K, device="cuda") // group]
    room = 0.5 + 15 * 2.0 ** -9 + (0.0 if symmetric else 0.5)
    assert bool(((w - b.double()).abs() <= room * step + 1e-30).all())
    assert bool((w[:, 0] == 0).all())
    # a group with a value that is not finite is NaN, the others are untouched
    b[K // 2, N - 1] = float("inf")
    p2, s2, z2 = g7.w4_quantize(b, group=group, symmetric=symmetric)
    u2 = g7.w4_unpack(p2, s2, z2, group=group, K=K)
    lo = K // 2 // group * group
    assert bool(u2[lo:lo + group, N - 1].isnan().all())
    u2[lo:lo + group, N - 1] = got[lo:lo + group, N - 1]
    if N > 1:
        assert torch.equal(u2, got)


# ------------------------------------------------------------------- norms

def _norm_case(seed, T, D, xt, yt, gate, post=True, pre=True, y=True, spread=True):
    g = _gen(seed)
    rows = torch.exp(_randn(g, T, 1)) if spread else 1.0
    c = dict(x=(_randn(g, T, D) * rows).to(xt), y=None, weight_post=None, gate=None,
             weight_pre=None)
    if y:
        c["y"] = (_randn(g, T, D) * 3).to(yt)
        c["weight_post"] = 1.0 + _randn(g, D, scale=0.2) if post else None
        shape = {"none": None, "channel": (D,), "row": (T, 1), "full": (T, D)}[gate]
        c["gate"] = None if shape is None else _randn(g, *shape)
    if pre:
        c["weight_pre"] = 1.0 + _randn(g, D, scale=0.2)
    return c


def _norm_ref(c, alpha, eps):
    return Norm(c["x"], c["y"], c["weight_post"], c["gate"], c["weight_pre"], alpha, eps)


def _norm_tols(ref, D, xt):
    """A mean over D terms in FP32, summed by at most 512 threads in runs of at
    most 32, then over 5 shuffles and 16 warps: 64 units, halved by the root but
    allowed whole; 16 more for the products around it."""
    n = 80 * EPS32
    tol_u = n * ref.u_size
    tol_h = None
    if ref.h is not None:
        tol_h = 2 * n * ref.u_size * ref.r1 * ref.w_pre.abs() * (1 + ref.u_size.mean(1, keepdim=True) * ref.r1) \
            + 2.0 ** -8 * ref.h.abs()
    return tol_u + ROUND[xt] * ref.u.abs(), tol_h


NORM_SHAPES = [(1, 1), (1, 64), (3, 8), (5, 100), (33, 1000), (17, 1024), (300, 256), (9, 3001),
               (7, 4096), (64, 4104), (3, 5001), (5, 8192), (2, 8200), (3, 16384), (2, 16383)]


@pytest.mark.parametrize("T,D", NORM_SHAPES)
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_norm_gate(T, D, xt, yt, gate):
    c = _norm_case(T * D, T, D, xt, yt, gate)
    ref = _norm_ref(c, 0.75, 1e-5)
    x_out, h = g7.gemm_norm_gate(**c, residual_scale=0.75, eps=1e-5)
    assert x_out.dtype == xt and h.dtype == BF16
    tu, th = _norm_tols(ref, D, xt)
    _close(x_out, ref.u, tu, "x_out")
    _close(h, ref.h, th, "h")


@pytest.mark.parametrize("post,pre,y", [(False, True, True), (True, False, True),
                                        (False, False, True), (False, True, False),
                                        (False, False, False)])
@pytest.mark.parametrize("D", [77, 2048])
def test_norm_gate_parts(post, pre, y, D):
    """Any of the norms, the gate and the block's output may be missing."""
    T = 301
    c = _norm_case(9, T, D, F32, BF16, "channel" if y else "none", post, pre, y)
    ref = _norm_ref(c, -1.5, 1e-6)
    x_out, h = g7.gemm_norm_gate(**c, residual_scale=-1.5)
    tu, th = _norm_tols(ref, D, F32)
    _close(x_out, ref.u, tu, "x_out")
    assert (h is None) == (not pre)
    if pre:
        _close(h, ref.h, th, "h")
    g = _gen(10)
    dxo = _randn(g, T, D)
    dh = _randn(g, T, D, dtype=BF16) if pre else None
    _check_grads(g7.gemm_norm_gate_bwd(**c, d_x_out=dxo, d_h=dh, residual_scale=-1.5), ref, dxo,
                 dh, F32, D)


def _check_grads(got, ref, dxo, dh, xt, D):
    want, size = ref.backward(dxo, dh)
    n = 4 * 80 * EPS32  # two more means on top of the forward's
    T = ref.x.shape[0]
    # a column's sum adds at most T / slots + slots / 8 + 8 terms in a chain
    col = n + (T + 16) * EPS32
    for name, field, round_, units in (("dx", got.dx, ROUND[xt], n), ("dy", got.dy, 2.0 ** -8, n),
                                       ("dw_post", got.dweight_post, 0, col),
                                       ("dw_pre", got.dweight_pre, 0, col),
                                       ("dgate", got.dgate, 0, col)):
        w = want.get(name)
        assert (field is None) == (w is None), name
        if w is not None:
            _close(field, w, units * size[name] + round_ * w.abs() + 1e-30, name)


@pytest.mark.parametrize("T,D", NORM_SHAPES + [(1000, 72), (400, 4096), (1300, 4000), (1300, 2999), (9000, 40), (700, 8192),
                                               (500, 6001), (400, 16384)])
@pytest.mark.parametrize("xt,yt,ht", [(F32, F32, F32), (BF16, F32, F32), (BF16, BF16, BF16),
                                      (F32, BF16, BF16)])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_norm_gate_bwd(T, D, xt, yt, ht, gate):
    c = _norm_case(T + D, T, D, xt, yt, gate)
    g = _gen(4)
    dxo, dh = _randn(g, T, D, dtype=xt), _randn(g, T, D, dtype=ht)
    ref = _norm_ref(c, 0.75, 1e-5)
    got = g7.gemm_norm_gate_bwd(**c, d_x_out=dxo, d_h=dh, residual_scale=0.75, eps=1e-5)
    _check_grads(got, ref, dxo, dh, xt, D)
    again = g7.gemm_norm_gate_bwd(**c, d_x_out=dxo, d_h=dh, residual_scale=0.75, eps=1e-5)
    assert all(torch.equal(a, b) for a, b in zip(got, again) if a is not None)


def test_norm_gate_strides_and_in_place():
    T, D = 21, 640
    for extra in (8, 3):
        c = _norm_case(3, T, D, BF16, F32, "full")
        plain = g7.gemm_norm_gate(**c)
        s = dict(c, x=_strided(c["x"], extra), y=_strided(c["y"], extra))
        x_out, h = g7.gemm_norm_gate(**s, x_out=s["x"],
                                     h=torch.empty((T, D + extra), dtype=BF16, device="cuda")[:, :D])
        assert x_out is s["x"]
        tol = 2.0 ** -7 * plain[0].double().abs() + 1e-6
        _close(x_out, plain[0].double(), tol)
        _close(h, plain[1].double(), 2.0 ** -7 * plain[1].double().abs() + 1e-6)


def test_norm_gate_rows_of_zeros_and_of_huge_values():
    T, D = 6, 512
    c = _norm_case(8, T, D, F32, F32, "none", spread=False)
    c["x"][0] = 0
    c["y"][0] = 0
    c["y"][1] = 0
    c["x"][2, 5] = float("nan")
    c["y"][3, 0] = float("inf")
    x_out, h = g7.gemm_norm_gate(**c)
    assert bool((h[0] == 0).all()) and bool((x_out[0] == 0).all())
    assert torch.equal(x_out[1], c["x"][1])
    assert bool(h[2].isnan().all()) and bool(x_out[2].isnan().sum() == 1)
    assert bool(x_out[3, 0].isnan())
    assert bool(x_out[4:].isfinite().all()) and bool(h[4:].isfinite().all())
    dh = torch.ones(T, D, device="cuda")
    d = g7.gemm_norm_gate_bwd(**c, d_x_out=dh, d_h=dh)
    for r in (0, 1, 4, 5):
        assert bool(d.dx[r].isfinite().all()) and bool(d.dy[r].isfinite().all())


def test_norm_gate_no_rows():
    c = _norm_case(8, 4, 24, F32, F32, "channel")
    e = dict(c, x=c["x"][:0], y=c["y"][:0])
    x_out, h = g7.gemm_norm_gate(**e)
    assert x_out.shape == (0, 24) and h.shape == (0, 24)
    d = g7.gemm_norm_gate_bwd(**e, d_x_out=x_out, d_h=x_out)
    for v in (d.dweight_post, d.dweight_pre, d.dgate):
        assert bool((v == 0).all())


def test_norm_gate_bwd_against_differences():
    """The gradient of sum(x_out * c) by central differences of the kernel itself
    (all FP32).  A step of 2^-6 leaves a cubic term of about step^2 / 6 of the
    third derivative (values near 1: 1e-4 allowed 1e-3) and a rounding of
    2^-24 * |loss terms| / step."""
    T, D, step = 3, 40, 2.0 ** -6
    c = _norm_case(12, T, D, F32, F32, "full", pre=False, spread=False)
    w = _randn(_gen(13), T, D)
    d = g7.gemm_norm_gate_bwd(**c, d_x_out=w)

    def loss(**new):
        return (g7.gemm_norm_gate(**dict(c, **new))[0].double() * w.double()).sum()

    for name, grad in (("y", d.dy), ("gate", d.dgate), ("weight_post", d.dweight_post), ("x", d.dx)):
        flat = c[name].reshape(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 20)):
            hi, lo = flat.clone(), flat.clone()
            hi[i] += step
            lo[i] -= step
            two = float((hi[i] - lo[i]).double())
            num = float(loss(**{name: hi.view_as(c[name])}) - loss(**{name: lo.view_as(c[name])})) / two
            have = float(grad.reshape(-1)[i])
            assert abs(num - have) <= 2.0 ** -8 * abs(have) + 2e-3, (name, i, num, have)


# ------------------------------------------------------------- checkpoints

CKPT_SHAPES = [(1, 1), (31, 3), (32, 128), (33, 129), (64, 256), (127, 1000), (200, 515), (1025, 64)]


def _ckpt_values(seed, T, N, dtype):
    g = _gen(seed)
    x = _randn(g, T, N) * torch.exp(3 * _randn(g, 1, N))
    if N > 2:
        x[:, 1] = 0.0
        x[:, 2] *= 1e-38  # runs below the smallest step's reach
    return x.to(dtype)


@pytest.mark.parametrize("T,N", CKPT_SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ckpt8_values(T, N, dtype):
    x = _ckpt_values(T + N, T, N, dtype)
    want = kept(x)
    for extra in (0, 1, 8):
        k = g7.gemm_ckpt8_pack(_strided(x, extra) if extra else x)
        for out in (F32, BF16):
            assert torch.equal(g7.gemm_ckpt8_unpack(k, out).double(), want)
    # the layout: row t, column n at ((t / 16) N + n) 16 + t % 16, zeros past T
    q = k.q.view(torch.int8).view(-1, N, 16).permute(0, 2, 1).reshape(-1, N).double()
    assert bool((q[T:] == 0).all())
    e = k.scales.double().repeat_interleave(32, 0) - 127
    assert torch.equal((q * torch.exp2(e))[:T], want)


def test_ckpt8_step_at_its_edges():
    """The largest magnitude just below, at and above 127 steps, ties, the
    smallest and largest finite numbers, and values that are not finite."""
    big = torch.finfo(F32).max
    tops = [127.0, 127.00001, 126.99999, 128.0, 1.984375, 1.9843751, 2.0 ** -126, 2.0 ** -140,
            127 * 2.0 ** -126, 128 * 2.0 ** -126, big, 63.5, 1.0]
    x = torch.zeros((64, len(tops) + 3), device="cuda")
    x[5, :len(tops)] = torch.tensor(tops, device="cuda")
    x[6, :len(tops)] = -0.5 * x[5, :len(tops)]
    x[7, 0], x[8, 0], x[9, 0] = 0.5, 1.5, -2.5  # ties at step 1
    x[40, len(tops)] = float("nan")
    x[40, len(tops) + 1] = float("inf")
    x[3, len(tops) + 2] = -float("inf")
    k = g7.gemm_ckpt8_pack(x)
    got, want = g7.gemm_ckpt8_unpack(k, F32).double(), kept(x)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))
    assert [float(v) for v in got[7:10, 0]] == [0.0, 2.0, -2.0]
    assert int(got.isnan().sum()) == 96


@pytest.mark.parametrize("T,N", CKPT_SHAPES)
@pytest.mark.parametrize("kind", ["none", "relu", "gelu"])
@pytest.mark.parametrize("zt,gt", [(F32, F32), (BF16, F32), (F32, BF16)])
def test_ckpt8_activation_and_gradient(T, N, kind, zt, gt):
    g = _gen(T * N)
    z, grad = _randn(g, T, N, scale=2.0, dtype=zt), _randn(g, T, N, dtype=gt)
    k, a = g7.gemm_ckpt8_pack(_strided(z, 3), activation=kind)
    assert torch.equal(g7.gemm_ckpt8_unpack(k, F32).double(), kept(z))
    want = act(z.double(), kind)
    # FP32 GELU: 1 + erf loses up to 4 units of 1, times |z| / 2
    _close(a, want, 2.0 ** -8 * want.abs() + 4 * EPS32 * z.double().abs(), "act")
    dz, db = g7.gemm_ckpt8_act_grad(_strided(grad, 5), k, kind)
    wz = grad.double() * act_slope(kept(z), kind)
    # the slope is at most 1.13 and its parts lose a few units of their size
    slack = 16 * EPS32 * grad.double().abs()
    _close(dz, wz, 2.0 ** -8 * wz.abs() + slack, "dz")
    _close(db, wz.sum(0), slack.sum(0) + (T + 16) * EPS32 * wz.abs().sum(0) + 1e-30, "dbias")
    dz2, none = g7.gemm_ckpt8_act_grad(grad, k, kind, bias_grad=False)
    assert none is None and torch.equal(dz2, dz)


def test_ckpt8_gelu_slope_against_differences():
    """act'(kept z) against central differences of the activation in 64 bits at the
    values kept: step 2^-10, cubic term below 1e-6."""
    z = torch.linspace(-6, 6, 32 * 25, device="cuda").view(32, 25)
    k, _ = g7.gemm_ckpt8_pack(z, activation="gelu")
    dz, _ = g7.gemm_ckpt8_act_grad(torch.ones_like(z), k, "gelu")
    v, h = kept(z), 2.0 ** -10
    num = (act(v + h, "gelu") - act(v - h, "gelu")) / (2 * h)
    _close(dz, num, 2.0 ** -8 * num.abs() + 1e-5)


WGRAD_SHAPES = [(1, 1, 1), (1, 130, 64), (31, 17, 9), (32, 128, 128), (65, 127, 129), (127, 127, 1000),
                (128, 256, 256), (300, 257, 264), (512, 100, 72), (1000, 513, 520), (2049, 300, 200),
                (700, 1000, 1001), (4096, 128, 256), (96, 2048, 640)]


@pytest.mark.parametrize("T,K,N", WGRAD_SHAPES)
def test_ckpt8_wgrad_exact_on_whole_numbers(T, K, N):
    """Whole numbers up to 127 with a 127 in every run are kept exactly (step 1), and
    their products with small whole numbers sum below 2^24: the gradient is exact."""
    g = _gen(T)
    x = torch.randint(-8, 9, (T, K), generator=g, device="cuda").float()
    x[::32] = torch.where(torch.rand((len(x[::32]), K), generator=g, device="cuda") < 0.5, 127.0, -127.0)
    dy = torch.randint(-3, 4, (T, N), generator=g, device="cuda").to(BF16)
    k = g7.gemm_ckpt8_pack(x)
    want = x.double().t() @ dy.double()
    assert torch.equal(g7.gemm_ckpt8_wgrad(k, dy).double(), want)
    guard = torch.full((K + 2, N + 5), 3.0, device="cuda")
    out = guard[1:K + 1, 2:N + 2]
    g7.gemm_ckpt8_wgrad(k, _strided(dy, 3), out=out, beta=-2.0)
    assert torch.equal(out.double(), want - 6.0)
    guard[1:K + 1, 2:N + 2] = 3.0
    assert bool((guard == 3.0).all())


@pytest.mark.parametrize("T,K,N", WGRAD_SHAPES + [(5000, 384, 512)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ckpt8_wgrad(T, K, N, dtype):
    x = _ckpt_values(T, T, K, dtype)
    dy = _randn(_gen(K), T, N, dtype=BF16)
    k = g7.gemm_ckpt8_pack(x)
    v = kept(x)
    got = g7.gemm_ckpt8_wgrad(k, dy)
    # tensor-core sums of at most 512 rows (32 steps, two units each) and one unit
    # for each of the T / 512 sums added in FP32
    units = 64 + 2 * (T // 512 + 2)
    _close(got, v.t() @ dy.double(), units * EPS32 * (v.abs().t() @ dy.double().abs()) + 1e-37)
    assert torch.equal(got, g7.gemm_ckpt8_wgrad(k, dy))


def test_ckpt8_wgrad_non_finite_runs_and_no_rows():
    T, K, N = 100, 140, 136
    x = _randn(_gen(1), T, K)
    x[40, 3] = float("nan")
    dy = _randn(_gen(2), T, N, dtype=BF16)
    out = g7.gemm_ckpt8_wgrad(g7.gemm_ckpt8_pack(x), dy)
    assert bool(out[3].isnan().all())
    out[3] = 0
    assert bool(out.isfinite().all())
    e = g7.gemm_ckpt8_pack(x[:0])
    old = _randn(_gen(3), K, N)
    assert torch.equal(g7.gemm_ckpt8_wgrad(e, dy[:0], out=old.clone(), beta=0.5), old * 0.5)
    assert bool((g7.gemm_ckpt8_wgrad(e, dy[:0]) == 0).all())
    dz, db = g7.gemm_ckpt8_act_grad(x[:0], e, "gelu")
    assert dz.shape == (0, K) and bool((db == 0).all())


# ----------------------------------------------- streams, graphs, refusals

def _all_ops(seed):
    a, codes, scales, z = _w4_case(seed, 3, 700, 200, 32, True)
    n = _norm_case(seed, 60, 520, BF16, F32, "channel")
    x, dy = _randn(_gen(seed), 160, 264), _randn(_gen(seed + 1), 160, 328, dtype=BF16)
    packed = g7.w4_pack(codes)

    def run():
        k, act_ = g7.gemm_ckpt8_pack(x, activation="gelu")
        dz, db = g7.gemm_ckpt8_act_grad(x, k, "gelu")
        return [g7.gemm_w4(a, packed, scales, zeros=z, group=32), *g7.gemm_norm_gate(**n),
                *g7.gemm_norm_gate_bwd(**n, d_x_out=n["x"], d_h=n["y"]), act_, dz, db,
                g7.gemm_ckpt8_wgrad(k, dy)]
    return run, (a, n["x"], n["y"], x, dy)


def test_layer_on_two_streams():
    runs = [_all_ops(s)[0] for s in (1, 2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [[], []]
    for _ in range(5):
        for i, (r, s) in enumerate(zip(runs, streams)):
            with torch.cuda.stream(s):
                got[i] = r()
    torch.cuda.synchronize()
    for w, o in zip(itertools.chain(*want), itertools.chain(*got)):
        assert torch.equal(w, o)
    assert g7.gemm_get_device_status() == 0


def test_layer_in_a_graph():
    run, inputs = _all_ops(5)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = run()
    for t in inputs:
        t.copy_(t.flip(0) * 0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in out]
    for w, o in zip(run(), got):
        assert torch.equal(w, o)


def test_layer_refusals():
    a, codes, scales, z = _w4_case(1, 2, 100, 20, 32, True)
    packed = g7.w4_pack(codes)
    n = _norm_case(2, 5, 16, F32, F32, "none")
    k = g7.gemm_ckpt8_pack(n["x"])
    bad_value = [
        lambda: g7.gemm_w4(a, packed, scales, zeros=z, group=48),
        lambda: g7.gemm_w4(a, packed, scales, zeros=z, group=64),
        lambda: g7.gemm_w4(a, packed[:-16], scales, zeros=z, group=32),
        lambda: g7.gemm_w4(a, packed, scales, zeros=z[:, :-1], group=32),
        lambda: g7.gemm_w4(a, packed, scales, zeros=z, group=32, beta=1.0),
        lambda: g7.gemm_w4(a, packed, scales, zeros=z, group=32, activation="tanh"),
        lambda: g7.gemm_w4(a, packed, scales, zeros=z, group=32, bias=a[0].float()),
        lambda: g7.gemm_w4(a[:, ::2], packed, scales, zeros=z, group=32),
        lambda: g7.gemm_w4(a[:1].expand(2, 100), packed, scales, zeros=z, group=32),
        lambda: g7.gemm_w4(a.cpu(), packed, scales, zeros=z, group=32),
        lambda: g7.w4_quantize(a, group=16),
        lambda: g7.gemm_norm_gate(n["x"], n["y"][:, :8]),
        lambda: g7.gemm_norm_gate(n["x"], gate=n["y"]),
        lambda: g7.gemm_norm_gate(n["x"], n["y"], gate=torch.ones(7, device="cuda")),
        lambda: g7.gemm_norm_gate(n["x"], n["y"], weight_pre=torch.ones(15, device="cuda")),
        lambda: g7.gemm_norm_gate(torch.ones((1, 16385), device="cuda")),
        lambda: g7.gemm_norm_gate_bwd(n["x"], n["y"], n["x"], n["x"]),
        lambda: g7.gemm_norm_gate_bwd(n["x"], n["y"], n["x"], weight_pre=n["weight_pre"]),
        lambda: g7.gemm_ckpt8_pack(n["x"], activation="silu"),
        lambda: g7.gemm_ckpt8_pack(n["x"], act_out=n["x"].to(BF16)),
        lambda: g7.gemm_ckpt8_unpack(k._replace(rows=40)),
        lambda: g7.gemm_ckpt8_act_grad(n["x"][:4], k, "relu"),
        lambda: g7.gemm_ckpt8_wgrad(k, n["x"][:4].to(BF16)),
        lambda: g7.gemm_ckpt8_wgrad(k, n["x"].to(BF16), beta=1.0),
    ]
    for i, f in enumerate(bad_value):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")
    bad_type = [
        lambda: g7.gemm_w4(a.float(), packed, scales, zeros=z, group=32),
        lambda: g7.gemm_w4(a, packed, scales.float(), zeros=z, group=32),
        lambda: g7.gemm_w4(a, packed, scales, zeros=z, group=32, out_dtype=torch.float16),
        lambda: g7.w4_pack(codes.int()),
        lambda: g7.gemm_norm_gate(n["x"].double()),
        lambda: g7.gemm_norm_gate_bwd(n["x"], n["y"], n["x"].to(BF16)),
        lambda: g7.gemm_ckpt8_pack(n["x"].half()),
        lambda: g7.gemm_ckpt8_wgrad(k, n["x"]),
        lambda: g7.gemm_ckpt8_unpack(k, torch.float16),
    ]
    for f in bad_type:
        with pytest.raises(TypeError):
            f()
    # a vector that starts off 16 bytes is taken element by element
    off = torch.ones(17, device="cuda")[1:]
    x_out, h = g7.gemm_norm_gate(n["x"], n["y"], weight_post=off, weight_pre=off)
    want = g7.gemm_norm_gate(n["x"], n["y"], weight_post=off.clone(), weight_pre=off.clone())
    _close(h, want[1].double(), 2.0 ** -7 * want[1].double().abs() + 1e-9)
    assert _abi.gemm_w4_packed_bytes(-1, 4) == -1


# ------------------------------------------------------------- together

def _rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_block_trains_and_decodes():
    """The example block against 64 bits.  BF16 operands and outputs round by 2^-9
    each, 8-bit checkpoints by at most half a step of 2 * max / 127 over 32 rows
    (about 0.5 % of a normal run's values): a few of these in a chain stay below 3 %."""
    from dense_gemm_07_gb300 import layer_example
    T, D, H = 192, 256, 640
    b = layer_example.Block(D, H, seed=3)
    g = _gen(4)
    x, dx, dh = (_randn(g, T, D, dtype=BF16), _randn(g, T, D, dtype=BF16), _randn(g, T, D))
    x_out, h, grads = layer_example.train_step(b, x, dx, dh)
    v = {n: getattr(b, n).double().requires_grad_() for n in ("w1", "b1", "w2", "pre", "post", "gate",
                                                              "next_pre")}
    v["x"] = x.double().requires_grad_()

    def block(x_, w1, w2, h_=None):
        r = lambda t: t / torch.sqrt((t ** 2).mean(1, keepdim=True) + 1e-6)  # noqa: E731
        h_ = r(x_) * v["pre"] if h_ is None else h_
        y = act(h_ @ w1 + v["b1"], "gelu") @ w2
        u = b.scale * x_ + v["gate"] * (r(y) * v["post"])
        return u, r(u) * v["next_pre"]

    u, hn = block(v["x"], v["w1"], v["w2"])
    assert _rel(x_out, u.detach()) < 0.01 and _rel(h, hn.detach()) < 0.01
    ((u * dx.double()).sum() + (hn * dh.double()).sum()).backward()
    for name, got in grads.items():
        assert _rel(got, v[name].grad) < 0.03, name

    rows = x[:5]
    _, h0 = g7.gemm_norm_gate(rows, weight_pre=b.pre)
    w1, w2 = (w4_weights(w4_layout_decode(q[0], *s).cuda(), q[1], q[2], b.group)
              for q, s in ((b.w1_q, (D, H)), (b.w2_q, (H, D))))
    du, dhn = layer_example.decode_step(b, rows, h0)
    u, hn = block(rows.double(), w1, w2, h0.double())
    assert _rel(du, u.detach()) < 0.01 and _rel(dhn, hn.detach()) < 0.01


def test_weight_gradient_gives_up_after_a_bounded_wait():
    """A first slice that is never copied: the wait runs out, the kernel unwinds and
    the status says so; the next call is exact."""
    T, K, N = 300, 300, 520
    x = torch.full((T, K), 127.0, device="cuda")
    dy = torch.ones((T, N), dtype=BF16, device="cuda")
    k = g7.gemm_ckpt8_pack(x)
    try:
        assert _abi.gemm_debug_inject(1, 2_000_000) == _abi.GEMM_OK
        g7.gemm_ckpt8_wgrad(k, dy)
        assert g7.gemm_get_device_status() == _abi.GEMM_ERR_TIMEOUT
    finally:
        assert _abi.gemm_debug_inject(0, 0) == _abi.GEMM_OK
    assert torch.equal(g7.gemm_ckpt8_wgrad(k, dy), torch.full((K, N), 127.0 * T, device="cuda"))
    assert g7.gemm_get_device_status() == _abi.GEMM_OK


def test_layer_large_offsets():
    """Rows past 2^31 elements of a buffer: a checkpoint, a norm and a gradient of the
    last rows of a long tensor equal those of the rows alone."""
    T, D = 262150, 8256  # 2.16e9 elements of BF16
    big = torch.empty((T, D), dtype=BF16, device="cuda")
    tail = _randn(_gen(1), 70, D, dtype=BF16)
    big[:-70] = 1.0
    big[-70:] = tail
    w = torch.ones(D, device="cuda")
    _, h = g7.gemm_norm_gate(big, weight_pre=w, x_out=big)
    _, want = g7.gemm_norm_gate(tail, weight_pre=w)
    assert torch.equal(h[-70:], want)
    del h
    k = g7.gemm_ckpt8_pack(big)
    assert int(k.q.numel()) > 2 ** 31
    got = kept(big[-38:])
    last = g7.gemm_ckpt8_unpack(k)[-38:]
    first = (T - 38) % 32
    assert first == 0 and torch.equal(last.double(), got)
    del last
    dy = torch.zeros((T, 8), dtype=BF16, device="cuda")
    dy[-38:] = 1.0
    dw = g7.gemm_ckpt8_wgrad(k, dy)
    s = got.abs().sum(0, keepdim=True).t()
    _close(dw, got.sum(0).view(-1, 1).expand(D, 8), 80 * EPS32 * s + 1e-30)
