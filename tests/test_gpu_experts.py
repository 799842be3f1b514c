"""The 8-bit floating-point products and the operators of a layer of experts against
their plain 64-bit forms, at the sizes, strides, types and values where they can go
wrong.

Tolerances.  EPS32 = 2^-23 is one unit of FP32, the loss of one truncated or rounded
operation relative to the magnitudes it adds.  An output rounded to a type adds half a
step of it, finfo.eps / 2 of the value: bf16 2^-8.  Codes and scales are exact: a
power of two divides exactly, so that the nearest code is the only rounding.
"""
import itertools
import math

import pytest
import torch

import dense_gemm_07_gb300 as g7
import experts_reference as ref
from dense_gemm_07_gb300 import _abi
from layer_reference import EPS32, act

pytestmark = pytest.mark.gpu

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
STEP = {F32: EPS32 / 2, BF16: 2.0 ** -8}  # the rounding to an output's type
NAN, INF = math.nan, math.inf


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _strided(t, extra):
    """The same values in rows `extra` elements further apart, off by one element when
    extra is odd; the gaps hold NaN."""
    r, c = t.shape
    buf = torch.full((r * (c + extra) + extra + 1,), NAN, dtype=t.dtype, device=t.device)
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


def _bits(codes):
    return codes.contiguous().view(torch.uint8)


def _rows16(codes, extra=0):
    """A copy of codes (R x K) in rows a multiple of 16 bytes apart, NaN codes between."""
    R, K = codes.shape
    buf = torch.full((R, -(-K // 16) * 16 + extra), 127, dtype=torch.uint8, device=codes.device)
    buf[:, :K] = _bits(codes).view(R, K)
    return buf.view(F8)[:, :K]


def _status():
    torch.cuda.synchronize()
    assert g7.gemm_get_device_status() == 0


# ---------------------------------------------------------------- quantising

def _spread(g, R, K, dtype=F32):
    """Values of very unlike sizes, with zeros among them and zero blocks."""
    x = _randn(g, R, K) * torch.exp(4 * _randn(g, R, 1)) * torch.exp(2 * _randn(g, 1, K))
    x = x * (torch.rand((R, K), generator=g, device="cuda") > 0.1)
    x[R // 2, : min(K, 130)] = 0
    return x.to(dtype)


QUANT = [(1, 1), (1, 128), (3, 127), (2, 129), (17, 300), (127, 1000), (16, 512), (33, 640),
         (130, 257), (1, 4096), (200, 1), (300, 72), (40, 132), (9, 1036)]


@pytest.mark.parametrize("R,K", QUANT)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("extra", [0, 4, 8, 3])
def test_quantize(R, K, dtype, extra):
    x = _spread(_gen(R * 1000 + K), R, K, dtype)
    arg = _strided(x, extra) if extra else x
    for square, transpose in itertools.product((False, True), repeat=2):
        q = g7.gemm_fp8_quantize(arg, square=square, transpose=transpose)
        codes, scales = ref.quantize(x.t() if transpose else x, square)
        assert q.codes.dtype == F8 and q.codes.shape == codes.shape and q.square == square
        assert torch.equal(q.scales.double(), scales), (square, transpose)
        assert torch.equal(_bits(q.codes), codes.to(torch.uint8)), (square, transpose)


def test_quantize_every_border():
    """All halfway points between codes and their neighbours, and the ends of a block's
    range, decide as the definition says."""
    table = ref.e4m3_numbers()
    mid = (table[1:] + table[:-1]) / 2
    v = torch.cat([table, mid, torch.nextafter(mid.float(), torch.tensor(INF)).double(),
                   torch.nextafter(mid.float(), torch.tensor(-INF)).double()]).float()
    v = torch.cat([v, -v])
    v = torch.nn.functional.pad(v, (0, -v.numel() % 127)).view(-1, 127)
    v = torch.cat([torch.full((v.shape[0], 1), 448.0), v], 1)  # the scale is 1
    for f, dtype in itertools.product((1.0, 2.0 ** 40, 2.0 ** -60, 2.0 ** -126), (F32, BF16)):
        x = (v * f).to(dtype).cuda()
        q = g7.gemm_fp8_quantize(x)
        codes, scales = ref.quantize(x.cpu())
        assert torch.equal(_bits(q.codes).cpu(), codes)
        assert torch.equal(q.scales.cpu().double(), scales)
    tops = torch.tensor([448.0, 449.0, 447.0, 2.0 ** -126, 2.0 ** -149, 2.0 ** -118, 3.4e38, 1.0,
                         448 * 2.0 ** -126, 449 * 2.0 ** -126, 1.75, 1.7500001])
    x = torch.zeros(tops.numel(), 128)
    x[:, 77] = tops
    q = g7.gemm_fp8_quantize(x.cuda())
    codes, scales = ref.quantize(x)
    assert torch.equal(_bits(q.codes).cpu(), codes) and torch.equal(q.scales.cpu().double(), scales)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_values_that_are_not_finite(bad, dtype):
    x = _randn(_gen(3), 140, 300, dtype=dtype)
    x[5, 140] = bad
    x[133, 299] = bad
    for square, transpose in itertools.product((False, True), repeat=2):
        q = g7.gemm_fp8_quantize(x, square=square, transpose=transpose)
        codes, scales = ref.quantize(x.t() if transpose else x, square)
        assert torch.equal(_bits(q.codes), codes) and torch.equal(q.scales.double(), scales)


@pytest.mark.parametrize("T,C,rows", [(1, 1, 1), (5, 129, 40), (100, 513, 7), (64, 1024, 300)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_picked_rows(T, C, rows, dtype):
    g = _gen(T)
    x = _spread(g, T, C, dtype)
    index = torch.randint(-2, T + 2, (rows,), generator=g, device="cuda", dtype=torch.int32)
    q = g7.gemm_fp8_quantize(x, index=index)
    on = (index >= 0) & (index < T)
    picked = torch.where(on[:, None], x[index.clamp(0, T - 1).to(torch.int64)], torch.zeros((), dtype=dtype, device="cuda"))
    codes, scales = ref.quantize(picked)
    codes = torch.where(on[:, None], codes, 0)
    assert torch.equal(_bits(q.codes), codes) and torch.equal(q.scales.double(), scales)


def test_quantize_several_matrices():
    x = _spread(_gen(9), 3 * 130, 200).view(3, 130, 200)
    wide = torch.full((3, 140, 210), NAN, device="cuda")
    wide[:, 5:135, :200] = x
    for arg, transpose in itertools.product((x, wide[:, 5:135, :200]), (False, True)):
        q = g7.gemm_fp8_quantize(arg, square=True, transpose=transpose)
        for e in range(3):
            codes, scales = ref.quantize(x[e].t() if transpose else x[e], True)
            assert torch.equal(_bits(q.codes[e]), codes) and torch.equal(q.scales[e].double(), scales)


def test_quantize_leaves_the_rest_of_its_rows():
    """Through the C entry point: bytes past a row's end and rows past the last stay."""
    x = _randn(_gen(2), 5, 200, dtype=BF16)
    for square, transpose in itertools.product((0, 1), repeat=2):
        R, K = (200, 5) if transpose else (5, 200)
        codes = torch.full((R + 2, 256), 7, dtype=torch.uint8, device="cuda")
        n = (-(-R // 128), -(-K // 128)) if square else (-(-K // 128), R)
        scales = torch.full((n[0] + 1, n[1] + 3), -1.0, device="cuda")
        a = _abi.GemmFp8QuantizeArgs(5, 200, x.data_ptr(), 200, 1, square, transpose, None, 0, 1, 0,
                                     codes.data_ptr(), 256, 0, scales.data_ptr(), n[1] + 3, 0)
        assert _abi.gemm_fp8_quantize(a, torch.cuda.current_stream().cuda_stream) == 0
        want, s = ref.quantize(x.t() if transpose else x, bool(square))
        assert torch.equal(codes[:R, :K], want) and torch.equal(scales[: n[0], : n[1]].double(), s)
        codes[:R, :K] = 7
        scales[: n[0], : n[1]] = -1
        assert bool((codes == 7).all()) and bool((scales == -1).all())


# ---------------------------------------------------------------- products

def _general(g, q, spread=1.0):
    """The same codes with scales that are not powers of two."""
    s = q.scales * torch.exp(spread * _randn(g, *q.scales.shape))
    return g7.Fp8(q.codes, s, q.square)


def _product_case(seed, M, N, K, square):
    g = _gen(seed)
    a = _general(g, g7.gemm_fp8_quantize(_spread(g, M, K) if M * K else torch.zeros(M, K, device="cuda")))
    b = _general(g, g7.gemm_fp8_quantize(_randn(g, N, K), square=square))
    return g, a, b


def _product_tol(va, vb, K):
    """In a block of 128 k the tensor core adds 32 products at a time: each of the 4
    additions, and the alignment inside each, loses at most one unit of the magnitudes.
    The product of the scales and the two roundings of a block's multiply-add lose
    half a unit each, and the sums of the blocks and of 8 partial sums one each."""
    return (8 + 2 + -(-K // 128) + 8) * EPS32 * (va.abs() @ vb.abs().transpose(-1, -2)) + 1e-300


PRODUCTS = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 127, 17), (3, 129, 385), (7, 1000, 3001),
            (16, 256, 640), (17, 300, 257), (32, 1, 129), (33, 520, 2048), (64, 130, 1000),
            (100, 128, 512), (127, 257, 300), (128, 128, 128), (129, 1000, 200), (200, 3, 4096),
            (255, 384, 1100), (256, 256, 256), (257, 513, 385), (300, 700, 129), (1000, 1000, 1000),
            (513, 2048, 512), (2047, 300, 700), (1500, 1100, 3001)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("square", [True, False])
def test_product(M, N, K, square):
    _, a, b = _product_case(M * 7 + K, M, N, K, square)
    va, vb = ref.values(*a), ref.values(*b)
    want, tol = va @ vb.t(), _product_tol(va, vb, K)
    out = g7.gemm_fp8(a, b)
    assert out.dtype == F32
    _close(out, want, tol, "product")
    low = g7.gemm_fp8(a, b, out_dtype=BF16)
    _close(low, want, tol + STEP[BF16] * (want.abs() + tol), "bf16")
    assert torch.equal(out, g7.gemm_fp8(a, b))
    _status()


@pytest.mark.parametrize("M,N,K", [(1, 77, 515), (16, 130, 1031), (140, 300, 384), (700, 1025, 640)])
@pytest.mark.parametrize("kind", ["none", "relu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("square", [True, False])
def test_product_epilogue_and_strides(M, N, K, kind, dtype, square):
    g, a, b = _product_case(5, M, N, K, square)
    a = g7.Fp8(a.codes, _strided(a.scales, 3))
    b = g7.Fp8(b.codes, _strided(b.scales, 5), square)
    a = g7.Fp8(_rows16(a.codes, 32), a.scales)
    bias, old = _randn(g, N), _randn(g, M, N, dtype=dtype)
    out = _strided(old, 3)
    va, vb = ref.values(*a), ref.values(*b)
    got = g7.gemm_fp8(a, b, out=out, alpha=0.5, beta=-2.0, bias=bias, activation=kind)
    assert got.data_ptr() == out.data_ptr()
    v = 0.5 * (va @ vb.t()) - 2.0 * old.double() + bias.double()
    # the epilogue: three roundings, GELU 4 units, and a slope of at most 1.13
    tol = 0.5 * _product_tol(va, vb, K) \
        + 4 * EPS32 * (0.5 * (va @ vb.t()).abs() + 2 * old.double().abs() + bias.double().abs())
    want = act(v, kind)
    _close(got, want, 1.13 * tol + 4 * EPS32 * v.abs() + STEP[dtype] * (want.abs() + tol), kind)


@pytest.mark.parametrize("M,N", [(3, 200), (150, 300), (600, 700)])
def test_product_guard_band(M, N):
    """Nothing outside C is written, and what lies behind the operands' rows (NaN codes)
    is not read as part of them."""
    K = 200
    _, a, b = _product_case(1, M, N, K, True)

    def padded(codes):
        more = torch.full((1, K), 127, dtype=torch.uint8, device="cuda").view(F8)
        return _rows16(torch.cat([_bits(codes).view(-1, K), _bits(more)]).view(F8), 16)[:-1]

    clean = g7.gemm_fp8(a, b)
    for dtype in (F32, BF16):
        guard = torch.full((M + 2, N + 8), 7.0, device="cuda", dtype=dtype)
        g7.gemm_fp8(g7.Fp8(padded(a.codes), a.scales), g7.Fp8(padded(b.codes), b.scales, True),
                    out=guard[1:M + 1, 4:4 + N])
        assert torch.equal(guard[1:M + 1, 4:4 + N], clean.to(dtype))
        guard[1:M + 1, 4:4 + N] = 7.0
        assert bool((guard == 7.0).all())


@pytest.mark.parametrize("M,N,K", [(5, 300, 700), (200, 300, 700), (520, 600, 400)])
@pytest.mark.parametrize("square", [True, False])
def test_product_values_that_are_not_finite(M, N, K, square):
    """A NaN code or an infinite scale shows in its row or column of C and nowhere else."""
    _, a, b = _product_case(2, M, N, K, square)
    clean = g7.gemm_fp8(a, b)
    codes = _rows16(a.codes)
    codes.view(torch.uint8)[M // 2, K - 1] = 127
    scales = b.scales.clone()
    if square:
        scales[1, 2] = INF
    else:
        scales[2, 130] = INF
    out = g7.gemm_fp8(g7.Fp8(codes, a.scales), g7.Fp8(b.codes, scales, square))
    cols = torch.zeros(N, dtype=torch.bool, device="cuda")
    cols[128:256] = square
    cols[130] = True
    assert bool(out[M // 2].isnan().all())
    rest = torch.arange(M, device="cuda") != M // 2
    assert not bool(torch.isfinite(out[rest][:, cols]).any())
    assert torch.equal(out[rest][:, ~cols], clean[rest][:, ~cols])


def test_product_of_nothing():
    g = _gen(0)
    bias, old = _randn(g, 5), _randn(g, 3, 5)
    empty = lambda r, s: g7.Fp8(torch.empty((r, 0), dtype=F8, device="cuda"),  # noqa: E731
                                torch.empty(s, device="cuda"))
    out = g7.gemm_fp8(empty(3, (0, 3)), empty(5, (0, 5)), out=old.clone(), beta=2.0, bias=bias)
    assert torch.equal(out, 2.0 * old + bias)
    x = g7.gemm_fp8_quantize(_randn(g, 4, 64))
    none = g7.gemm_fp8_quantize(torch.empty((0, 64), device="cuda"))
    assert g7.gemm_fp8(none, x).shape == (0, 4) and g7.gemm_fp8(x, none).shape == (4, 0)


def test_product_gradients():
    """Both gradients of C = A B^T by the same operator, on quantised factors."""
    M, N, K = 200, 260, 300
    g = _gen(8)
    x, w, dy = _randn(g, M, K, dtype=BF16), _randn(g, N, K, dtype=BF16), _randn(g, M, N, dtype=BF16)
    dq, wt = g7.gemm_fp8_quantize(dy), g7.gemm_fp8_quantize(w, square=True, transpose=True)
    va, vb = ref.values(*dq), ref.values(*wt)
    _close(g7.gemm_fp8(dq, wt), va @ vb.t(), _product_tol(va, vb, N), "dA")
    # (a code is off by at most 2^-4 of its value, or 2^-10 of its block's scale)
    assert float((va @ vb.t() - dy.double() @ w.double()).norm()) < 0.07 * float(
        (dy.double().abs() @ w.double().abs()).norm())
    dt, xt = g7.gemm_fp8_quantize(dy, transpose=True), g7.gemm_fp8_quantize(x, transpose=True)
    va, vb = ref.values(*dt), ref.values(*xt)
    _close(g7.gemm_fp8(dt, xt), va @ vb.t(), _product_tol(va, vb, M), "dB")


# ---------------------------------------------------------------- experts

def _experts_case(seed, lengths, N, K):
    g = _gen(seed)
    E, R = len(lengths), sum(lengths)
    a = _general(g, g7.gemm_fp8_quantize(_randn(g, R, K))) if R else g7.gemm_fp8_quantize(
        torch.zeros((0, K), device="cuda"))
    b = _general(g, g7.gemm_fp8_quantize(_randn(g, E, N, K), square=True))
    offsets = torch.tensor([0, *itertools.accumulate(lengths)], dtype=torch.int32, device="cuda")
    return g, a, b, offsets


EXPERTS = [([1], 1, 1), ([0, 1, 0], 130, 200), ([5, 0, 0, 3, 17], 300, 513), ([2] * 40, 64, 128),
           ([128, 1, 129, 0, 256], 257, 385), ([300, 20, 0, 700, 1], 512, 640), ([1000], 200, 300),
           ([0] * 33 + [40, 1], 128, 256), ([16, 15, 17, 1, 31, 33], 1000, 1000),
           ([257, 255, 511, 513, 2, 90], 700, 1100), ([600, 900, 400], 1030, 512)]


@pytest.mark.parametrize("lengths,N,K", EXPERTS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_experts(lengths, N, K, dtype):
    g, a, b, offsets = _experts_case(N + K, lengths, N, K)
    bias = _randn(g, len(lengths), N)
    at = offsets.tolist()
    va, vb = ref.values(*a), ref.values(*b)
    for kind, use in (("none", None), ("gelu", bias), ("relu", bias)):
        out = g7.gemm_fp8_experts(a, b, offsets, bias=use, activation=kind, out_dtype=dtype)
        for e in range(len(lengths)):
            r = slice(at[e], at[e + 1])
            v = va[r] @ vb[e].t()
            tol = _product_tol(va[r], vb[e], K) + 4 * EPS32 * v.abs()
            if use is not None:
                v = v + bias[e].double()
                tol = tol + 4 * EPS32 * bias[e].double().abs()
            want = act(v, kind)
            _close(out[r], want, 1.13 * tol + 4 * EPS32 * v.abs() + STEP[dtype] * (want.abs() + tol),
                   f"expert {e} {kind}")
    _status()


def test_experts_rows_outside_stay():
    """Rows before the first offset and from the last one on are left as they were, and
    offsets that make no sense are held to the rows there are."""
    g, a, b, _ = _experts_case(3, [100, 200, 60], 200, 256)
    va, vb = ref.values(*a), ref.values(*b)
    for given, held in (([10, 50, 50, 300], [10, 50, 50, 300]),
                        ([-5, 100, 90, 9999], [0, 100, 100, 360]),
                        ([400, 400, 400, 400], [360, 360, 360, 360]),
                        ([0, 0, 0, 0], [0, 0, 0, 0]),
                        ([200, 100, 2 ** 31 - 1, -2 ** 31], [200, 200, 360, 360])):
        offsets = torch.tensor(given, dtype=torch.int32, device="cuda")
        old = _randn(g, 360, 200)
        out = g7.gemm_fp8_experts(a, b, offsets, out=old.clone(), alpha=2.0, beta=0.5)
        want, tol = old.double(), torch.zeros_like(old, dtype=torch.float64)
        for e in range(3):
            r = slice(held[e], held[e + 1])
            v = va[r] @ vb[e].t()
            want[r] = 2.0 * v + 0.5 * old[r].double()
            tol[r] = 2.0 * _product_tol(va[r], vb[e], 256) + 4 * EPS32 * (2 * v.abs() + old[r].double().abs())
        _close(out, want, tol, str(given))
    _status()


def test_experts_are_the_dense_product():
    """One expert with all rows is gemm_fp8, bit for bit where both take the same tiles."""
    g, a, b, offsets = _experts_case(11, [600], 500, 900)
    dense = g7.gemm_fp8(a, g7.Fp8(b.codes[0], b.scales[0], True))
    some = g7.gemm_fp8_experts(a, b, offsets)
    va, vb = ref.values(*a), ref.values(*b)
    _close(some, dense.double(), 2 * _product_tol(va, vb[0], 900))


# ---------------------------------------------------------------- routing

def _check_route(logits, k, **kw):
    r = g7.gemm_route(logits, k, **kw)
    index, weight, slot, source, offsets = ref.route(logits, k, **kw)
    assert torch.equal(r.index.cpu(), index)
    assert torch.equal(r.slot.cpu(), slot)
    assert torch.equal(r.source.cpu(), source)
    assert torch.equal(r.offsets.cpu(), offsets)
    # the exponential and a quotient lose 2 units each, a sum of 1024 numbers (32 a lane,
    # then 5 steps) 40; the difference in the exponent half a unit of its size
    far = torch.where(torch.isfinite(logits), logits, torch.zeros((), dtype=logits.dtype, device="cuda"))
    far = float(far.double().abs().max()) if far.numel() else 0.0
    got = r.weight.cpu().double()
    assert torch.equal(got.isnan(), weight.isnan())
    ok = ~weight.isnan()
    assert bool(((got - weight).abs()[ok] <= (64 + 2 * far) * EPS32 * weight.abs()[ok] + 1e-37).all())
    return r


ROUTES = [(1, 1, 1), (1, 64, 4), (2, 8, 8), (5, 33, 3), (127, 60, 6), (128, 256, 8), (129, 100, 5),
          (300, 512, 12), (260, 257, 5), (300, 33, 3), (1000, 72, 2), (3, 1024, 32), (200, 600, 10), (513, 16, 1)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route(T, E, k, score, dtype):
    g = _gen(T + E)
    logits = _randn(g, T, E, dtype=dtype, scale=2.0)
    bias = _randn(g, E, scale=0.1)
    for renorm, b in itertools.product((True, False), (None, bias, torch.zeros_like(bias))):
        _check_route(logits, k, score=score, bias=b, renormalize=renorm, scale=2.5)
    _check_route(_strided(logits, 3), k, score=score, bias=bias)


GROUPED = [(1, 16, 2, 4, 2), (40, 256, 8, 8, 4), (130, 64, 4, 8, 3), (33, 60, 4, 5, 2),
           (20, 1024, 8, 32, 5), (50, 96, 6, 3, 1), (17, 32, 2, 32, 4), (260, 160, 6, 8, 3)]


@pytest.mark.parametrize("T,E,k,groups,kept", GROUPED)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2])
def test_route_groups(T, E, k, groups, kept, score, top):
    g = _gen(T + E + top)
    for dtype in (F32, BF16):
        logits = _randn(g, T, E, dtype=dtype, scale=2.0)
        for bias in (None, _randn(g, E, scale=0.1)):
            _check_route(logits, k, score=score, bias=bias, groups=groups, groups_kept=kept,
                         group_top=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_route_ties(score, groups, kept):
    """Logits with many equal values and biases with few: the lowest index wins."""
    g = _gen(4)
    logits = torch.randint(-3, 4, (300, 64), generator=g, device="cuda").float() / 2
    for bias in (None, torch.zeros(64, device="cuda"),
                 torch.randint(0, 2, (64,), generator=g, device="cuda").float() / 8):
        _check_route(logits, 8, score=score, bias=bias, groups=groups, groups_kept=kept)
    logits[:, ::2] = 0.0
    logits[:, 1::2] = -0.0
    _check_route(logits, 8, score=score, groups=groups, groups_kept=kept)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 3)])
def test_route_scores_closer_than_fp32_tells(score, groups, kept):
    """score + bias within a few units of FP32 of each other: decided in 64 bits."""
    g = _gen(6)
    E = 64
    one = _randn(g, E, scale=2.0)
    s = torch.softmax(one.double(), 0) if score == "softmax" else torch.sigmoid(one.double())
    bias = (1.5 - s).float()
    v = s + bias.double()
    assert float(v.max() - v.min()) < 2e-7  # all of them closer than FP32 resolves
    logits = one.repeat(50, 1)
    _check_route(logits, 6, score=score, bias=bias, groups=groups, groups_kept=kept)
    near = logits + 1e-7 * _randn(g, 50, E)
    _check_route(near, 6, score=score, bias=bias, groups=groups, groups_kept=kept)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [9, 400])
def test_route_closed_experts_and_padding(score, T):
    g = _gen(7)
    logits = _randn(g, T, 24)
    logits[torch.rand((T, 24), generator=g, device="cuda") < 0.5] = -INF
    logits[1] = -INF                       # a token of padding
    logits[2, 1:] = -INF                   # one expert left
    logits[T - 3:] = -INF                  # behind the last sequence
    lowest = logits.clone()
    lowest[3] = torch.finfo(F32).min       # masked with the type's lowest value
    lowest[4, 5:] = torch.finfo(F32).min
    bias = _randn(g, 24, scale=0.1)
    closed = bias.clone()
    closed[3], closed[7] = -INF, NAN
    for l, b, n in itertools.product((logits, lowest), (None, bias, closed), (1, 4)):
        r = _check_route(l, 4, score=score, bias=b, groups=n, groups_kept=max(1, n - 1))
        assert int((r.index[1] >= 0).sum()) == 0 and float(r.weight[1].abs().sum()) == 0
    none = torch.full((T, 24), -INF, device="cuda")
    r = _check_route(none, 3, score=score)
    assert int(r.offsets.abs().sum()) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_values_that_are_not_finite(score):
    logits = _randn(_gen(1), 6, 40)
    logits[1, 3] = NAN
    logits[2, 39] = INF
    logits[4] = INF
    for bias in (None, torch.zeros(40, device="cuda")):
        for groups in (1, 4):
            _check_route(logits, 5, score=score, bias=bias, groups=groups, groups_kept=groups)


def test_route_without_tokens():
    r = g7.gemm_route(torch.empty((0, 12), device="cuda"), 3)
    assert r.index.shape == (0, 3) and torch.equal(r.offsets.cpu(), torch.zeros(13, dtype=torch.int32))


@pytest.mark.parametrize("T", [5000, 20000])
def test_route_long(T):
    """Many blocks of tokens, against a sort (the token-by-token form takes too long)."""
    g = _gen(T)
    E, k = 256, 8
    logits = _randn(g, T, E)
    logits[T - 11:] = -INF
    r = g7.gemm_route(logits, k)
    best, index = logits.sort(dim=1, descending=True, stable=True)
    index = torch.where(best > -INF, index, -1)[:, :k].to(torch.int32)
    assert torch.equal(r.index, index)
    key = torch.where(index < 0, E, index).reshape(-1)
    order = torch.sort(key, stable=True).indices
    n = int((key < E).sum())
    assert torch.equal(r.offsets[1:], (key[:, None] == torch.arange(E, device="cuda")).sum(0).cumsum(0).to(torch.int32))
    assert torch.equal(r.source[:n], (order[:n] // k).to(torch.int32)) and bool((r.source[n:] == -1).all())
    slot = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    slot[order[:n]] = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(r.slot.reshape(-1), slot)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (7, 64, 4), (100, 257, 6), (33, 60, 32), (9, 1024, 8),
                                   (600, 512, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_gradient(T, E, k, score, renorm, dtype):
    g = _gen(T + E)
    logits = _strided(_randn(g, T, E, dtype=dtype), 3)
    index = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), dim=1)[:, :k].to(torch.int32)
    index[0, 0] = -1
    if T > 3:
        index[1] = -1
        index[2, -1] = E + 7
        index[3, -1] = index[3, 0]  # the same expert twice
    d = _randn(g, T, k)
    out = _strided(torch.zeros(T, E, dtype=dtype, device="cuda"), 5)
    got = g7.gemm_route_bwd(logits, index, d, score=score, renormalize=renorm, scale=1.5, out=out)
    assert got.dtype == dtype and got.data_ptr() == out.data_ptr()
    want, size = ref.route_grad(logits, index, d, score, renorm, 1.5)
    # sums of 32 terms by halves and of 1024 scores (40 units), exponentials and quotients
    far = float(logits.double().abs().max())
    tol = (96 + 4 * far) * EPS32 * size + STEP[dtype] * want.abs() + 1e-37
    _close(got, want, tol, "gradient")
    assert torch.equal(got, g7.gemm_route_bwd(logits, index, d, score=score, renormalize=renorm, scale=1.5))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("low", [-60.0, -88.0, -95.0, -150.0, -400.0])
def test_route_logits_far_below_zero(score, low):
    """Sigmoids that FP32 does not hold have quotients that it does."""
    g = _gen(3)
    T, E, k = 150, 48, 4
    logits = _randn(g, T, E) + low
    logits[0, 5] = 2.0                      # one score that is not small
    bias = _randn(g, E)
    for b in (None, bias):
        _check_route(logits, k, score=score, bias=b)
    masked = logits.clone()
    masked[1, 5:] = torch.finfo(F32).min    # experts masked with the lowest value
    masked[4] = torch.finfo(F32).min
    # as _check_route's bound, by the logits that are not masks: a mask's exponent is
    # taken to 0 or from its like
    step = (64 + 2 * (abs(low) + 10)) * EPS32
    got, want = g7.gemm_route(masked, k, score=score), ref.route(masked, k, score=score)
    assert torch.equal(got.index.cpu(), want[0])
    _close(got.weight.cpu(), want[1], step * want[1] + 1e-37, "weights")
    index = torch.argsort(torch.rand((T, E), generator=g, device="cuda"), dim=1)[:, :k].to(torch.int32)
    index[0, 0], index[1, 0], index[2, 3] = 5, 0, -1
    d = 3.0 * _randn(g, T, k)
    got = g7.gemm_route_bwd(masked, index, d, score=score)
    want, size = ref.route_grad(masked, index, d, score, True, 1.0)
    assert float(want.abs().max()) > 0.1
    # as test_route_gradient's
    _close(got, want, (96 + 4 * (abs(low) + 10)) * EPS32 * size + 1e-37, "gradient")


# ---------------------------------------------------------------- combining

def _pairs(g, T, k, R, holes=True):
    n = T * k
    slot = torch.argsort(torch.rand(max(R, n), generator=g, device="cuda"))[:n].to(torch.int32)
    slot = slot.view(T, k)
    if holes and n:
        slot[torch.rand((T, k), generator=g, device="cuda") < 0.2] = -1
        slot[-1] = -1
    return slot, torch.rand((T, k), generator=g, device="cuda") - 0.3


COMBINES = [(1, 1, 1, 1), (1, 4096, 8, 8), (3, 129, 2, 10), (50, 1000, 5, 250), (17, 3001, 3, 40),
            (64, 512, 32, 2048), (5, 8200, 4, 30), (300, 64, 1, 300), (9, 16, 12, 100)]


@pytest.mark.parametrize("T,D,k,R", COMBINES)
@pytest.mark.parametrize("rows_type,x_type,out_type", list(itertools.product((F32, BF16), (None, F32, BF16),
                                                                       (F32, BF16))))
def test_combine(T, D, k, R, rows_type, x_type, out_type):
    g = _gen(T + D)
    rows = _randn(g, R, D, dtype=rows_type)
    slot, w = _pairs(g, T, k, R)
    x = None if x_type is None else _randn(g, T, D, dtype=x_type)
    want, size = ref.combine(rows, slot, w, x)
    tol = (k + 2) * EPS32 * size + STEP[out_type] * want.abs()
    _close(g7.gemm_combine(rows, slot, w, x=x, out_dtype=out_type), want, tol, "aligned")
    out = _strided(torch.zeros(T, D, dtype=out_type, device="cuda"), 3)
    got = g7.gemm_combine(_strided(rows, 5), slot, w, x=None if x is None else _strided(x, 1), out=out)
    assert got.data_ptr() == out.data_ptr()
    _close(got, want, tol, "strided")
    wide = _strided(torch.zeros(T, D, dtype=out_type, device="cuda"), 8)
    _close(g7.gemm_combine(_strided(rows, 16), slot, w, x=x, out=wide), want, tol, "wide strides")


@pytest.mark.parametrize("T,D,k,R", COMBINES)
@pytest.mark.parametrize("rows_type,out_type", list(itertools.product((F32, BF16), repeat=2)))
def test_combine_gradient(T, D, k, R, rows_type, out_type):
    g = _gen(T + D)
    rows, d = _randn(g, R, D, dtype=rows_type), _randn(g, T, D, dtype=out_type)
    slot, w = _pairs(g, T, k, R)
    for extra in (0, 3, 8):
        before = _randn(g, R, D, dtype=rows_type)
        pad = (lambda t: _strided(t, extra)) if extra else (lambda t: t.clone())  # noqa: E731
        d_rows, d_weight = g7.gemm_combine_bwd(pad(d), pad(rows), slot, w, d_rows=pad(before))
        want, dw, size = ref.combine_grad(d, rows, slot, w, before)
        _close(d_rows, want, STEP[rows_type] * want.abs() + 1e-40, "rows")
        # a thread adds every 256th (or 2048th, eight at a time) product, then 256 sums by halves
        _close(d_weight, dw, (D // 256 + 24) * EPS32 * size, "weights")


def test_combine_in_place_and_non_finite_weights():
    g = _gen(1)
    rows, x = _randn(g, 20, 300, dtype=BF16), _randn(g, 4, 300)
    slot = torch.tensor([[1, -1], [-1, -1], [25, 3], [4, 5]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 2.0], [1.0, 1.0], [1.0, 1.0], [1.0, 1.0]], device="cuda")
    want, size = ref.combine(rows, slot, w, x)
    y = x.clone()
    assert g7.gemm_combine(rows, slot, w, x=y, out=y).data_ptr() == y.data_ptr()
    _close(y, want, 4 * EPS32 * size)
    assert torch.equal(y[1], x[1])
    w[0, 1] = NAN
    w[1, 0] = INF
    out = g7.gemm_combine(rows, slot, w, x=x)
    assert bool(out[:2].isnan().all()) and torch.equal(out[2:], y[2:])
    # the gradient of rows in the rows' own place
    w = torch.rand((4, 2), generator=g, device="cuda")
    same = rows.clone()
    a = g7.gemm_combine_bwd(x, rows, slot, w, d_rows=rows.clone())
    b = g7.gemm_combine_bwd(x, same, slot, w, d_rows=same)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_combine_of_nothing():
    rows = torch.ones((0, 8), device="cuda")
    slot = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.ones((3, 2), device="cuda")
    x = torch.randn((3, 8), device="cuda")
    assert torch.equal(g7.gemm_combine(rows, slot, w, x=x), x)
    assert torch.equal(g7.gemm_combine(rows, slot, w), torch.zeros_like(x))
    none = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    assert torch.equal(g7.gemm_combine(rows, none, none.float(), x=x), x)
    assert g7.gemm_combine(rows, slot[:0], w[:0]).shape == (0, 8)
    d_rows, d_w = g7.gemm_combine_bwd(x, rows, slot, w)
    assert d_rows.shape == (0, 8) and torch.equal(d_w, torch.zeros_like(w))


# ---------------------------------------------------------------- refusals

def _refused(kind, f, *a, **kw):
    with pytest.raises(kind):
        f(*a, **kw)


def test_refusals():
    g = _gen(0)
    x = _randn(g, 8, 64)
    q, w = g7.gemm_fp8_quantize(x), g7.gemm_fp8_quantize(x, square=True)
    R = lambda *a, **kw: _refused(ValueError, *a, **kw)  # noqa: E731
    R(g7.gemm_fp8_quantize, x[0])
    R(g7.gemm_fp8_quantize, x.t())
    R(g7.gemm_fp8_quantize, x.view(2, 4, 64))
    R(g7.gemm_fp8_quantize, x, square=True, index=torch.zeros(2, dtype=torch.int32, device="cuda"))
    R(g7.gemm_fp8_quantize, x, index=torch.zeros(2, dtype=torch.int64, device="cuda"))
    R(g7.gemm_fp8_quantize, x.cpu())
    _refused(TypeError, g7.gemm_fp8_quantize, x.half())
    R(g7.gemm_fp8, w, q)
    R(g7.gemm_fp8, q, g7.gemm_fp8_quantize(_randn(g, 8, 65)))
    R(g7.gemm_fp8, q, g7.Fp8(q.codes, q.scales, True))
    R(g7.gemm_fp8, q, q, beta=1.0)
    R(g7.gemm_fp8, q, q, bias=torch.zeros(9, device="cuda"))
    R(g7.gemm_fp8, q, q, activation="tanh")
    _refused(TypeError, g7.gemm_fp8, q, q, out_dtype=torch.float16)
    _refused(TypeError, g7.gemm_fp8, g7.Fp8(q.codes.float(), q.scales), q)
    odd = torch.zeros(8 * 65 + 16, dtype=torch.uint8, device="cuda").view(F8)
    R(g7.gemm_fp8, g7.Fp8(odd[: 8 * 65].view(8, 65)[:, :64], q.scales), q)   # rows off 16 bytes
    R(g7.gemm_fp8, g7.Fp8(odd[1:513].view(8, 64), q.scales), q)              # a start off 16 bytes
    e = g7.gemm_fp8_quantize(_randn(g, 3, 8, 64), square=True)
    offsets = torch.tensor([0, 2, 5, 8], dtype=torch.int32, device="cuda")
    R(g7.gemm_fp8_experts, q, w, offsets)
    R(g7.gemm_fp8_experts, q, e, offsets[:3])
    R(g7.gemm_fp8_experts, q, e, offsets.long())
    R(g7.gemm_fp8_experts, q, g7.Fp8(e.codes, e.scales), offsets)
    R(g7.gemm_fp8_experts, q, g7.Fp8(e.codes[::2], e.scales[::2].contiguous(), True), offsets[:3])
    R(g7.gemm_fp8_experts, q, e, offsets, bias=torch.zeros(8, device="cuda"))
    l = _randn(g, 4, 12)
    for kw in (dict(k=0), dict(k=13), dict(k=2, groups=5), dict(k=7, groups=2, groups_kept=1),
               dict(k=2, groups=2, groups_kept=3), dict(k=2, group_top=3), dict(k=2, score="tanh"),
               dict(k=2, bias=torch.zeros(11, device="cuda")), dict(k=2, groups=0)):
        R(g7.gemm_route, l, **kw)
    R(g7.gemm_route, torch.zeros((2, 1025), device="cuda"), 2)
    r = g7.gemm_route(l, 3)
    R(g7.gemm_route_bwd, l, r.index.long(), r.weight)
    R(g7.gemm_route_bwd, l, r.index, r.weight[:, :2])
    rows = _randn(g, 12, 16)
    R(g7.gemm_combine, rows, r.slot, r.weight[:2])
    R(g7.gemm_combine, rows, r.slot.long(), r.weight)
    R(g7.gemm_combine, rows, r.slot, r.weight, x=_randn(g, 4, 15))
    R(g7.gemm_combine, rows, torch.zeros((2, 33), dtype=torch.int32, device="cuda"),
      torch.zeros((2, 33), device="cuda"))
    R(g7.gemm_combine_bwd, _randn(g, 3, 16), rows, r.slot, r.weight)
    _refused(TypeError, g7.gemm_combine_bwd, _randn(g, 4, 16), rows, r.slot, r.weight,
             d_rows=rows.to(BF16))
