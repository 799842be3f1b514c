"""The 8-bit products and the operators of a layer of experts without a GPU: argument
checks of the C entry points (made before any device is looked for), and the 64-bit
reference forms against tables and differences."""
import ctypes
import math

import pytest
import torch

import dense_gemm_07_gb300 as g7
import experts_reference as ref
from dense_gemm_07_gb300 import _abi

INVALID, OK = _abi.GEMM_ERR_INVALID_ARG, _abi.GEMM_OK
P = 256  # a 16-byte aligned address that no check dereferences


@pytest.fixture(scope="module", autouse=True)
def lib():
    return _abi.lib()


def _make(cls, defaults, **kw):
    d = dict(defaults, **kw)
    return cls(*[d[n] for n, _ in cls._fields_])


def test_structs_match_the_header():
    assert ctypes.sizeof(_abi.GemmFp8) == 40
    assert ctypes.sizeof(_abi.GemmFp8QuantizeArgs) == 128
    assert ctypes.sizeof(_abi.GemmRouteArgs) == 80
    assert ctypes.sizeof(_abi.GemmCombineArgs) == 96


QUANT = dict(T=4, C=200, x=P, ldx=200, x_type=0, square=0, transpose=0, index=None, rows=0, batch=1,
             x_step=0, codes=P, ld=208, codes_step=0, scales=P, ld_scales=4, scales_step=0)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(C=2 ** 30 + 1), dict(x=None), dict(ldx=199), dict(x_type=2), dict(square=2),
    dict(transpose=-1), dict(index=P, square=1), dict(index=P, transpose=1), dict(index=P, rows=-1),
    dict(index=P, rows=9), dict(batch=2), dict(batch=-1), dict(batch=65536, square=1), dict(codes=None),
    dict(codes=P + 8), dict(ld=200), dict(ld=192), dict(scales=None), dict(ld_scales=3),
    dict(square=1, ld_scales=1), dict(transpose=1, ld_scales=199), dict(ldx=2 ** 61),
    dict(square=1, batch=2, x_step=-1), dict(square=1, batch=2, codes_step=8),
    dict(square=1, batch=2, scales_step=2 ** 61)])
def test_quantize_refusals(change):
    assert _abi.gemm_fp8_quantize(_make(_abi.GemmFp8QuantizeArgs, QUANT, **change), None) == INVALID
    assert _abi.gemm_fp8_quantize(None, None) == INVALID


A8 = dict(codes=P, ld=256, scales=P, ld_scales=8, square=0)
B8 = dict(codes=P, ld=256, scales=P, ld_scales=2, square=1)


def _a(**kw):
    return _make(_abi.GemmFp8, A8, **kw)


def _b(**kw):
    return _make(_abi.GemmFp8, B8, **kw)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(N=2 ** 30 + 1), dict(K=-1), dict(A=None), dict(B=None), dict(A=_a(square=1)),
    dict(A=_a(codes=None)), dict(A=_a(codes=P + 4)), dict(A=_a(ld=250)), dict(A=_a(ld=240)),
    dict(A=_a(scales=None)), dict(A=_a(ld_scales=3)), dict(B=_b(ld_scales=1)), dict(B=_b(square=3)),
    dict(B=_b(square=0, ld_scales=63)), dict(C=None), dict(ldc=63), dict(c_type=2),
    dict(A=_a(ld=2 ** 40)), dict(epi=_abi.GemmEpilogue(1.0, 0.0, None, 9))])
def test_product_refusals(change):
    a = dict(M=8, N=64, K=250, A=_a(), B=_b(), C=P, ldc=64, c_type=0, epi=None)
    a.update(change)
    assert _abi.gemm_fp8(*a.values(), None) == INVALID


@pytest.mark.parametrize("change", [
    dict(E=0), dict(E=1025), dict(B=_b(square=0, ld_scales=999)), dict(B=_b(codes=P + 8)),
    dict(offsets=None), dict(N=2 ** 29), dict(B=_b(ld=249)), dict(B=_b(ld_scales=1)), dict(B=None)])
def test_experts_refusals(change):
    a = dict(E=4, M=8, N=64, K=250, A=_a(), B=_b(), offsets=P, C=P, ldc=2 ** 30, c_type=0, epi=None)
    a.update(change)
    assert _abi.gemm_fp8_experts(*a.values(), None) == INVALID


ROUTE = dict(T=4, E=16, k=2, logits=P, ld=16, type=0, score=0, bias=None, groups=4, groups_kept=2,
             group_top=2, renormalize=1, scale=1.0)
BAD_ROUTES = [dict(T=-1), dict(E=0), dict(E=1025, groups=1, groups_kept=1, ld=1025), dict(k=0),
              dict(k=33), dict(logits=None), dict(ld=15), dict(type=5), dict(score=2),
              dict(renormalize=2), dict(T=2 ** 30, k=8)]


@pytest.mark.parametrize("change", BAD_ROUTES + [
    dict(groups=0), dict(groups=3), dict(groups=33), dict(groups_kept=0), dict(groups_kept=5),
    dict(group_top=0), dict(group_top=3), dict(k=9)])
def test_route_refusals(change):
    args = _make(_abi.GemmRouteArgs, ROUTE, **change)
    assert _abi.gemm_route(args, P, P, P, P, P, P, None) == INVALID


def test_route_output_refusals():
    args = _make(_abi.GemmRouteArgs, ROUTE)
    for i in range(5):
        out = [P] * 5
        out[i] = None
        assert _abi.gemm_route(args, *out, P, None) == INVALID
    many = _make(_abi.GemmRouteArgs, ROUTE, T=129)
    assert _abi.gemm_route(many, P, P, P, P, P, None, None) == INVALID
    assert _abi.gemm_route(many, P, P, P, P, P, P + 2, None) == INVALID
    assert _abi.gemm_route(None, P, P, P, P, P, P, None) == INVALID
    assert _abi.gemm_route_workspace_bytes(128, 256) == 0
    assert _abi.gemm_route_workspace_bytes(129, 256) > 0
    assert _abi.gemm_route_workspace_bytes(-1, 256) == -1
    assert _abi.gemm_route_workspace_bytes(5, 1025) == -1


@pytest.mark.parametrize("change", BAD_ROUTES)
def test_route_bwd_refusals(change):
    args = _make(_abi.GemmRouteArgs, ROUTE, **change)
    assert _abi.gemm_route_bwd(args, P, P, P, 2000, None) == INVALID


def test_route_bwd_output_refusals():
    args = _make(_abi.GemmRouteArgs, ROUTE)
    assert _abi.gemm_route_bwd(args, None, P, P, 16, None) == INVALID
    assert _abi.gemm_route_bwd(args, P, None, P, 16, None) == INVALID
    assert _abi.gemm_route_bwd(args, P, P, None, 16, None) == INVALID
    assert _abi.gemm_route_bwd(args, P, P, P, 15, None) == INVALID


COMBINE = dict(T=4, D=16, k=2, R=8, rows=P, ld_rows=16, rows_type=0, slot=P, weight=P, x=P, ldx=16,
               x_type=0)
BAD_COMBINES = [dict(T=-1), dict(D=2 ** 30 + 1), dict(k=-1), dict(k=33), dict(R=-1), dict(rows=None),
                dict(ld_rows=15), dict(rows_type=2), dict(slot=None), dict(weight=None),
                dict(ldx=15), dict(x_type=-1), dict(T=2 ** 30, k=8)]


@pytest.mark.parametrize("change", BAD_COMBINES)
def test_combine_refusals(change):
    args = _make(_abi.GemmCombineArgs, COMBINE, **change)
    assert _abi.gemm_combine(args, P, 16, 0, None) == INVALID
    assert _abi.gemm_combine_bwd(args, P, 16, 0, P, 16, P, None) == INVALID


def test_combine_output_refusals():
    args = _make(_abi.GemmCombineArgs, COMBINE)
    assert _abi.gemm_combine(args, None, 16, 0, None) == INVALID
    assert _abi.gemm_combine(args, P, 15, 0, None) == INVALID
    assert _abi.gemm_combine(args, P, 16, 7, None) == INVALID
    assert _abi.gemm_combine_bwd(args, None, 16, 0, P, 16, P, None) == INVALID
    assert _abi.gemm_combine_bwd(args, P, 15, 0, P, 16, P, None) == INVALID
    assert _abi.gemm_combine_bwd(args, P, 16, 3, P, 16, P, None) == INVALID
    assert _abi.gemm_combine_bwd(args, P, 16, 0, None, 16, P, None) == INVALID
    assert _abi.gemm_combine_bwd(args, P, 16, 0, P, 15, P, None) == INVALID
    assert _abi.gemm_combine_bwd(args, P, 16, 0, P, 16, None, None) == INVALID


def test_nothing_to_do_needs_no_gpu():
    quant = _make(_abi.GemmFp8QuantizeArgs, QUANT, T=0, x=None, codes=None, scales=None)
    assert _abi.gemm_fp8_quantize(quant, None) == OK
    assert _abi.gemm_fp8(0, 64, 250, _a(codes=None, scales=None), _b(), None, 64, 0, None, None) == OK
    assert _abi.gemm_fp8(8, 0, 250, _a(), _b(codes=None, scales=None), None, 1, 0, None, None) == OK
    combine = _make(_abi.GemmCombineArgs, COMBINE, T=0, slot=None, weight=None)
    assert _abi.gemm_combine(combine, None, 16, 0, None) == OK
    route = _make(_abi.GemmRouteArgs, ROUTE, T=0, logits=None)
    assert _abi.gemm_route_bwd(route, None, None, None, 16, None) == OK


def test_cpu_tensors_are_refused():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        g7.gemm_fp8_quantize(x)
    with pytest.raises(ValueError):
        g7.gemm_route(x, 2)
    with pytest.raises(ValueError):
        g7.gemm_combine(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))


# ------------------------------------------------------ the reference forms

def test_reference_codes_are_torchs():
    table = ref.e4m3_numbers()
    codes = torch.arange(127, dtype=torch.uint8)
    assert torch.equal(codes.view(torch.float8_e4m3fn).double(), table)
    g = torch.Generator().manual_seed(0)
    v = (torch.rand(20000, generator=g) * 2 - 1) * torch.exp(4 * torch.randn(20000, generator=g))
    v = torch.cat([v.clamp(-448, 448), table.float(), -table.float(),
                   ((table[1:] + table[:-1]) / 2).float()])
    assert torch.equal(ref.nearest_code(v.double()).to(torch.uint8), v.to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("square", [False, True])
def test_reference_codes_are_within_half_a_step(square):
    g = torch.Generator().manual_seed(1)
    x = torch.randn((150, 300), generator=g) * torch.exp(3 * torch.randn((150, 1), generator=g))
    codes, scales = ref.quantize(x, square)
    v = ref.values(codes.view(torch.float8_e4m3fn), scales, square)
    s = scales.repeat_interleave(128, 0).repeat_interleave(128, 1)[:150, :300] if square else \
        scales.t().repeat_interleave(128, 1)[:, :300]
    # half a step: 2^-4 of the value, or of the smallest step 2^-9 of the scale
    assert bool(((v - x.double()).abs() <= torch.maximum(x.double().abs() / 16, s * 2.0 ** -10)).all())
    again, s2 = ref.quantize(v, square)
    assert torch.equal(ref.values(again.view(torch.float8_e4m3fn), s2, square), v)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_reference_route_gradient_against_differences(score, renorm):
    g = torch.Generator().manual_seed(2)
    l = torch.randn((4, 9), generator=g, dtype=torch.float64)
    index = torch.argsort(torch.rand((4, 9), generator=g), dim=1)[:, :3]
    d = torch.randn((4, 3), generator=g, dtype=torch.float64)
    got, size = ref.route_grad(l, index, d, score, renorm, 1.5)
    loss = lambda v: float((ref.route_weights(v, index, score, renorm, 1.5) * d).sum())  # noqa: E731
    for i in range(l.numel()):
        hi, lo = l.clone(), l.clone()
        hi.view(-1)[i] += 1e-5
        lo.view(-1)[i] -= 1e-5
        # central differences: 1e-10 of a third derivative, 1e-16 / 1e-5 of rounding
        assert abs(float(got.reshape(-1)[i]) - (loss(hi) - loss(lo)) / 2e-5) < 1e-8
    assert bool((got.abs() <= size + 1e-15).all())


def test_reference_combine_gradient_against_differences():
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    rows, w, x, d = r(7, 5), r(3, 2), r(3, 5), r(3, 5)
    slot = torch.tensor([[4, 0], [-1, 6], [2, -1]], dtype=torch.int32)
    d_rows, d_weight, _ = ref.combine_grad(d, rows, slot, w, torch.zeros(7, 5, dtype=torch.float64))
    loss = lambda rows, w: float((ref.combine(rows, slot, w, x)[0] * d).sum())  # noqa: E731
    for t, grad, f in ((rows, d_rows, lambda v: loss(v, w)), (w, d_weight, lambda v: loss(rows, v))):
        for i in range(t.numel()):
            hi, lo = t.clone(), t.clone()
            hi.view(-1)[i] += 1e-4
            lo.view(-1)[i] -= 1e-4
            # linear in either: rounding alone
            assert abs(float(grad.reshape(-1)[i]) - (f(hi) - f(lo)) / 2e-4) < 1e-10


def test_reference_route_is_a_sort():
    g = torch.Generator().manual_seed(4)
    l = torch.randn((20, 12), generator=g)
    index, weight, slot, source, offsets = ref.route(l, 3, score="sigmoid", renormalize=False)
    best = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :3]
    assert torch.equal(index, best.to(torch.int32))
    assert torch.allclose(weight, torch.sigmoid(l.double()).gather(1, best))
    assert int(offsets[-1]) == 60 and math.isclose(float(weight.sum()), float(torch.sigmoid(l.double()).gather(1, best).sum()))
    for t in range(20):
        for j in range(3):
            n = int(slot[t, j])
            assert int(source[n]) == t and int(offsets[index[t, j]]) <= n < int(offsets[index[t, j] + 1])
