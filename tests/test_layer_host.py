"""The layer operators without a GPU: argument checks of the C entry points (made
before any device is looked for), the packed order, the checkpoint's step, and
the 64-bit reference forms against differences."""
import ctypes

import pytest
import torch

import dense_gemm_07_gb300 as g7
from dense_gemm_07_gb300 import _abi
from layer_reference import Norm, act, act_slope, kept

INVALID = _abi.GEMM_ERR_INVALID_ARG
P = 256  # a 16-byte aligned address that no check dereferences


@pytest.fixture(scope="module", autouse=True)
def lib():
    return _abi.lib()


def _w4(**kw):
    d = dict(packed=P, scales=P, ld_scales=64, zeros=None, ld_zeros=64, group=128)
    d.update(kw)
    return _abi.GemmW4(*[d[n] for n, _ in _abi.GemmW4._fields_])


def test_sizes():
    assert _abi.gemm_w4_packed_bytes(128, 16) == 1024
    assert _abi.gemm_w4_packed_bytes(129, 17) == 4096
    assert _abi.gemm_w4_packed_bytes(0, 17) == 0
    assert _abi.gemm_w4_packed_bytes(1, -1) == -1
    assert _abi.gemm_w4_packed_bytes(2 ** 31, 1) == -1
    assert _abi.gemm_ckpt8_bytes(33, 5) == 64 * 5
    assert _abi.gemm_ckpt8_bytes(0, 5) == 0
    assert _abi.gemm_ckpt8_bytes(-1, 5) == -1


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(M=524281), dict(N=2 ** 31), dict(K=-5), dict(lda=127), dict(ldc=63), dict(A=None),
    dict(C=None), dict(c_type=2), dict(w=None), dict(w=_w4(group=96)), dict(w=_w4(packed=None)),
    dict(w=_w4(packed=P + 8)), dict(w=_w4(scales=None)), dict(w=_w4(ld_scales=63)),
    dict(w=_w4(zeros=P, ld_zeros=1)), dict(epi=_abi.GemmEpilogue(1.0, 0.0, None, 9)),
    dict(lda=2 ** 61)])
def test_w4_refusals(change):
    a = dict(M=4, N=64, K=128, A=P, lda=128, w=_w4(), C=P, ldc=64, c_type=0, epi=None)
    a.update(change)
    assert _abi.gemm_w4(*a.values(), None) == INVALID


def test_w4_helpers_refuse():
    assert _abi.gemm_w4_pack(8, 8, None, 8, P, None) == INVALID
    assert _abi.gemm_w4_pack(8, 8, P, 7, P, None) == INVALID
    assert _abi.gemm_w4_pack(8, 8, P, 8, P + 4, None) == INVALID
    assert _abi.gemm_w4_quantize(8, 8, 31, P, 8, 0, P, P, 8, None, 8, None) == INVALID
    assert _abi.gemm_w4_quantize(8, 8, 32, P, 8, 5, P, P, 8, None, 8, None) == INVALID
    assert _abi.gemm_w4_quantize(8, 8, 32, None, 8, 0, P, P, 8, None, 8, None) == INVALID
    assert _abi.gemm_w4_unpack(8, 64, _w4(), None, 64, None) == INVALID
    assert _abi.gemm_w4_unpack(8, 64, _w4(), P, 63, None) == INVALID


def _norm(**kw):
    d = dict(T=4, D=16, x=P, ldx=16, x_type=0, y=P, ldy=16, y_type=0, w_post=P, gate=None,
             ld_gate=16, gate_mode=0, w_pre=P, alpha=1.0, eps=0.0)
    d.update(kw)
    return _abi.GemmNormGateArgs(*[d[n] for n, _ in _abi.GemmNormGateArgs._fields_])


BAD_NORMS = [dict(T=-1), dict(D=0), dict(D=_abi.NORM_MAX_WIDTH + 1), dict(x=None), dict(ldx=15),
             dict(x_type=3), dict(y_type=-1), dict(ldy=1), dict(y=None),
             dict(gate=P), dict(gate_mode=1), dict(gate=P, gate_mode=4),
             dict(gate=P, gate_mode=3, ld_gate=15), dict(eps=-1.0), dict(eps=float("nan"))]


@pytest.mark.parametrize("change", BAD_NORMS)
def test_norm_refusals(change):
    assert _abi.gemm_norm_gate(_norm(**change), P, 16, P, 16, None) == INVALID


def test_norm_output_refusals():
    assert _abi.gemm_norm_gate(_norm(), P, 15, P, 16, None) == INVALID
    assert _abi.gemm_norm_gate(_norm(), P, 16, P, 15, None) == INVALID
    assert _abi.gemm_norm_gate(_norm(), P, 16, None, 16, None) == INVALID
    assert _abi.gemm_norm_gate(_norm(w_pre=None), P, 16, P, 16, None) == INVALID
    assert _abi.gemm_norm_gate(None, P, 16, P, 16, None) == INVALID


def _grads(**kw):
    d = dict(d_x_out=P, ld_d_x_out=16, dh=P, ld_dh=16, dh_type=0, dx=P, ld_dx=16, dy=P, ld_dy=16,
             dgate=None, dw_post=P, dw_pre=P)
    d.update(kw)
    return _abi.GemmNormGateGrads(*[d[n] for n, _ in _abi.GemmNormGateGrads._fields_])


@pytest.mark.parametrize("change", [
    dict(dh=None), dict(dx=None), dict(dy=None), dict(dgate=P), dict(dw_post=None),
    dict(dw_pre=None), dict(ld_dx=3), dict(ld_dh=3), dict(dh_type=7), dict(ld_d_x_out=2),
    dict(ld_dy=15)])
def test_norm_bwd_refusals(change):
    assert _abi.gemm_norm_gate_bwd(_norm(), _grads(**change), None) == INVALID
    assert _abi.gemm_norm_gate_bwd(_norm(), None, None) == INVALID


def test_ckpt_refusals():
    pack, unpack = _abi.gemm_ckpt8_pack, _abi.gemm_ckpt8_unpack
    grad, wgrad = _abi.gemm_ckpt8_act_grad, _abi.gemm_ckpt8_wgrad
    assert pack(4, 8, None, 8, 0, P, P, 0, None, 8, None) == INVALID
    assert pack(4, 8, P, 7, 0, P, P, 0, None, 8, None) == INVALID
    assert pack(4, 8, P, 8, 2, P, P, 0, None, 8, None) == INVALID
    assert pack(4, 8, P, 8, 0, P + 1, P, 0, None, 8, None) == INVALID
    assert pack(4, 8, P, 8, 0, P, None, 0, None, 8, None) == INVALID
    assert pack(4, 8, P, 8, 0, P, P, 3, P, 8, None) == INVALID
    assert pack(4, 8, P, 8, 0, P, P, 0, P, 7, None) == INVALID
    assert unpack(4, 8, P, P, None, 8, 0, None) == INVALID
    assert unpack(4, 8, P, P, P, 8, 9, None) == INVALID
    assert grad(4, 8, P, 8, 0, P, P, 5, P, 8, None, None) == INVALID
    assert grad(4, 8, P, 8, 0, None, P, 1, P, 8, None, None) == INVALID
    assert grad(4, 8, P, 8, 0, P, P, 1, None, 8, None, None) == INVALID
    assert wgrad(4, 8, 8, P, P, P, 7, P, 8, 0.0, None) == INVALID
    assert wgrad(4, 8, 8, P, P, None, 8, P, 8, 0.0, None) == INVALID
    assert wgrad(4, 8, 8, P, P, P, 8, None, 8, 0.0, None) == INVALID
    assert wgrad(4, 8, 8, P + 8, P, P, 8, P, 8, 0.0, None) == INVALID


def test_nothing_to_do_needs_no_gpu():
    assert _abi.gemm_w4(0, 64, 128, None, 128, _w4(), None, 64, 0, None, None) == _abi.GEMM_OK
    assert _abi.gemm_ckpt8_pack(0, 8, None, 8, 0, None, None, 0, None, 8, None) == _abi.GEMM_OK
    assert _abi.gemm_ckpt8_wgrad(5, 0, 8, None, None, None, 8, None, 8, 0.0, None) == _abi.GEMM_OK
    assert _abi.gemm_norm_gate(_norm(T=0, x=None), None, 16, None, 16, None) == _abi.GEMM_OK


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError):
        g7.gemm_norm_gate(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        g7.gemm_ckpt8_pack(torch.zeros(2, 8))


def test_structs_match_the_header():
    assert ctypes.sizeof(_abi.GemmW4) == 48
    assert ctypes.sizeof(_abi.GemmNormGateArgs) == 112
    assert ctypes.sizeof(_abi.GemmNormGateGrads) == 96


def test_kept_is_within_half_a_step():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((100, 40), generator=g) * torch.exp(5 * torch.randn((1, 40), generator=g))
    v = kept(x)
    top = torch.nn.functional.pad(x.double(), (0, 0, 0, 28)).view(4, 32, 40).abs().amax(1)
    top = top.repeat_interleave(32, 0)[:100]
    # the step is below 2 * max / 127, so half of it is below max / 127
    assert bool(((v - x.double()).abs() <= top / 127 + 1e-45).all())
    assert torch.equal(kept(v), v)


@pytest.mark.parametrize("gate", [None, "channel", "row", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False)])
def test_reference_gradient_against_differences(gate, post, pre):
    g = torch.Generator().manual_seed(1)
    T, D, a, eps = 3, 10, 0.75, 1e-3
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    v = dict(x=r(T, D), y=r(T, D), w_post=r(D) if post else None,
             gate=None if gate is None else r(*{"channel": (D,), "row": (T, 1), "full": (T, D)}[gate]),
             w_pre=r(D) if pre else None)
    c1, c2 = r(T, D), r(T, D)

    def loss(**new):
        n = Norm(**dict(v, **new), alpha=a, eps=eps)
        return (n.u * c1).sum() + ((n.h * c2).sum() if pre else 0.0)

    got, _ = Norm(**v, alpha=a, eps=eps).backward(c1, c2 if pre else None)
    names = dict(x="dx", y="dy", w_post="dw_post", gate="dgate", w_pre="dw_pre")
    for name, t in v.items():
        if t is None:
            continue
        num = torch.empty_like(t)
        for i in range(t.numel()):
            hi, lo = t.clone(), t.clone()
            hi.view(-1)[i] += 1e-5
            lo.view(-1)[i] -= 1e-5
            num.view(-1)[i] = (loss(**{name: hi}) - loss(**{name: lo})) / 2e-5
        # central differences: 1e-10 of a third derivative, 1e-16 / 1e-5 of rounding
        assert torch.allclose(got[names[name]].reshape(t.shape), num, rtol=1e-6, atol=1e-6), name


def test_reference_slope_against_differences():
    v = torch.linspace(-5, 5, 101, dtype=torch.float64) + 0.01
    for kind in ("relu", "gelu", "none"):
        num = (act(v + 1e-5, kind) - act(v - 1e-5, kind)) / 2e-5
        assert torch.allclose(act_slope(v, kind), num, atol=1e-8)
