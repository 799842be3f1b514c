"""The operators of a layer of experts where a comparison, a mask or a tensor that the
call makes could go wrong unseen."""
import itertools

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import dense_gemm_07_gb300 as g7
import experts_reference as ref
from layer_reference import EPS32, act
from test_gpu_experts import (BF16, F32, INF, NAN, STEP, _check_route, _close, _experts_case, _gen,
                              _product_tol, _randn, _status)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- routing

def _pairs_of_near_sums(g, T, groups, score, spread):
    """Logits of `groups` groups of two experts whose scores add up to nearly the same in
    every group (times a common factor for softmax)."""
    a = 0.3 + 0.4 * torch.rand((T, groups), generator=g, device="cuda", dtype=torch.float64)
    d = spread * torch.randn((T, groups), generator=g, device="cuda", dtype=torch.float64)
    s = torch.stack([a, 1.0 + d - a], 2).view(T, 2 * groups)
    return (torch.logit(s) if score == "sigmoid" else torch.log(s)).float()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [32.0, 100.0, 3000.0])
@pytest.mark.parametrize("groups,kept", [(2, 1), (8, 3)])
def test_route_groups_whose_biases_cancel(score, size, groups, kept):
    """Biases of opposite sign leave a group's sum small, and its error as large as theirs."""
    g = _gen(int(size) + groups)
    sign = torch.tensor([size, -size], device="cuda").repeat(groups)
    unlike = sign * torch.repeat_interleave(1 + torch.arange(groups, device="cuda") % 3, 2)
    for spread, bias in itertools.product((1e-5, 1e-6 * size), (sign, unlike)):
        logits = _pairs_of_near_sums(g, 1500, groups, score, spread)
        _check_route(logits, min(3, 2 * kept), score=score, bias=bias, groups=groups,
                     groups_kept=kept, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("mask", [torch.finfo(F32).min, -2.5e38])
def test_route_groups_masked_by_the_bias(score, mask):
    """Two masks add up to less than FP32 holds: the group comes last, but it is there."""
    g = _gen(2)
    logits = _randn(g, 70, 24)
    logits[5, 8:12] = -INF                  # a closed group besides
    bias = _randn(g, 24, scale=0.1)
    for groups in ((0, 1, 2, 3, 4, 5), (1, 2, 4), (0, 1, 3, 4, 5)):
        masked = bias.clone()
        for i in groups:
            masked[4 * i:4 * i + 4] = mask
        for kept, k in ((1, 4), (3, 8), (5, 20)):
            _check_route(logits, k, score=score, bias=masked, groups=6, groups_kept=kept, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("alike,k,groups,kept", [(2, 1, 1, 1), (3, 2, 1, 1), (5, 1, 1, 1), (34, 32, 1, 1), (4, 3, 2, 1)])
def test_route_equal_experts_before_a_near_one(score, alike, k, groups, kept):
    """The last one chosen ties with the next, and a third one, behind both in FP32, is
    ahead of them in 64 bits."""
    g = _gen(alike)
    E = 2 * alike + 2
    one = _randn(g, 1, E)
    one[:, :alike] = one[:, :1]
    logits = one + 1e-7 * _randn(g, 1500, E)
    logits[:, :alike] = logits[:, :1]       # experts that are the same in everything
    s = torch.softmax(one.double(), 1) if score == "softmax" else torch.sigmoid(one.double())
    bias = (1.5 - s[0]).float()
    bias[alike + 1:] -= 3.0                 # one expert is near them, the others are not
    _check_route(logits, k, score=score, bias=bias, groups=groups, groups_kept=kept)


def test_route_all_places_taken():
    """32 chosen experts with a bias, near ties at the last place among them."""
    g = _gen(8)
    for E in (32, 33, 70, 300):
        logits = _randn(g, 200, E)
        bias = _randn(g, E, scale=0.3)
        near = (1.5 - torch.sigmoid(logits[:1].double()))[0].float()
        for b in (bias, torch.zeros_like(bias), near):
            _check_route(logits, 32, score="sigmoid", bias=b)
            _check_route(logits[:1] + 1e-7 * _randn(g, 200, E), 32, score="sigmoid", bias=b)


def test_route_logits_whose_scores_are_equal():
    """Sigmoids that are 1, and softmax scores that are 0, in 64 bits too: without a bias
    the logits tell experts, and groups of one expert each, apart."""
    up = torch.tensor([[40.0, 50.0, 41.0, 60.0, -1.0, 70.0]], device="cuda")
    down = torch.tensor([[-900.0, -950.0, -990.0, -800.0, 3.0, -801.0]], device="cuda")
    for logits, score in ((up, "sigmoid"), (down, "softmax"), (down, "sigmoid")):
        want = logits.sort(dim=1, descending=True).indices
        r = g7.gemm_route(logits, 4, score=score)
        assert r.index.tolist() == want[:, :4].tolist(), score
        best = logits.view(3, 2).amax(1).sort(descending=True).indices[:2].tolist()
        inside = [e for e in want[0].tolist() if e // 2 in best]
        r = g7.gemm_route(logits, 4, score=score, groups=3, groups_kept=2, group_top=1)
        assert r.index[0].tolist() == inside, score


@pytest.mark.parametrize("low", [-30.0, -900.0, torch.finfo(F32).min])
def test_route_chosen_scores_that_leave_64_bits(low):
    """Renormalised softmax weights are a softmax over the chosen, however far below the
    largest logit they are, whichever precision chose them; their gradient is that's."""
    logits = torch.full((6, 4), low, device="cuda")
    logits[:, 0] = 1.0
    logits[:, 2] -= 1.0
    want = torch.softmax(logits[:, 1:3].double(), 1)
    d = torch.tensor([[1.0, -2.0]], device="cuda").repeat(6, 1)
    for near in (0.5, 0.25):            # (equal biases: scores of 0 that FP32 cannot tell)
        bias = torch.tensor([-INF, 0.5, near, -4.0], device="cuda")
        r = g7.gemm_route(logits, 2, bias=bias)
        assert r.index.tolist() == [[1, 2]] * 6
        _close(r.weight, want, 8 * EPS32 * want, near)
        got = g7.gemm_route_bwd(logits, r.index, d)
        grad = want * (d.double() - (d.double() * want).sum(1, keepdim=True))
        full = torch.zeros(6, 4, dtype=torch.float64, device="cuda")
        full[:, 1:3] = grad
        _close(got, full, 16 * EPS32 * full.abs(), near)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_route_gradient_of_closed_experts(score, dtype):
    """Experts whose logits are all -infinity have weights of 0, and gradients of 0."""
    g = _gen(5)
    logits = _randn(g, 20, 40, dtype=dtype)
    logits[3] = -INF
    logits[4, :8] = -INF
    index = torch.arange(8, dtype=torch.int32, device="cuda").repeat(20, 1)
    index[3, 2], index[4, 5] = -1, 3
    d = _randn(g, 20, 8)
    for renorm in (True, False):
        got = g7.gemm_route_bwd(logits, index, d, score=score, renormalize=renorm)
        zero = torch.zeros_like(got[3:5])
        assert torch.equal(got[3:5], zero), renorm
        kept = [i for i in range(20) if i not in (3, 4)]
        want = g7.gemm_route_bwd(logits[kept], index[kept], d[kept], score=score, renormalize=renorm)
        assert torch.equal(got[kept], want) and bool((want != 0).any(1).all())


# -------------------------------------------- tensors that the call makes

def _leave(value, *shapes):
    """Leaves a value in memory that the next tensors of these shapes are likely to get."""
    blocks = [torch.full(s, value, dtype=d, device="cuda") for s, d in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("D", [64, 1000, 3001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_combine_gradient_of_rows_without_a_slot(D, dtype):
    """A new d_rows has zeros in rows that no slot names; one that is passed keeps them."""
    g = _gen(D)
    logits = _randn(g, 40, 12)
    logits[30:] = -INF
    r = g7.gemm_route(logits, 3)
    rows, d = _randn(g, 120, D, dtype=dtype), _randn(g, 40, D)
    slot = r.slot.clone()
    slot[2] = -1
    named = torch.zeros(120, dtype=torch.bool, device="cuda")
    named[slot[slot >= 0].long()] = True
    old = _randn(g, 120, D, dtype=dtype)
    want, dw = g7.gemm_combine_bwd(d, rows, slot, r.weight, d_rows=old.clone())
    assert torch.equal(want[~named], old[~named])
    want[~named] = 0
    other = torch.cuda.Stream()
    for stream in (None, other):
        for _ in range(3):
            _leave(NAN, ((120, D), dtype), ((40, 3), F32))
            other.wait_stream(torch.cuda.current_stream())
            got, w = g7.gemm_combine_bwd(d, rows, slot, r.weight, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got, want) and torch.equal(w, dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, w = g7.gemm_combine_bwd(d, rows, slot, r.weight)
    for _ in range(2):
        got.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(w, dw)
    # no slot at all
    none = torch.full_like(slot, -1)
    _leave(NAN, ((120, D), dtype))
    got, w = g7.gemm_combine_bwd(d, rows, none, r.weight)
    assert torch.equal(got, torch.zeros_like(got)) and torch.equal(w, torch.zeros_like(w))
    empty = torch.empty((40, 0), dtype=torch.int32, device="cuda")
    _leave(NAN, ((120, D), dtype))
    got, _ = g7.gemm_combine_bwd(d, rows, empty, empty.float())
    assert torch.equal(got, torch.zeros_like(got))


class _Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.names = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.names.append(str(func))
        return func(*args, **(kwargs or {}))


def _calls(stream=None):
    """What makes its own tensors, of the operators with rows that a call leaves alone
    first: their names and outputs."""
    g = _gen(9)
    x, rows = _randn(g, 50, 256, dtype=BF16), _randn(g, 150, 64)
    logits = _randn(g, 50, 8)
    logits[40:] = -INF
    r = g7.gemm_route(logits, 3)
    a = g7.gemm_fp8_quantize(x, index=r.source)
    w = g7.gemm_fp8_quantize(_randn(g, 8, 96, 256), square=True)
    few = g7.gemm_fp8_quantize(_randn(g, 96, 256), square=True)
    n = int(r.offsets[-1])
    torch.cuda.synchronize()

    def experts():
        out = g7.gemm_fp8_experts(a, w, r.offsets, stream=stream)
        return out[:n], out[n:]

    return experts, dict(
        route=lambda: g7.gemm_route(logits, 3, stream=stream),
        quantize=lambda: g7.gemm_fp8_quantize(x, transpose=True, stream=stream)[:2],
        fp8=lambda: (g7.gemm_fp8(a, few, stream=stream),),
        route_bwd=lambda: (g7.gemm_route_bwd(logits, r.index, r.weight, stream=stream),),
        combine=lambda: (g7.gemm_combine(rows, r.slot, r.weight, stream=stream),),
        combine_bwd=lambda: g7.gemm_combine_bwd(rows[:50], rows, r.slot, r.weight, stream=stream),
        norm=lambda: (g7.gemm_norm_gate(x, x, stream=stream)[0],),
        ckpt8=lambda: g7.gemm_ckpt8_pack(x.float(), activation="gelu", stream=stream)[1:])


def _same(u, v):
    as_bytes = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    return torch.equal(as_bytes(u), as_bytes(v))


@pytest.mark.parametrize("other", [False, True])
def test_new_tensors_are_filled_in_deterministic_mode(other):
    """torch's deterministic mode fills memory that nothing has been written to, on the
    stream that the call runs on; what a call writes is the same."""
    stream = torch.cuda.Stream() if other else None
    experts, calls = _calls(stream)
    want = {name: f() for name, f in calls.items()}
    written = experts()[0]
    torch.cuda.synchronize()
    torch.use_deterministic_algorithms(True)
    try:
        for _ in range(5):
            _leave(0.0, ((150, 96), F32))
            got, rest = experts()
            torch.cuda.synchronize()
            assert torch.equal(got, written) and rest.numel() > 0 and bool(rest.isnan().all())
            for name, f in calls.items():
                out = f()
                torch.cuda.synchronize()
                assert all(_same(u, v) for u, v in zip(out, want[name])), name
    finally:
        torch.use_deterministic_algorithms(False)


def test_new_tensors_are_seen_by_dispatch_modes():
    experts, calls = _calls()
    for name, f in [("experts", experts), *calls.items()]:
        want = f()
        with _Seen() as seen:
            got = f()
        assert any(n.startswith("aten.empty") for n in seen.names), (name, seen.names)
        assert all(_same(u, v) for u, v in zip(got, want) if u.numel() and name != "experts"), name


# ---------------------------------------------------------------- products

# rows an expert and columns on each side of the rules that choose the tiles
SEGMENTS = [([10, 20, 6], 200, 256), ([3] * 70, 130, 640), ([40, 2, 60], 257, 1024),
            ([100, 200, 60], 4100, 256), ([70] * 40, 300, 200), ([128, 1, 129, 0, 256], 2100, 385),
            ([300, 20, 0, 700, 1], 1300, 640), ([1000], 2200, 300), ([257, 255, 511, 513, 2, 90], 1100, 300)]


@pytest.mark.parametrize("lengths,N,K", SEGMENTS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_outside_the_offsets_stay(lengths, N, K, dtype):
    """Rows that no expert has are left as they were, and offsets that make no sense are
    held to the rows there are and to their running maximum."""
    E, M = len(lengths), sum(lengths)
    g, a, b, offsets = _experts_case(E + K, lengths, N, K)
    va, vb = ref.values(*a), ref.values(*b)
    good = offsets.tolist()
    inner = [good[1], *good[1:-1], good[-2]]            # rows before and behind the experts'
    wild = [-7, *good[1:]]
    wild[E // 2] = wild[max(E // 2 - 1, 0)] - 1         # one goes back
    wild[-1] = 2 ** 31 - 1
    back = [v if i % 2 else -2 ** 31 for i, v in enumerate(good)]
    for given in (good, inner, wild, back, [M + 9] * (E + 1), [0] * (E + 1), [M] + [0] * E):
        held, top = [], 0
        for v in given:
            top = max(top, min(max(v, 0), M))
            held.append(top)
        old = _randn(g, M, N, dtype=dtype)
        out = g7.gemm_fp8_experts(a, b, torch.tensor(given, dtype=torch.int32, device="cuda"),
                                  out=old.clone(), alpha=2.0, beta=0.5)
        want, tol = old.double(), torch.zeros((M, N), dtype=torch.float64, device="cuda")
        for e in range(E):
            r = slice(held[e], held[e + 1])
            v = va[r] @ vb[e].t()
            want[r] = 2.0 * v + 0.5 * old[r].double()
            size = 2.0 * _product_tol(va[r], vb[e], K) + 4 * EPS32 * (2 * v.abs() + old[r].double().abs())
            tol[r] = size + STEP[dtype] * (want[r].abs() + size)
        _close(out, want, tol, str(given[:8]))
    _status()


@pytest.mark.parametrize("M,N,K", [(1, 16400, 640), (16, 16384, 512), (64, 16385, 300), (65, 15700, 300),
                                   (128, 15500, 256)])
def test_few_rows_of_many_columns(M, N, K):
    """On each side of the rule by rows; one expert with all rows is the same product."""
    g, a, b, offsets = _experts_case(M, [M], N, K)
    va, vb = ref.values(*a), ref.values(*b)[0]
    bias = _randn(g, 1, N)
    want, tol = va @ vb.t() + bias.double(), _product_tol(va, vb, K)
    tol = tol + 4 * EPS32 * ((va @ vb.t()).abs() + bias.double().abs())
    dense = g7.gemm_fp8(a, g7.Fp8(b.codes[0], b.scales[0], True), bias=bias[0])
    _close(dense, want, tol, "dense")
    _close(g7.gemm_fp8_experts(a, b, offsets, bias=bias), want, tol, "experts")
    _status()


@pytest.mark.parametrize("M,N,K", [(8, 300, 2000), (16, 128, 640), (600, 4100, 300)])
def test_one_expert_with_all_rows_is_the_dense_product(M, N, K):
    """On the same tiles with the same parts of K, so bit for bit."""
    g, a, b, offsets = _experts_case(M, [M], N, K)
    bias = _randn(g, 1, N)
    dense = g7.gemm_fp8(a, g7.Fp8(b.codes[0], b.scales[0], True), bias=bias[0], activation="gelu")
    assert torch.equal(g7.gemm_fp8_experts(a, b, offsets, bias=bias, activation="gelu"), dense)


@pytest.mark.parametrize("M,N", [(5, 3000), (200, 16400)])
@pytest.mark.parametrize("size", [2.0 ** -12, 2.0 ** -6, 1.0])
def test_gelu_of_both_kernels(M, N, size):
    """K = 1: a product of two codes is exact and its sum with the bias one rounding, so
    that the activation's argument is known; 2^-20 of it is allowed."""
    g = _gen(M)
    a = g7.gemm_fp8_quantize(_randn(g, M, 1))
    b = g7.gemm_fp8_quantize(_randn(g, N, 1), square=True)
    bias = _randn(g, N, scale=3.0 * size)
    b = g7.Fp8(b.codes, b.scales * size, True)
    v = (ref.values(*a) @ ref.values(*b).t()).float() + bias
    got = g7.gemm_fp8(a, b, bias=bias, activation="gelu")
    _close(got, act(v.double(), "gelu"), 2.0 ** -20 * v.double().abs() + 1e-40)


@pytest.mark.parametrize("M,N", [(5, 300), (200, 16400)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_activations_of_nan(M, N, dtype):
    """A block that was not finite is NaN, through GELU too; ReLU gives 0."""
    g = _gen(N)
    x = _randn(g, M, 200)
    x[1, 150], x[4, 3] = INF, NAN
    a, b = g7.gemm_fp8_quantize(x), g7.gemm_fp8_quantize(_randn(g, N, 200), square=True)
    rest = [i for i in range(M) if i not in (1, 4)]
    for kind in ("none", "gelu", "relu"):
        out = g7.gemm_fp8(a, b, activation=kind, out_dtype=dtype)
        bad = out[[1, 4]]
        assert bool((bad == 0).all() if kind == "relu" else bad.isnan().all()), kind
        assert not bool(out[rest].isnan().any())
