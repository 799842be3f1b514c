"""Corners of the layer operators that their plain sizes do not reach: the tile
variants of large matrices, poisoned neighbours, reused stages of a ring, calls
after a bounded wait ran out, outputs in place of inputs.

Sizes are chosen for a device of 152 SMs (the variants go by the SM count)."""
import pytest
import torch

import dense_gemm_07_gb300 as g7
from dense_gemm_07_gb300 import _abi
from layer_reference import EPS32, w4_weights
from test_gpu_layer import (_check_grads, _close, _gen, _norm_case, _norm_ref, _randn, _strided,
                            _w4_case, _w4_tol)

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------- 4-bit weights

# K ends in the first group of its last 128 rows, and a warp's ring comes round
# to a stage that held groups of the matrix.
@pytest.mark.parametrize("M,K,N,group", [
    (1, 8256, 9729, 64), (2, 8256, 5001, 64), (4, 8225, 5001, 32), (3, 8225, 9729, 32),
    (8, 8256, 9729, 64), (5, 320, 9729, 64), (7, 8225, 9729, 32), (6, 8256, 5001, 64),
    (16, 8256, 5001, 64), (16, 8225, 5001, 32), (12, 2112, 401, 64)])
def test_w4_groups_past_the_matrix_add_nothing(M, K, N, group):
    """The groups that fill up the last 128 rows weigh nothing, whatever scales a
    column's neighbours, its other groups or the gaps between rows hold: a column
    of NaN scales is NaN and changes no other, one of infinite scales (positive
    products) is infinite."""
    a, codes, scales, _ = _w4_case(M + K, M, K, N, group, False)
    a = a.abs() + 1.0
    nan, inf = N // 3, N - 2
    codes[:, inf] = 15
    packed = g7.w4_pack(codes)
    clean = g7.gemm_w4(a, packed, scales, group=group)
    poisoned = scales.clone()
    poisoned[:, nan] = float("nan")
    poisoned[:, inf] = float("inf")
    # rows an odd number of elements apart, NaN between them
    out = g7.gemm_w4(a, packed, _strided(poisoned, 2), group=group)
    assert bool(out[:, nan].isnan().all())
    assert bool((out[:, inf] == float("inf")).all())
    rest = [c for c in range(N) if c not in (nan, inf)]
    assert torch.equal(out[:, rest], clean[:, rest])


# One tile of columns a warp, two, and four: N at the limits between them (4848 and
# 9712 columns on 152 SMs) and odd remainders of a warp's tiles; K in one step, in
# three, and cut over the blocks of a cluster.
@pytest.mark.parametrize("M", [1, 4, 5, 8, 9, 16])
@pytest.mark.parametrize("K,N", [(129, 4853), (320, 9729), (33, 9713), (1100, 4848), (257, 16401)])
@pytest.mark.parametrize("group,zeros", [(32, False), (64, True), (128, False), (32, True)])
def test_w4_of_wide_matrices(M, K, N, group, zeros):
    a, codes, scales, z = _w4_case(M * 31 + N, M, K, N, group, zeros)
    out = g7.gemm_w4(a, g7.w4_pack(codes), scales, zeros=z, group=group)
    w = w4_weights(codes, scales, z, group)
    _close(out, a.double() @ w, _w4_tol(a, w, K, group, out), "product")


# ------------------------------------------------------------------- norms

@pytest.mark.parametrize("D", [77, 520, 5000])
@pytest.mark.parametrize("gate", ["none", "channel", "row", "full"])
def test_norm_gate_bwd_without_norms_does_not_look_at_y(D, gate):
    """Without post norm and pre norm dy = gate * d_x_out: a value of y that is not
    finite stays out of it."""
    T = 6
    c = _norm_case(D, T, D, F32, F32, gate, post=False, pre=False)
    w = _randn(_gen(D), T, D)
    want = g7.gemm_norm_gate_bwd(**c, d_x_out=w)
    c["y"][1, 3], c["y"][4, D - 1] = float("inf"), float("nan")
    got = g7.gemm_norm_gate_bwd(**c, d_x_out=w)
    assert torch.equal(got.dy, want.dy) and torch.equal(got.dx, want.dx)
    gates = torch.ones((), device="cuda") if c["gate"] is None else c["gate"]
    assert torch.equal(got.dy, (gates * w).to(BF16))


@pytest.mark.parametrize("T,D,extra", [(9, 520, 8), (9, 520, 3), (5, 77, 1), (1, 64, 5), (6, 1, 2),
                                       (3, 5000, 16)])
def test_norm_gate_takes_a_gate_of_any_row_stride(T, D, extra):
    """A gate per element is a matrix like the others; its gradient has its shape."""
    c = _norm_case(D, T, D, BF16, F32, "full")
    dxo, dh = _randn(_gen(1), T, D, dtype=BF16), _randn(_gen(2), T, D)
    s = dict(c, gate=_strided(c["gate"], extra))
    # (rows off the 16-byte grid are summed in another order: half a unit of BF16)
    for got, want in zip(g7.gemm_norm_gate(**s), g7.gemm_norm_gate(**c)):
        assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -7, atol=1e-6)
    got = g7.gemm_norm_gate_bwd(**s, d_x_out=dxo, d_h=dh)
    want = g7.gemm_norm_gate_bwd(**c, d_x_out=dxo, d_h=dh)
    assert got.dgate.shape == (T, D)
    ref = _norm_ref(c, 1.0, 1e-6)
    _check_grads(got, ref, dxo, dh, BF16, D)
    _check_grads(want, ref, dxo, dh, BF16, D)


@pytest.mark.parametrize("D", [520, 77, 4096, 5000, 8192])
@pytest.mark.parametrize("place", ["x", "d_x_out"])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_norm_gate_bwd_in_place(D, place, xt):
    """dx may be x or d_x_out: enough rows that a block's copies run ahead."""
    T = 700
    c = _norm_case(D, T, D, xt, F32, "channel")
    dxo, dh = _randn(_gen(1), T, D, dtype=xt), _randn(_gen(2), T, D)
    want = g7.gemm_norm_gate_bwd(**c, d_x_out=dxo, d_h=dh)
    dx = c["x"] if place == "x" else dxo
    out = [torch.empty_like(t) for t in want]
    kind = _abi.TYPE_BF16 if xt == BF16 else _abi.TYPE_F32
    args = _abi.GemmNormGateArgs(
        T, D, c["x"].data_ptr(), D, kind, c["y"].data_ptr(), D, _abi.TYPE_F32,
        c["weight_post"].data_ptr(), c["gate"].data_ptr(), D, _abi.GATE_CHANNEL,
        c["weight_pre"].data_ptr(), 1.0, 1e-6)
    grads = _abi.GemmNormGateGrads(
        dxo.data_ptr(), D, dh.data_ptr(), D, _abi.TYPE_F32, dx.data_ptr(), D,
        out[1].data_ptr(), D, out[3].data_ptr(), out[2].data_ptr(), out[4].data_ptr())
    assert _abi.gemm_norm_gate_bwd(args, grads, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(dx, want.dx)
    assert all(torch.equal(a, b) for a, b in zip(out[1:], want[1:]))


def test_norm_gate_refuses_gates_with_gaps_or_overlaps():
    c = _norm_case(1, 5, 16, F32, F32, "none")
    for gate in (torch.ones((16, 2), device="cuda")[:, 0],       # per channel, every other value
                 torch.ones((5, 2), device="cuda")[:, :1],       # per row
                 torch.ones((1, 16), device="cuda").expand(5, 16),  # rows that overlap
                 torch.ones((5, 32), device="cuda")[:, ::2],
                 torch.ones((5, 16), device="cuda").to(BF16)):
        with pytest.raises((ValueError, TypeError)):
            g7.gemm_norm_gate(c["x"], c["y"], gate=gate)


# ------------------------------------------------- 8-bit weight gradient

def _whole(seed, T, K, N):
    """A checkpoint of whole numbers (step 1), a dY and their exact gradient (every
    sum stays below 2^24)."""
    g = _gen(seed)
    x = torch.randint(-8, 9, (T, K), generator=g, device="cuda").float()
    x[::32] = 127.0
    dy = torch.randint(-3, 4, (T, N), generator=g, device="cuda").to(BF16)
    return g7.gemm_ckpt8_pack(x), dy, x.double().t() @ dy.double()


# (76 pairs) a second tile for some pairs, two and three whole waves; shared tiles
# alone, in two and in three parts; a whole wave before shared ones; rows that the
# copy engine cannot read in place
@pytest.mark.parametrize("T,K,N", [
    (130, 2560, 2100), (257, 4000, 2304), (640, 3900, 3841), (4096, 2816, 2048), (4100, 2700, 2041),
    (8448, 1000, 3001), (8700, 2048, 1536), (3500, 4096, 2560), (3521, 4090, 2501)])
def test_ckpt8_wgrad_of_many_tiles(T, K, N):
    kept, dy, want = _whole(T, T, K, N)
    got = g7.gemm_ckpt8_wgrad(kept, dy)
    assert torch.equal(got.double(), want)
    out = got.clone()
    g7.gemm_ckpt8_wgrad(kept, dy, out=out, beta=-2.0)
    assert torch.equal(out.double(), -want)
    # and within the bound of test_ckpt8_wgrad on values that round, bit for bit again
    x = _randn(_gen(T), T, K)
    dy = _randn(_gen(N), T, N, dtype=BF16)
    k = g7.gemm_ckpt8_pack(x)
    v = g7.gemm_ckpt8_unpack(k, F32).double()
    got = g7.gemm_ckpt8_wgrad(k, dy)
    units = 64 + 2 * (T // 512 + 2)
    _close(got, v.t() @ dy.double(), units * EPS32 * (v.abs().t() @ dy.double().abs()) + 1e-37)
    assert torch.equal(got, g7.gemm_ckpt8_wgrad(k, dy))


# one tile in two parts; tiles in two and three parts; more tiles than pairs, whose
# parts are summed one early and one late in the launch
@pytest.mark.parametrize("T,K,N", [(4096, 128, 256), (8448, 1000, 3001), (4096, 2816, 2048)])
def test_calls_after_one_pair_gave_up_are_exact(T, K, N):
    """One pair's first copy is withheld: it gives up, and the pairs that share
    its tiles have counted their parts.  The calls after it find no trace of that,
    nor does the gradient through an activation, which counts in the same words."""
    first, second = _whole(1, T, K, N), _whole(2, T, K, N)
    z = [_randn(_gen(s), 512, 8192) for s in (3, 4)]
    kept = [g7.gemm_ckpt8_pack(v) for v in z]
    dbias = [g7.gemm_ckpt8_act_grad(v, k, "relu")[1] for v, k in zip(z, kept)]
    for after in ("wgrad", "act_grad"):
        assert torch.equal(g7.gemm_ckpt8_wgrad(*first[:2]).double(), first[2])
        try:
            assert _abi.gemm_debug_inject(2, 2_000_000) == _abi.GEMM_OK
            g7.gemm_ckpt8_wgrad(*first[:2])
            assert g7.gemm_get_device_status() == _abi.GEMM_ERR_TIMEOUT
        finally:
            assert _abi.gemm_debug_inject(0, 0) == _abi.GEMM_OK
        for i in range(2):
            if after == "act_grad":
                assert torch.equal(g7.gemm_ckpt8_act_grad(z[i], kept[i], "relu")[1], dbias[i])
            x, dy, want = (second, first)[i]
            assert torch.equal(g7.gemm_ckpt8_wgrad(x, dy).double(), want)
    assert g7.gemm_get_device_status() == _abi.GEMM_OK
