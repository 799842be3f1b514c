"""The operators of a layer of experts as they are used: together, on other streams, in
graphs, from several host threads, after a wait that ran out, and past 2^31 elements."""
import threading

import pytest
import torch

import dense_gemm_07_gb300 as g7
import experts_reference as ref
from dense_gemm_07_gb300 import _abi, experts_example
from layer_reference import act
from test_gpu_experts import (BF16, F32, INF, _close, _experts_case, _gen, _product_case,
                              _product_tol, _randn, _status)

pytestmark = pytest.mark.gpu


def _layer64(e, x, r):
    """The layer in 64 bits from the same choice of experts: out as a function of double
    leaves, for autograd."""
    leaves = {k: v.double().requires_grad_() for k, v in
              dict(x=x, router=e.router, w1=e.w1, w2=e.w2, b1=e.b1).items()}
    index = r.index.long()
    on = index >= 0
    logits = leaves["x"] @ leaves["router"]
    s = torch.where(on, torch.sigmoid(logits).gather(1, index.clamp(min=0)), 0.0)
    w = 1.5 * s / s.sum(1, keepdim=True).clamp(min=1e-300)
    out = leaves["x"]
    for i in range(e.w1.shape[0]):
        z = leaves["x"] @ leaves["w1"][i].t() + leaves["b1"][i]
        y = act(z, "gelu") @ leaves["w2"][i].t()
        out = out + torch.where(index == i, w, 0.0).sum(1, keepdim=True) * y
    return out, leaves


def test_layer_of_experts():
    """Rounding to 8 bits moves a factor by at most 2^-4 of itself, in the mean square by
    less than 2^-5.  out passes four such factors (x, W1, h, W2), a gradient at most six
    and one kept pre-activation; their errors are independent, so that the relative error
    in norm stays below sqrt(4) and sqrt(7) times 2^-5; twice that is allowed."""
    e = experts_example.Experts(256, 384, 8, 2, groups=4, groups_kept=2)
    g = _gen(0)
    x, d = _randn(g, 200, 256, dtype=BF16), _randn(g, 200, 256, dtype=BF16)
    open_ = torch.ones(200, dtype=torch.bool, device="cuda")
    open_[190:] = False
    out, grads = experts_example.train_step(e, x, d, open_)
    _, r = e.route(x, open_)
    want, leaves = _layer64(e, x, r)
    want.backward(d.double())

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())

    inner = want.detach() - x.double()
    assert off(out.double() - x.double(), inner) < 2 * 2 * 2.0 ** -5
    assert torch.equal(out[190:], x[190:])
    for name, leaf in leaves.items():
        got, ref_grad = grads[name], leaf.grad
        if name == "x":
            got, ref_grad = got.double() - d.double(), ref_grad - d.double()
        assert off(got, ref_grad) < 2 * 7 ** 0.5 * 2.0 ** -5, name
    serve = experts_example.serve_step(e, x, open_)
    assert off(serve.double() - x.double(), inner) < 2 * 2 * 2.0 ** -5
    assert torch.equal(serve, experts_example.serve_step(e, x, open_))
    _status()


def test_routed_rows_end_to_end_are_exact():
    """Route, pick, product and combine with whole numbers, where nothing is rounded: each
    token's rows come back to it."""
    g = _gen(5)
    T, E, k, K, N = 300, 16, 4, 256, 200
    x = torch.randint(-8, 9, (T, K), generator=g, device="cuda").to(BF16)
    x[:, ::128] = 448.0  # a block's scale is one
    w = torch.randint(-4, 5, (E, N, K), generator=g, device="cuda").to(BF16)
    w[:, ::128, ::128] = 448.0
    logits = _randn(g, T, E)
    r = g7.gemm_route(logits, k)
    y = g7.gemm_fp8_experts(g7.gemm_fp8_quantize(x, index=r.source),
                            g7.gemm_fp8_quantize(w, square=True), r.offsets)
    out = g7.gemm_combine(y, r.slot, torch.ones_like(r.weight))
    want = torch.zeros((T, N), dtype=torch.float64, device="cuda")
    for j in range(k):
        want += torch.einsum("tk,tnk->tn", x.double(), w.double()[r.index[:, j].long()])
    assert torch.equal(out.double(), want)


def test_example_runs(capsys):
    experts_example.main(["--tokens", "64", "--width", "256", "--hidden", "128", "--experts", "8",
                          "--chosen", "2"])
    assert "serve step" in capsys.readouterr().out


# ------------------------------------------------------------ streams and graphs

def test_on_another_stream():
    g = _gen(1)
    x, bias = _randn(g, 1000, 64), _randn(g, 64, scale=0.1)
    _, a, b, offsets = _experts_case(2, [40, 0, 300], 200, 384)
    want = g7.gemm_route(x, 6, score="sigmoid", bias=bias), g7.gemm_fp8_experts(a, b, offsets)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        r = g7.gemm_route(x, 6, score="sigmoid", bias=bias, stream=s)
        p = g7.gemm_fp8_experts(a, b, offsets, stream=s)
        # memory that the call has given back is taken and written on the current stream
        torch.full((4096,), 255, dtype=torch.uint8, device="cuda")
        s.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(r, want[0])) and torch.equal(p, want[1])
        torch.cuda.current_stream().wait_stream(s)


def test_graphs():
    """A captured step, replayed on new inputs, and two captured steps replayed at the same
    time on two streams."""
    e = experts_example.Experts(256, 256, 8, 2)
    g = _gen(3)
    static = [_randn(g, T, 256, dtype=BF16) for T in (16, 300)]
    experts_example.serve_step(e, static[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in static:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(experts_example.serve_step(e, x))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for i in range(5):
        for x in static:
            x.copy_(_randn(g, *x.shape, dtype=BF16))
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for x, out in zip(static, outs):
            assert torch.equal(out, experts_example.serve_step(e, x)), i
    _status()


def test_gradients_in_a_graph():
    g = _gen(4)
    logits = _randn(g, 50, 32)
    r = g7.gemm_route(logits, 3)
    d_w = _randn(g, 50, 3)
    rows, d = _randn(g, 150, 128, dtype=BF16), _randn(g, 50, 128)
    calls = lambda: (g7.gemm_route_bwd(logits, r.index, d_w),  # noqa: E731
                     *g7.gemm_combine_bwd(d, rows, r.slot, r.weight))
    want = calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_from_host_threads():
    """Calls of unlike sizes at once, each thread on a stream of its own."""
    cases, bad = [], []
    for i, (M, N, K, square) in enumerate([(1, 700, 640, True), (100, 300, 385, False),
                                           (600, 2048, 256, True), (30, 128, 1100, True)]):
        _, a, b = _product_case(i, M, N, K, square)
        x = _randn(_gen(i), 100 + 200 * i, 16 * (i + 1))
        cases.append((a, b, x, g7.gemm_fp8(a, b), g7.gemm_route(x, 3)))
    torch.cuda.synchronize()
    start = threading.Barrier(len(cases))

    def work(a, b, x, product, routing):
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            for _ in range(200):
                p, r = g7.gemm_fp8(a, b), g7.gemm_route(x, 3)
            stream.synchronize()
            if not torch.equal(p, product) or not all(torch.equal(u, v) for u, v in zip(r, routing)):
                bad.append(x.shape)

    threads = [threading.Thread(target=work, args=c) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    _status()


@pytest.mark.parametrize("M,N,K", [(4, 600, 2048), (100, 300, 1000), (1000, 2200, 640)])
def test_a_wait_that_runs_out(M, N, K):
    """The first stage of every block is never copied: its waits end, the status says so,
    and the next call is right."""
    _, a, b = _product_case(7, M, N, K, True)
    want = g7.gemm_fp8(a, b)
    for mode in (1, 2):
        assert g7.gemm_get_device_status() == 0
        assert _abi.gemm_debug_inject(mode, 5_000_000) == 0
        try:
            g7.gemm_fp8(a, b)
            status = g7.gemm_get_device_status()
            assert status == (_abi.GEMM_ERR_TIMEOUT if mode == 1 or M == 1000 else 0)
        finally:
            assert _abi.gemm_debug_inject(0, 0) == 0
        assert torch.equal(g7.gemm_fp8(a, b), want)
        assert g7.gemm_get_device_status() == 0


# ------------------------------------------------------------ the largest and the odd

def test_tensors_past_2_31_elements():
    """Rows whose offsets do not fit 32 bits: the last ones are the right ones."""
    T, D = 540_000, 4096  # 2.2e9 elements
    x = torch.zeros((T, D), dtype=BF16, device="cuda")
    g = _gen(6)
    x[-256:] = _randn(g, 256, D, dtype=BF16)
    q = g7.gemm_fp8_quantize(x)
    small = g7.gemm_fp8_quantize(x[-256:].clone())
    assert torch.equal(q.codes[-256:].view(torch.uint8), small.codes.view(torch.uint8))
    assert torch.equal(q.scales[:, -256:], small.scales)
    b = g7.gemm_fp8_quantize(_randn(g, 64, D), square=True)
    tail = g7.gemm_fp8(small, b)
    # (products of another number of rows share K among other blocks, so that their sums
    # are rounded in another order: both are within the bound of the exact one)
    tol = 2 * _product_tol(ref.values(*small), ref.values(*b), D)
    _close(g7.gemm_fp8(q, b)[-256:], tail.double(), tol)
    offsets = torch.tensor([0, T - 256, T], dtype=torch.int32, device="cuda")
    two = g7.Fp8(torch.stack([b.codes, b.codes]), torch.stack([b.scales, b.scales]), True)
    _close(g7.gemm_fp8_experts(q, two, offsets)[-256:], tail.double(), tol)
    del q
    slot = torch.tensor([[T - 1, 0], [T - 200, T - 7]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 1.0], [2.0, -1.0]], device="cuda")
    want, size = ref.combine(x[-256:], slot - (T - 256), w)
    _close(g7.gemm_combine(x, slot, w, out_dtype=F32), want, 4 * 2.0 ** -23 * size)
    d = _randn(g, 2, D, dtype=BF16)
    d_rows, _ = g7.gemm_combine_bwd(d, x, slot, w, d_rows=x)
    assert torch.equal(d_rows[T - 1], (0.5 * d[0].float()).to(BF16))
    _status()


def test_experts_with_many_experts_and_few_rows():
    g, a, b, offsets = _experts_case(8, [1 if i % 7 == 0 else 0 for i in range(1024)], 48, 128)
    va, vb = ref.values(*a), ref.values(*b)
    out = g7.gemm_fp8_experts(a, b, offsets)
    e = torch.arange(0, 1024, 7, device="cuda")
    want = torch.einsum("rk,rnk->rn", va, vb[e])
    _close(out, want, _product_tol(va[:, None], vb[e], 128)[:, 0])
    _, a, b, offsets = _experts_case(9, [130] * 40 + [0, 129, 257], 300, 200)
    va, vb, at = ref.values(*a), ref.values(*b), offsets.tolist()
    out = g7.gemm_fp8_experts(a, b, offsets)
    for i in range(43):
        r = slice(at[i], at[i + 1])
        _close(out[r], va[r] @ vb[i].t(), _product_tol(va[r], vb[i], 200))
    _status()


def test_masked_rows_have_no_gradient():
    """Closed experts (logit -inf) and tokens of padding."""
    g = _gen(9)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            logits = _randn(g, 40, 12)
            logits[:, 5] = -INF
            logits[30:] = -INF
            logits[3, 1:] = -INF
            r = g7.gemm_route(logits, 4, score=score, renormalize=renorm)
            d = g7.gemm_route_bwd(logits, r.index, _randn(g, 40, 4), score=score, renormalize=renorm)
            assert bool(torch.isfinite(d[:30]).all()) and float(d[:30, 5].abs().sum()) == 0
            assert float(d[30:].abs().sum()) == 0


