"""The layer operators called by several host threads at once through the C ABI
(ctypes releases the interpreter's lock for a call), each thread on a stream of its
own and with sizes of its own: a kernel's launch needs another amount of shared
memory in every thread.  Every call is accepted and every result is the one of a
call alone."""
import threading

import pytest
import torch

import dense_gemm_07_gb300 as g7
from dense_gemm_07_gb300 import _abi
from test_gpu_layer import _gen, _norm_case, _randn, _w4_case

pytestmark = pytest.mark.gpu

F32 = torch.float32
REPS = 1500


def _together(calls):
    """Each of `calls` REPS times in a thread with a stream of its own."""
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    start, bad = threading.Barrier(len(calls)), []

    def work(call, stream):
        start.wait()
        for i in range(REPS):
            s = call(stream.cuda_stream)
            if s != _abi.GEMM_OK:
                bad.append((i, s))
                return

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad, bad
    assert g7.gemm_get_device_status() == 0


def test_w4_of_unlike_rows_from_host_threads():
    K, N, group = 1000, 200, 32
    calls, outs, wants = [], [], []
    for M in (1, 2, 3, 4):
        a, codes, scales, _ = _w4_case(M, M, K, N, group, False)
        packed = g7.w4_pack(codes)
        wants.append(g7.gemm_w4(a, packed, scales, group=group))
        out = torch.zeros_like(wants[-1])
        w = _abi.GemmW4(packed.data_ptr(), scales.data_ptr(), N, None, N, group)

        def call(stream, M=M, a=a, w=w, out=out, keep=(packed, scales)):
            return _abi.gemm_w4(M, N, K, a.data_ptr(), K, w, out.data_ptr(), N, _abi.TYPE_F32,
                                None, stream)
        calls.append(call)
        outs.append(out)
    _together(calls)
    for out, want in zip(outs, wants):
        assert torch.equal(out, want)


def test_norm_gradients_of_unlike_widths_from_host_threads():
    calls, outs, wants = [], [], []
    for D in (1024, 2048, 3000, 4096):
        T = 8
        c = _norm_case(D, T, D, F32, F32, "full")
        dxo, dh = _randn(_gen(D), T, D), _randn(_gen(D + 1), T, D)
        wants.append(g7.gemm_norm_gate_bwd(**c, d_x_out=dxo, d_h=dh))
        out = g7.NormGateGrads(*[torch.zeros_like(t) for t in wants[-1]])
        args = _abi.GemmNormGateArgs(
            T, D, c["x"].data_ptr(), D, _abi.TYPE_F32, c["y"].data_ptr(), D, _abi.TYPE_F32,
            c["weight_post"].data_ptr(), c["gate"].data_ptr(), D, _abi.GATE_FULL,
            c["weight_pre"].data_ptr(), 1.0, 1e-6)
        grads = _abi.GemmNormGateGrads(
            dxo.data_ptr(), D, dh.data_ptr(), D, _abi.TYPE_F32, out.dx.data_ptr(), D,
            out.dy.data_ptr(), D, out.dgate.data_ptr(), out.dweight_post.data_ptr(),
            out.dweight_pre.data_ptr())

        def call(stream, args=args, grads=grads, keep=(c, dxo, dh)):
            return _abi.gemm_norm_gate_bwd(args, grads, stream)
        calls.append(call)
        outs.append(out)
    _together(calls)
    for out, want in zip(outs, wants):
        assert all(torch.equal(a, b) for a, b in zip(out, want))
