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
from test_gpu_layer import _w4_case

pytestmark = pytest.mark.gpu

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

