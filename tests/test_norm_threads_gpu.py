"""Gated residual and norm called from several host threads at once, each on a stream of its own.

The widths share kernels but not the amount of shared memory that a launch asks for, so a call that left
its own amount behind as the kernel's limit would have another thread's launch refused. Every result has
to equal the one of a single thread, bit for bit.
"""
import threading

import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa

pytestmark = pytest.mark.gpu

CALLS = 3000
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build
    build.build()
    sa.load_library()


@pytest.mark.parametrize("dtype,widths", [(BF, (5120, 4096, 4608, 2560)), (F32, (4096, 3584, 2560, 5120)), (BF, (5119, 4095, 3001, 8191))])
def test_threads_on_their_own_streams(dtype, widths):
    g = torch.Generator(device="cuda").manual_seed(1)

    def r(*s):
        return torch.randn(s, generator=g, device="cuda").to(dtype)
    calls = []
    for C in widths:
        x, y, dh = r(1, 3, C), r(1, 3, C), r(1, 3, C)
        outs = [torch.empty_like(x) for _ in range(4)]
        calls.append((C, x, y, dh, outs))
    lib, code = sa.load_library(), sa._dtype_code(calls[0][1])

    def once(call, stream):
        """Forward and gradient through the C entry points: little else between two launches."""
        C, x, y, dh, (xo, h, dx, dy) = call
        st = lib.sol_attn_residual_norm(x.data_ptr(), y.data_ptr(), None, 0, None, None, 0, None, 0, None, code, 1, 0, 1.0, 1e-6,
                                        1, 3, C, xo.data_ptr(), h.data_ptr(), stream)
        if st == sa.SOL_OK:
            st = lib.sol_attn_residual_norm_bwd(dh.data_ptr(), None, x.data_ptr(), y.data_ptr(), None, 0, None, None, 0, None, code,
                                                1, 0, 1.0, 1e-6, 1, 3, C, dx.data_ptr(), dy.data_ptr(), None, None, None, None,
                                                None, None, 0, stream)
        return st
    want = []
    for c in calls:
        assert once(c, None) == sa.SOL_OK
        torch.cuda.synchronize()
        want.append([t.clone() for t in c[4]])
    refused = []
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(c, s):
        for i in range(CALLS):
            if once(c, s.cuda_stream) != sa.SOL_OK:
                refused.append((c[0], i, lib.sol_attn_last_error().decode()))
                return
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, refused
    for c, w in zip(calls, want):
        for got, ref in zip(c[4], w):
            assert torch.equal(got, ref), c[0]
