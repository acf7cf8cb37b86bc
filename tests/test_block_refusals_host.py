"""Calls of the dense operators that the host refuses because a kernel could not answer them rightly: nothing is
launched, no GPU is needed."""
import ctypes

import pytest

from block_sparse_attention_41_b200 import build as builder
from block_sparse_attention_41_b200 import sol_attn as sa

# fake, 16-byte aligned device addresses: validation must reject before any of them is used
P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(16)]
B16, F32 = sa.SOL_BF16, sa.SOL_F32


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return sa.load_library()


def _strides(v):
    return (ctypes.c_int64 * 3)(*v)


def rope(lib, B=2, Hq=3, Hk=2, L=4, d=64, qs=(768, 256, 64), ks=(512, 256, 64), qos=(768, 256, 64), kos=(512, 256, 64),
         pos_b=0, q=P[0], k=P[1], qo=P[2], ko=P[3]):
    """The status of a rotary call; SOL_ECUDA or SOL_EUNSUPPORTED of a machine without a B200 mean that its arguments passed."""
    return lib.sol_attn_rope(q, _strides(qs), k, _strides(ks), B16, P[4], pos_b, 1, None, P[5], 1.0, 0, 0, B, Hq, Hk, L, d, d, qo,
                             _strides(qos), ko, _strides(kos), None)


def refused(status):
    return status == sa.SOL_EINVAL


def host_only():
    import torch
    if torch.cuda.is_available():
        pytest.skip("the accepted calls have made-up addresses")


def test_rope_refuses_positions_before_their_buffer(lib):
    assert refused(rope(lib, pos_b=-1)) and refused(rope(lib, pos_b=-4))
    host_only()
    assert not refused(rope(lib, pos_b=0)) and not refused(rope(lib, pos_b=4))
    assert not refused(rope(lib, B=1, pos_b=-1))  # one entry: the stride is not used


def test_rope_refuses_outputs_whose_rows_overlap(lib):
    for bad in (dict(qos=(768, 64, 64)), dict(qos=(767, 256, 64)), dict(qos=(768, 255, 64)), dict(qos=(64, 64, 64)),
                dict(kos=(512, 64, 65)), dict(kos=(256, 256, 64)), dict(qos=(768, 256, 63)), dict(qos=(2**62, 256, 63)),
                dict(B=1, qos=(1, 64, 64)), dict(Hq=1, qos=(255, 1, 64)), dict(L=1, qos=(191, 64, 1)),
                dict(L=1, Hq=1 << 15, qos=(2**62, 2**62, 1), kos=(64, 64, 1))):
        assert refused(rope(lib, **bad)), bad
    host_only()
    for good in (dict(), dict(qos=(768, 64, 192)), dict(qos=(64, 512, 128)), dict(qos=(1000, 264, 66)),  # b, h, l in any order
                 dict(B=1, qos=(0, 256, 64), kos=(0, 256, 64)), dict(L=1, qos=(192, 64, 0), kos=(128, 64, 0)),
                 dict(L=1, Hq=1 << 15, qos=(2**62, 2**40, 1))):
        assert not refused(rope(lib, **good)), good


def test_rope_refuses_one_buffer_for_two_sides(lib):
    same = dict(Hk=3, ks=(768, 256, 64), kos=(768, 256, 64))
    for bad in (dict(ko=P[2]), dict(qo=P[1]), dict(ko=P[0]), dict(k=P[0], qo=P[0], ko=P[0]), dict(k=P[0], qo=P[0])):
        assert refused(rope(lib, **same, **bad)), bad
    host_only()
    for good in (dict(), dict(k=P[0]), dict(qo=P[0], ko=P[1]), dict(qo=P[0])):
        assert not refused(rope(lib, **same, **good)), good


def norm(lib, xo=P[2], h=P[3], x=P[0], y=P[1]):
    return lib.sol_attn_residual_norm(x, y, None, 0, None, None, 0, None, 0, None, B16, 1, 0, 1.0, 1e-6, 1, 4, 64, xo, h, None)


def norm_bwd(lib, dx=P[3], dy=P[4]):
    return lib.sol_attn_residual_norm_bwd(P[0], None, P[1], P[2], None, 0, None, None, 0, None, B16, 1, 0, 1.0, 1e-6, 1, 4, 64, dx, dy,
                                          None, None, None, None, None, None, 0, None)


def linear(lib, M=4, out=P[4], z=P[5], res=P[3], ws=P[6]):
    return lib.sol_attn_linear(P[0], P[1], P[2], res, 1, M, 64, 64, out, z, ws, 256, None)


def linear_bwd(lib, dx=P[4], dw=P[5], db=P[6]):
    return lib.sol_attn_linear_bwd(P[0], P[1], P[2], P[3], 1, 64, 64, 64, dx, dw, db, P[7], 1 << 30, None)


def test_one_buffer_for_two_outputs_or_for_an_input_of_other_blocks_is_refused(lib):
    assert refused(norm(lib, xo=P[3])) and refused(norm_bwd(lib, dx=P[4]))
    for bad in (dict(z=P[4]), dict(out=P[0]), dict(out=P[1]), dict(z=P[0]), dict(z=P[1]), dict(z=P[3]), dict(out=P[6]), dict(z=P[6])):
        assert refused(linear(lib, **bad)) and refused(linear(lib, M=300, **bad)), bad
    for bad in (dict(dx=P[0]), dict(dx=P[1]), dict(dx=P[2]), dict(dx=P[3]), dict(dw=P[0]), dict(dw=P[1]), dict(dw=P[4]), dict(db=P[5]),
                dict(db=P[7]), dict(dx=P[7])):
        assert refused(linear_bwd(lib, **bad)), bad
    host_only()
    assert not refused(norm(lib)) and not refused(norm(lib, xo=P[0])) and not refused(norm_bwd(lib))
    assert not refused(linear(lib)) and not refused(linear(lib, out=P[3])) and not refused(linear(lib, z=None, res=None, ws=None))
    assert not refused(linear_bwd(lib)) and not refused(linear_bwd(lib, dx=None, db=None))
