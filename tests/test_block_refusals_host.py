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
