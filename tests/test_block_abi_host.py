"""Host-side refusals of the dense operators' entry points: nothing is launched, no GPU is needed."""
import ctypes
import math

import numpy as np
import pytest
import torch

from block_sparse_attention_41_b200 import build as builder
from block_sparse_attention_41_b200 import sol_attn as sa
from oracle import block_oracle as bo

# fake, 16-byte aligned device addresses: validation must reject before any of them is used
P = [ctypes.c_void_p(0x1000 * (i + 1)) for i in range(16)]
ODD = ctypes.c_void_p(0x1008)


@pytest.fixture(scope="module")
def lib():
    builder.build()
    return sa.load_library()


def norm(lib, x=P[0], y=P[1], gate=P[2], gs=0, gain=P[3], scale=P[4], shift=P[5], pg=None, dt=sa.SOL_BF16, n=1, pn=0, a=1.0,
         eps=1e-6, B=1, T=4, C=64, xo=P[6], h=P[7], ss=0):
    return lib.sol_attn_residual_norm(x, y, gate, gs, gain, scale, ss, shift, 0, pg, dt, n, pn, a, eps, B, T, C, xo, h, None)


def test_residual_norm_rejects_invalid_arguments(lib):
    for bad in (dict(x=None), dict(h=None), dict(x=ODD), dict(h=ODD), dict(xo=ODD), dict(xo=None), dict(B=0), dict(T=0),
                dict(C=0), dict(dt=5), dict(n=0), dict(n=3), dict(pn=3), dict(eps=0.0), dict(eps=math.nan),
                dict(eps=math.inf), dict(a=math.inf), dict(pg=P[8]), dict(gate=ctypes.c_void_p(0x1002)),
                dict(B=2, gs=-64), dict(y=None), dict(y=None, gate=None, a=2.0), dict(y=None, gate=None)):
        assert norm(lib, **bad) == sa.SOL_EINVAL, bad
    assert norm(lib, C=8193) == sa.SOL_EUNSUPPORTED
    assert "8192" in lib.sol_attn_last_error().decode()
    assert norm(lib, B=1 << 16, T=1 << 15) == sa.SOL_EUNSUPPORTED


def norm_bwd(lib, dh=P[0], dxo=P[1], x=P[2], y=P[3], gate=P[4], gain=P[5], scale=P[6], pg=None, B=1, T=4, C=64, dx=P[7],
             dy=P[8], dgate=P[9], dgain=P[10], dscale=P[11], dshift=P[12], dpg=None, ws=P[13], nbytes=1 << 30):
    return lib.sol_attn_residual_norm_bwd(dh, dxo, x, y, gate, 0, gain, scale, 0, pg, sa.SOL_BF16, 1, 0, 1.0, 1e-6, B, T, C,
                                          dx, dy, dgate, dgain, dscale, dshift, dpg, ws, nbytes, None)


def test_residual_norm_bwd_rejects_invalid_arguments(lib):
    for bad in (dict(dh=None), dict(dx=None), dict(dy=None), dict(x=None), dict(dh=ODD), dict(dxo=ODD), dict(dy=ODD),
                dict(gate=None), dict(gain=None), dict(scale=None), dict(dpg=P[14]), dict(ws=None), dict(nbytes=16),
                dict(ws=ODD), dict(dgain=ctypes.c_void_p(0x1001)), dict(y=None, dy=None, gate=None, dgate=None)):
        assert norm_bwd(lib, **bad) == sa.SOL_EINVAL, bad
    assert norm_bwd(lib, B=65536, T=1) == sa.SOL_EUNSUPPORTED


def test_residual_norm_workspace_bytes(lib):
    f = lib.sol_attn_residual_norm_bwd_workspace_bytes
    assert f(0, 1, 1) == f(1, 0, 1) == f(1, 1, 0) == f(1, 1, 8193) == 0
    # at least one slot of three sums per batch entry, and bounded however long the sequence
    assert f(3, 1, 64) >= 3 * 3 * 64 * 4
    assert f(1, 10_000_000, 8192) == f(1, 1_000_000, 8192) <= 128 << 20


def freq(lib, rot=8, base=1e4, axes=1, sec=None, scaling=0, factor=1.0, length=100.0, lo=1.0, hi=32.0):
    out, m = (ctypes.c_double * 64)(), ctypes.c_float()
    c = None if sec is None else (ctypes.c_int * len(sec))(*sec)
    return lib.sol_attn_rope_inv_freq(rot, base, axes, c, scaling, factor, length, lo, hi, out, ctypes.byref(m)), out, m.value


def test_rope_inv_freq_rejects_invalid_arguments(lib):
    for bad in (dict(rot=7), dict(rot=0), dict(axes=0), dict(axes=5), dict(axes=3), dict(axes=2, sec=(1, 2)),
                dict(axes=2, sec=(5, -1)), dict(base=1.0), dict(base=math.inf), dict(scaling=4), dict(scaling=1, factor=0.5),
                dict(scaling=1, factor=math.nan), dict(scaling=3, factor=2.0, length=0.0),
                dict(scaling=3, factor=2.0, lo=3.0, hi=3.0)):
        assert freq(lib, **bad)[0] == sa.SOL_EINVAL, bad


@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
@pytest.mark.parametrize("rot,sections", [(128, None), (128, (22, 21, 21)), (2, None), (10, (5, 0, 0)), (6, (1, 1, 1))])
def test_rope_inv_freq_matches_oracle(lib, rot, sections, scaling, factor):
    f, m = sa.sol_attn_rope_inv_freq(rot, 10000.0, sections, scaling, factor, original_length=4096.0)
    ref, rm = bo.rope_inv_freq(rot, 10000.0, sections, scaling, factor, original_length=4096.0)
    # a power, a division and a blend: a few 64-bit roundings
    assert f.dtype == torch.float64 and np.allclose(f.numpy(), ref, rtol=1e-13, atol=0)
    assert abs(m - rm) <= 2.0 ** -24 * rm


def rope(lib, q=P[0], k=P[1], qs=(512, 64, 64), ks=(512, 64, 64), dt=sa.SOL_BF16, pos=P[2], axes=1, sec=None, f=P[3], m=1.0,
         layout=0, B=1, Hq=2, Hk=2, L=4, d=64, rot=64, qo=P[4], qos=(512, 256, 64), ko=P[5], kos=(512, 256, 64)):
    i64 = lambda v: None if v is None else (ctypes.c_int64 * 3)(*v)  # noqa: E731
    c = None if sec is None else (ctypes.c_int * len(sec))(*sec)
    return lib.sol_attn_rope(q, i64(qs), k, i64(ks), dt, pos, 0, axes, c, f, m, layout, 0, B, Hq, Hk, L, d, rot, qo, i64(qos),
                             ko, i64(kos), None)


def test_rope_rejects_invalid_arguments(lib):
    for bad in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(f=None), dict(qs=None),
                dict(kos=None), dict(dt=3), dict(layout=2), dict(B=0), dict(Hq=0), dict(Hk=-1), dict(L=0), dict(d=0),
                dict(rot=0), dict(rot=63), dict(rot=66), dict(axes=2), dict(axes=2, sec=(16, 17)), dict(m=math.inf),
                dict(q=ctypes.c_void_p(0x1001)), dict(f=ctypes.c_void_p(0x1004)), dict(pos=ctypes.c_void_p(0x1002)),
                dict(qs=(512, -64, 64)), dict(qos=(512, 256, 0)), dict(kos=(512, 0, 64)),
                dict(qo=P[0])):  # in place with other strides
        assert rope(lib, **bad) == sa.SOL_EINVAL, bad
    assert rope(lib, d=514, rot=64) == sa.SOL_EUNSUPPORTED
    assert rope(lib, d=65, rot=64) == sa.SOL_EUNSUPPORTED
    assert rope(lib, B=70000) == sa.SOL_EUNSUPPORTED


def tables(lib, pos=P[0], axes=1, f=P[1], m=1.0, L=4, rot=64, c=P[2], s=P[3]):
    return lib.sol_attn_rope_tables(pos, axes, None, f, m, L, rot, c, s, None)


def test_rope_tables_rejects_invalid_arguments(lib):
    for bad in (dict(pos=None), dict(f=None), dict(c=None), dict(s=None), dict(L=0), dict(rot=0), dict(rot=5), dict(axes=3),
                dict(m=math.nan), dict(c=ctypes.c_void_p(0x1002))):
        assert tables(lib, **bad) == sa.SOL_EINVAL, bad


def test_bindings_refuse_cpu_tensors(lib):
    x = torch.zeros(1, 4, 64)
    with pytest.raises(TypeError):
        sa.sol_attn_residual_norm(x)
    with pytest.raises(TypeError):
        sa.sol_attn_residual_norm_bwd(x, x)
    q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(TypeError):
        sa.sol_attn_rope(q, q, torch.arange(4), torch.ones(32))
    with pytest.raises(TypeError):
        sa.sol_attn_rope_tables(torch.arange(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64))


def linear(lib, x=P[0], w=P[1], bias=P[2], res=P[3], act=1, M=4, N=64, K=64, out=P[4], z=P[5], ws=P[6], nbytes=256):
    return lib.sol_attn_linear(x, w, bias, res, act, M, N, K, out, z, ws, nbytes, None)


def linear_bwd(lib, dy=P[0], x=P[1], w=P[2], z=P[3], act=1, M=4, N=64, K=64, dx=P[4], dw=P[5], db=P[6], ws=P[7], nbytes=1 << 30):
    return lib.sol_attn_linear_bwd(dy, x, w, z, act, M, N, K, dx, dw, db, ws, nbytes, None)


def test_linear_rejects_invalid_arguments(lib):
    for bad in (dict(x=None), dict(w=None), dict(out=None), dict(x=ODD), dict(w=ODD), dict(bias=ODD), dict(res=ODD), dict(z=ODD),
                dict(out=ODD), dict(ws=ODD), dict(nbytes=255), dict(act=4), dict(act=-1), dict(M=0), dict(N=0), dict(K=-8)):
        assert linear(lib, **bad) == sa.SOL_EINVAL, bad
    for bad in (dict(N=60), dict(K=4), dict(M=1 << 28, N=1 << 28)):
        assert linear(lib, **bad) == sa.SOL_EUNSUPPORTED, bad


def test_linear_bwd_rejects_invalid_arguments(lib):
    for bad in (dict(dy=None), dict(x=None), dict(w=None), dict(z=None), dict(act=0), dict(ws=None), dict(nbytes=512),
                dict(dx=None, dw=None, db=None), dict(dy=ODD), dict(dw=ODD), dict(db=ctypes.c_void_p(0x1002)), dict(act=9),
                dict(M=0)):
        assert linear_bwd(lib, **bad) == sa.SOL_EINVAL, bad
    assert linear_bwd(lib, N=4) == linear_bwd(lib, K=12) == sa.SOL_EUNSUPPORTED


def test_linear_workspace_bytes(lib):
    f = lib.sol_attn_linear_bwd_workspace_bytes
    assert f(0, 8, 0) == f(8, 0, 0) == f(8, 8, 4) == 0
    # error words, one row of partial sums at least, and dz where there is an activation
    assert f(1, 64, 0) >= 256 + 64 * 4
    assert f(1000, 64, 1) - f(1000, 64, 0) == 1000 * 64 * 2
    assert f(1 << 24, 64, 0) == f(1 << 22, 64, 0) <= 32 << 20


def test_linear_forward_workspace_bytes(lib):
    f = lib.sol_attn_linear_workspace_bytes
    assert f(0, 8, 8) == f(8, 4, 8) == f(8, 8, 12) == f(1 << 28, 1 << 28, 8) == 0
    assert f(128, 4096, 4096) == f(33272, 16384, 4096) == f(8191, 768, 768) == f(200, 768, 64) == 256
    assert 256 < f(200, 4096, 4096) <= 32 << 20


def test_linear_bindings_refuse_cpu_tensors(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        sa.sol_attn_linear(x, x)
    with pytest.raises(TypeError):
        sa.sol_attn_linear_bwd(x, x, x)
