"""GPU parity of the rotary positions and of their tables against the float64 oracle.

Tolerances, u = 2^-24: cosine and sine come from an angle reduced in 64 bits and rounded once to fp32
(pi u of angle, |y| <= 1 in units of pi), a function good to 2 steps, and the factor: within 8 u of the
factor. A turned value adds two products in fp32: 12 u (|a| + |b|) m; a stored bf16 value half a step,
2^-8 of its size, a stored fp32 one u.
"""
import numpy as np
import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa
from block_sparse_attention_41_b200 import workloads as wl
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build
    build.build()
    sa.load_library()


def _np(t):
    return t.double().cpu().numpy()


def check(got, x, pos, f, sections, m, layout, inverse, dtype):
    cos, sin = bo.rope_tables(pos.cpu().numpy(), f.cpu().numpy(), sections, m)
    ref = bo.rope(_np(x), cos, sin, layout, inverse)
    mag = bo.rope(np.abs(_np(x)), np.full_like(cos, abs(m)), np.full_like(sin, -abs(m)), layout)  # (|a| + |b|) m
    half = 2 * cos.shape[-1]
    ia = np.arange(0, half, 2) if layout == "interleaved" else np.arange(half // 2)
    ib = ia + 1 if layout == "interleaved" else ia + half // 2
    mag[..., ib] = mag[..., ia]
    tol = STEP[dtype] * np.abs(ref) + 12 * U * mag
    tol[..., half:] = 0.0  # channels past rot are copied
    err = np.abs(_np(got) - ref)
    assert (err <= tol).all(), float((err - tol).max())


def inputs(B, Hq, Hk, L, d, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + L + d)
    return [torch.randn((B, h, L, d), generator=g, device="cuda").to(DT[dtype]) for h in (Hq, Hk)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("B,Hq,Hk,L,d,rot", [(1, 1, 1, 1, 2, 2), (2, 3, 1, 5, 64, 64), (1, 4, 2, 77, 128, 128),
                                             (2, 5, 5, 33, 96, 48), (1, 2, 2, 9, 128, 50), (1, 40, 8, 3, 256, 64),
                                             (1, 2, 1, 300, 30, 14), (1, 3, 3, 1000, 64, 62), (1, 9, 7, 2, 512, 512)])
def test_rope(B, Hq, Hk, L, d, rot, layout, dtype):
    q, k = inputs(B, Hq, Hk, L, d, dtype)
    f, m = sa.sol_attn_rope_inv_freq(rot, scaling="yarn", factor=4.0, original_length=256.0, device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda") * 7 + 3
    for inverse in (False, True):
        qo, ko = sa.sol_attn_rope(q, k, pos, f, layout=layout, attn_factor=m, inverse=inverse)
        torch.cuda.synchronize()
        check(qo, q, pos, f, None, m, layout, inverse, dtype)
        check(ko, k, pos, f, None, m, layout, inverse, dtype)
    q2, k2 = q.clone(), k.clone()  # in place
    qo, ko = sa.sol_attn_rope(q, k, pos, f, layout=layout, attn_factor=m)
    gq, gk = sa.sol_attn_rope(q2, k2, pos, f, layout=layout, attn_factor=m, Q_out=q2, K_out=k2)
    assert gq is q2 and torch.equal(q2, qo) and torch.equal(k2, ko)
    only, none = sa.sol_attn_rope(q, None, pos, f, layout=layout, attn_factor=m)
    assert none is None and torch.equal(only, qo)


@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("start", [0, 1_000_003, 2_000_000_000])
def test_far_positions_and_position_axes(layout, start):
    B, H, L, d, sections = 2, 3, 120, 64, (12, 10, 10)
    q, k = inputs(B, H, H, L, d, "f32")
    i = torch.arange(L)
    one = torch.stack([i // 40 + start, i // 8 % 5, i % 8])
    pos = torch.stack([one, one + torch.tensor([[1], [0], [-7]])]).to(torch.int32).cuda()  # of its own per batch entry
    f, m = sa.sol_attn_rope_inv_freq(d, sections=sections, device="cuda")
    qo, ko = sa.sol_attn_rope(q, k, pos, f, layout=layout, sections=sections)
    torch.cuda.synchronize()
    check(qo, q, pos, f, sections, m, layout, False, "f32")
    check(ko, k, pos, f, sections, m, layout, False, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("d,rot", [(128, 96), (128, 88), (128, 92), (128, 94), (72, 72), (68, 40), (66, 12), (20, 8)])
@pytest.mark.parametrize("shift", [0, 1, 2, 4, 8])
def test_every_width_of_access(layout, dtype, d, rot, shift):
    """Lengths, strides and addresses that divide by 8, 4, 2 or 1 values."""
    B, H, L = 2, 3, 21
    g = torch.Generator(device="cuda").manual_seed(d + rot + shift)
    wide = torch.randn((B, L, H, d + shift + (-d - shift) % 8), generator=g, device="cuda").to(DT[dtype])
    q = wide[..., shift:shift + d].transpose(1, 2)
    f, _ = sa.sol_attn_rope_inv_freq(rot, device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda") * 11
    ref, _ = sa.sol_attn_rope(q.contiguous(), None, pos, f, layout=layout)
    check(ref, q, pos, f, None, 1.0, layout, False, dtype)
    got, _ = sa.sol_attn_rope(q, None, pos, f, layout=layout)
    assert torch.equal(got, ref)
    back = torch.full_like(wide, 7.0)  # the gradient into a slice, the rest stays
    sa.sol_attn_rope(ref, None, pos, f, layout=layout, inverse=True, Q_out=back[..., shift:shift + d].transpose(1, 2))
    want, _ = sa.sol_attn_rope(ref, None, pos, f, layout=layout, inverse=True)
    assert torch.equal(back[..., shift:shift + d].transpose(1, 2), want)
    assert bool((back[..., :shift] == 7.0).all()) and bool((back[..., shift + d:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("d,pad", [(64, 0), (64, 8), (48, 3)])
def test_token_major_in_and_out(layout, dtype, d, pad):
    B, Hq, Hk, L = 2, 6, 3, 37
    g = torch.Generator(device="cuda").manual_seed(d + pad)
    qkv = torch.randn((B, L, Hq + 2 * Hk, d + pad), generator=g, device="cuda").to(DT[dtype])[..., :d]
    q, k = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
    f, m = sa.sol_attn_rope_inv_freq(32, device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    qo, ko = sa.sol_attn_rope(q, k, pos, f, layout=layout)
    assert qo.is_contiguous() and ko.is_contiguous()
    qc, kc = sa.sol_attn_rope(q.contiguous(), k.contiguous(), pos, f, layout=layout)
    assert torch.equal(qo, qc) and torch.equal(ko, kc)
    check(qo, q, pos, f, None, m, layout, False, dtype)
    # the way back, into slices of one buffer whose other slices stay as they are
    back = torch.full_like(qkv, 7.0)
    bq, bk = back[:, :, :Hq].transpose(1, 2), back[:, :, Hq:Hq + Hk].transpose(1, 2)
    sa.sol_attn_rope(qo, ko, pos, f, layout=layout, inverse=True, Q_out=bq, K_out=bk)
    cq, ck = sa.sol_attn_rope(qo, ko, pos, f, layout=layout, inverse=True)
    assert torch.equal(bq, cq) and torch.equal(bk, ck) and bool((back[:, :, Hq + Hk:] == 7.0).all())


def test_the_rest_passes_through_infinities_and_nan():
    q, _ = inputs(1, 2, 2, 4, 64, "bf16")
    q[..., 50] = float("nan")
    q[..., 51] = float("inf")
    f, _ = sa.sol_attn_rope_inv_freq(50, device="cuda")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    for layout in ("interleaved", "half"):
        out, _ = sa.sol_attn_rope(q, None, pos, f, layout=layout)
        assert torch.equal(out[..., 50:].view(torch.int16), q[..., 50:].contiguous().view(torch.int16))
        assert torch.isfinite(out[..., :50]).all()


def test_shared_heads_of_an_expanded_input():
    q, k = inputs(1, 1, 1, 20, 64, "bf16")
    f, _ = sa.sol_attn_rope_inv_freq(64, device="cuda")
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    one, _ = sa.sol_attn_rope(q, None, pos, f)
    many, _ = sa.sol_attn_rope(q.expand(1, 5, 20, 64), None, pos, f)
    assert all(torch.equal(many[:, h], one[:, 0]) for h in range(5))


@pytest.mark.parametrize("L,rot,sections", [(1, 2, None), (77, 64, None), (1000, 128, (22, 21, 21)), (50, 10, (2, 0, 3))])
def test_tables(L, rot, sections):
    f, m = sa.sol_attn_rope_inv_freq(rot, sections=sections, scaling="yarn", factor=8.0, original_length=100.0, device="cuda")
    axes = len(sections) if sections else 1
    pos = torch.stack([(torch.arange(L) * (a + 3) + 900_000) for a in range(axes)]).to(torch.int32).cuda()
    cos, sin = sa.sol_attn_rope_tables(pos, f, sections=sections, attn_factor=m)
    rc, rs = bo.rope_tables(pos.cpu().numpy(), f.cpu().numpy(), sections, m)
    assert np.abs(_np(cos) - rc).max() <= 8 * U * m and np.abs(_np(sin) - rs).max() <= 8 * U * m


def test_tables_feed_the_fused_norm_pass():
    """The 3-D tables of the input generator, built on the GPU, and the rotary call against the fused
    norm + rotary + pooling pass with unit rows: the same turned keys."""
    grid, d = (3, 7, 13), 64
    L = 3 * 7 * 13
    sections = (d // 2 - 2 * (d // 2 // 3), d // 2 // 3, d // 2 // 3)
    i = np.arange(L)
    pos = torch.from_numpy(np.stack([i // 91, i // 13 % 7, i % 13]).astype(np.int32)).cuda()
    f, _ = sa.sol_attn_rope_inv_freq(d, sections=sections, device="cuda")
    cos, sin = sa.sol_attn_rope_tables(pos, f, sections=sections)
    hc, hs = wl.rope_tables(grid, d)
    assert np.abs(_np(cos) - hc).max() <= 9 * U and np.abs(_np(sin) - hs).max() <= 9 * U
    q = (torch.randint(0, 2, (1, 2, L, d), device="cuda") * 2 - 1).to(torch.bfloat16)  # rows of +-1: rms 1
    gain = torch.ones(d, device="cuda")
    Qo, Ko, *_ = sa.sol_attn_qknorm_rope_pool(q, q, q, gain, gain, cos, sin, 128, eps=1e-12)
    ro, _ = sa.sol_attn_rope(q, None, pos, f, sections=sections)
    # both round fp32 values that differ by a few u: equal, or one bf16 step at a rounding border
    err = (Qo.double() - ro.double()).abs()
    assert bool((err <= 2.0 ** -7 * ro.double().abs() + 1e-6).all()) and float((err == 0).double().mean()) > 0.995


def test_more_elements_than_32_bits():
    L, H, d = 450_000, 40, 128  # 2.3e9 values
    q = torch.zeros((1, H, L, d), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 1, L // 2, L - 2, L - 1], device="cuda")
    q[:, :, rows] = torch.randn((1, H, 5, d), device="cuda").to(torch.bfloat16)
    f, _ = sa.sol_attn_rope_inv_freq(d, device="cuda")
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    for layout in ("interleaved", "half"):
        out, _ = sa.sol_attn_rope(q, None, pos, f, layout=layout)
        want, _ = sa.sol_attn_rope(q[:, :, rows].contiguous(), None, pos[rows].contiguous(), f, layout=layout)
        assert torch.equal(out[:, :, rows], want)
        del out


def test_streams_and_graphs():
    q, k = inputs(1, 4, 2, 500, 128, "bf16")
    f, _ = sa.sol_attn_rope_inv_freq(128, device="cuda")
    pos = torch.arange(500, dtype=torch.int32, device="cuda")
    ref = sa.sol_attn_rope(q, k, pos, f)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sa.sol_attn_rope(q, k, pos, f, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sa.sol_attn_rope(q, k, pos, f)
        tab = sa.sol_attn_rope_tables(pos, f)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, out))
    assert all(torch.equal(a, b) for a, b in zip(sa.sol_attn_rope_tables(pos, f), tab))


def test_refusals():
    q, k = inputs(1, 2, 2, 8, 64, "bf16")
    f, _ = sa.sol_attn_rope_inv_freq(64, device="cuda")
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    ok = dict(Q=q, K=k, pos=pos, inv_freq=f)
    for bad, err in ((dict(pos=pos.long()), TypeError), (dict(pos=pos[:4]), ValueError), (dict(inv_freq=f.float()), TypeError),
                     (dict(K=k.float()), TypeError), (dict(K=k[..., :32]), ValueError), (dict(layout="thirds"), ValueError),
                     (dict(Q=q.transpose(2, 3)), ValueError), (dict(Q=q.half()), TypeError), (dict(sections=(16, 16)), ValueError),
                     (dict(sections=(31,)), sa.SolAttnError), (dict(Q_out=q[..., :32]), ValueError),
                     (dict(Q_out=torch.empty((1, 1, 8, 64), dtype=q.dtype, device="cuda").expand(1, 2, 8, 64)), sa.SolAttnError),
                     (dict(Q=q[:, :, :0], K=None, pos=pos[:0]), sa.SolAttnError),
                     (dict(inv_freq=torch.ones(40, dtype=torch.float64, device="cuda")), sa.SolAttnError)):
        with pytest.raises(err):
            sa.sol_attn_rope(**{**ok, **bad})
    with pytest.raises(ValueError):
        sa.sol_attn_rope(q, None, pos, f, K_out=k)
