"""GPU parity of the linear layer and its gradients against the float64 oracle.

Two kinds of inputs. Small whole numbers: every product and every partial sum is a whole number below
2^24, so the fp32 accumulation is exact in any order and outputs must equal the oracle's value
rounded once to bf16, bit for bit. Random values: a product of two bf16 numbers is exact in fp32; one
MMA adds 16 of them and the accumulator, each cut to 24 bits at the largest term (2^-23 each), so a
sum over K is within 17 (K / 16 + 1) 2^-23 of the sum of magnitudes. The activations add 2^-24 per
operation: 16 of those of |z|, and an exponential's argument u is off by 4 x 2^-24 |u|, which its
value takes as a relative error: 16 (1 + |u|) 2^-24 |z| covers all three forms with |u| <= 1.6 |z| (1 +
0.045 z^2). A slope of at most 1.13 carries the error of z. A stored bf16 value is off by at most
2^-8 of its size; dz is stored so before the two products.
"""
import numpy as np
import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = 2.0 ** -8
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build
    build.build()
    sa.load_library()


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _gen(*key):
    return torch.Generator(device="cuda").manual_seed(sum(k * p for k, p in zip(key, (1, 1009, 10007, 100003))))


def ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(BF)


def same_bits(got, want, what):
    """got (bf16 or fp32) against exact float64 values rounded once."""
    want = torch.from_numpy(np.ascontiguousarray(want)).to(got.dtype).cuda()
    bad = (got != want).nonzero()
    assert bad.numel() == 0, f"{what}: {bad.shape[0]} of {got.numel()} values differ, the first at {bad[0].tolist()}"


FEW = [1, 2, 15, 16, 17, 33, 64, 65, 127, 128]
MANY = [129, 255, 256, 257, 300, 1000]
SIZES = [(8, 8), (8, 64), (64, 8), (72, 136), (128, 64), (256, 1032), (264, 520), (520, 256)]


@pytest.mark.parametrize("N,K", SIZES)
@pytest.mark.parametrize("M", FEW + MANY)
def test_whole_numbers_are_exact(M, N, K):
    g = _gen(M, N, K)
    x, w, res = ints(g, -3, 3, M, K), ints(g, -2, 2, N, K), ints(g, -9, 9, M, N)
    bias = torch.randint(-5, 6, (N,), generator=g, device="cuda").float()
    plain, _ = bo.linear(_np(x), _np(w))
    full, z = bo.linear(_np(x), _np(w), _np(bias), "none", _np(res))
    same_bits(sa.sol_attn_linear(x, w), plain, "x w^T")
    out, zz = sa.sol_attn_linear(x, w, bias, residual=res, want_z=True)
    same_bits(out, full, "out")
    same_bits(zz, z, "z")


@pytest.mark.parametrize("N,K", SIZES + [(8, 2048), (2048, 8)])
@pytest.mark.parametrize("M", [1, 7, 64, 65, 129, 300, 1000])
def test_whole_number_gradients_are_exact(M, N, K):
    g = _gen(M, N, K, 1)
    dy, x, w = ints(g, -3, 3, M, N), ints(g, -2, 2, M, K), ints(g, -3, 3, N, K)
    dx, dw, db = sa.sol_attn_linear_bwd(dy, x, w)
    rx, rw, rb = bo.linear_bwd(_np(dy), _np(x), _np(w))
    same_bits(dx, rx, "dx")
    same_bits(dw, rw, "dw")
    same_bits(db, rb, "db")


def test_many_tiles_per_sm_and_a_deep_ring():
    # every CTA walks several tiles, slices wrap around the ring, all three tile widths
    for M, N, K in ((2568, 2056, 200), (1288, 1000, 1544), (5000, 136, 72), (20000, 264, 128)):
        g = _gen(M, N, K, 2)
        x, w = ints(g, -2, 2, M, K), ints(g, -2, 2, N, K)
        same_bits(sa.sol_attn_linear(x, w), bo.linear(_np(x), _np(w))[0], f"{M} {N} {K}")
        dy = ints(g, -2, 2, M, N)
        dx, dw, db = sa.sol_attn_linear_bwd(dy, x, w)
        rx, rw, rb = bo.linear_bwd(_np(dy), _np(x), _np(w))
        same_bits(dx, rx, f"dx {M} {N} {K}")
        same_bits(dw, rw, f"dw {M} {N} {K}")
        same_bits(db, rb, f"db {M} {N} {K}")


@pytest.mark.parametrize("M,N,K", [(4104, 4096, 136), (4104, 136, 4096), (136, 4104, 4096), (4000, 4360, 72), (2304, 20000, 8)])
def test_many_large_tiles(M, N, K):
    # enough outputs in one of the three products for tiles of two SMs, ragged at the ends
    g = _gen(M, N, K, 6)
    x, w, dy = ints(g, -2, 2, M, K), ints(g, -2, 2, N, K), ints(g, -2, 2, M, N)
    res = ints(g, -9, 9, M, N)
    bias = torch.randint(-5, 6, (N,), generator=g, device="cuda").float()
    out, z = sa.sol_attn_linear(x, w, bias, residual=res, want_z=True)
    ref, rz = bo.linear(_np(x), _np(w), _np(bias), "none", _np(res))
    same_bits(out, ref, "out")
    same_bits(z, rz, "z")
    dx, dw, db = sa.sol_attn_linear_bwd(dy, x, w)
    rx, rw, rb = bo.linear_bwd(_np(dy), _np(x), _np(w))
    same_bits(dx, rx, "dx")
    same_bits(dw, rw, "dw")
    same_bits(db, rb, "db")


@pytest.mark.parametrize("M,N,K", [(129, 136, 4104), (200, 4096, 4096), (300, 72, 8192), (1000, 5120, 4104), (1500, 264, 4104)])
def test_split_products_of_few_tiles(M, N, K):
    lib = sa.load_library()
    assert lib.sol_attn_linear_workspace_bytes(M, N, K) > 256
    g = _gen(M, N, K, 7)
    x, w, res = ints(g, -2, 2, M, K), ints(g, -2, 2, N, K), ints(g, -9, 9, M, N)
    bias = torch.randint(-5, 6, (N,), generator=g, device="cuda").float()
    ref, rz = bo.linear(_np(x), _np(w), _np(bias), "none", _np(res))
    out, z = sa.sol_attn_linear(x, w, bias, residual=res, want_z=True)
    same_bits(out, ref, "out")
    same_bits(z, rz, "z")
    again = res.clone()
    assert torch.equal(sa.sol_attn_linear(x, w, bias, residual=again, out=again), out)  # in place of the residual
    unsplit = sa.sol_attn_linear(x, w, bias, residual=res, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    assert torch.equal(unsplit, out)  # whole sums do not depend on the order
    # an activation on split sums: the same z, so the same bits
    for act in ("gelu", "gelu_tanh", "silu"):
        small = (w.float() / 64).to(BF)
        a = sa.sol_attn_linear(x, small, bias, act, res)
        b = sa.sol_attn_linear(x, small, bias, act, res, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
        assert torch.equal(a, b), act


def sum_error(K):
    return 17 * (K / 16 + 1) * 2.0 ** -23


def close(got, ref, extra, step, what):
    err = np.abs(_np(got) - ref)
    assert np.isfinite(_np(got)).all(), what
    worst = float((err / (step * np.abs(ref) + extra + 1e-30)).max())
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def act_error(z):
    a = np.abs(z)
    return 16 * U * a * (1 + 1.6 * a * (1 + 0.045 * a * a))


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,K", [(1, 768, 768), (3, 136, 4096), (100, 200, 72), (128, 1024, 512), (129, 136, 264), (700, 264, 768)])
def test_activations(M, N, K, act):
    g = _gen(M, N, K, 3)
    x = torch.randn((M, K), generator=g, device="cuda").to(BF)
    w = (torch.randn((N, K), generator=g, device="cuda") * (2.0 / K ** 0.5)).to(BF)
    bias = torch.randn(N, generator=g, device="cuda")
    res = torch.randn((M, N), generator=g, device="cuda").to(BF)
    out, z = sa.sol_attn_linear(x, w, bias, act, res, want_z=True)
    ref, rz = bo.linear(_np(x), _np(w), _np(bias), act, _np(res))
    ez = sum_error(K) * (np.abs(_np(x)) @ np.abs(_np(w)).T) + U * (np.abs(rz) + np.abs(_np(bias)))
    close(z, rz, ez, HALF_STEP, "z")
    close(out, ref, 1.13 * ez + act_error(rz) + 2 * U * np.abs(_np(res)), HALF_STEP, "out")
    # the same without z, in place of the residual
    again = res.clone()
    assert sa.sol_attn_linear(x, w, bias, act, again, out=again) is again and torch.equal(again, out)


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,K", [(1, 768, 72), (130, 136, 264), (3000, 264, 136), (257, 520, 520)])
def test_activation_gradients(M, N, K, act):
    g = _gen(M, N, K, 4)
    r = lambda *s, a=1.0: (torch.randn(s, generator=g, device="cuda") * a).to(BF)  # noqa: E731
    dy, x, w, z = r(M, N), r(M, K), r(N, K, a=N ** -0.5), r(M, N, a=2.0)
    dx, dw, db = sa.sol_attn_linear_bwd(dy, x, w, z, act)
    rx, rw, rb = bo.linear_bwd(_np(dy), _np(x), _np(w), _np(z), act)
    dz = _np(dy) * bo.activation_slope(_np(z), act)
    e = np.abs(_np(dy)) * act_error(np.maximum(np.abs(_np(z)), 1.0)) * 4  # products of four such factors
    stored = HALF_STEP * np.abs(dz) + e
    mag = np.abs(dz) + stored
    aw, ax = np.abs(_np(w)), np.abs(_np(x))
    close(dx, rx, stored @ aw + sum_error(N) * (mag @ aw), HALF_STEP, "dx")
    close(dw, rw, stored.T @ ax + sum_error(M) * (mag.T @ ax), HALF_STEP, "dw")
    # fp32 sums of at most M additions in a chain, usually far fewer
    close(db, rb, e.sum(0) + M * U * mag.sum(0), U, "db")


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])
def test_gradients_against_differences_of_the_forward(act):
    """<dx, v> against the forward at x + v and x - v: a step of 2^-4 in whole quarters keeps x exact in
    bf16. The stored z is rounded, so the comparison is to 2 %."""
    g = _gen(5, 6, 7)
    M, N, K = 130, 136, 72
    x = ints(g, -8, 8, M, K) / 4
    v = ints(g, -1, 1, M, K) / 16
    w = (torch.randn((N, K), generator=g, device="cuda") * K ** -0.5).to(BF)
    dy = torch.randn((M, N), generator=g, device="cuda").to(BF)
    _, z = sa.sol_attn_linear(x, w, act=act, want_z=True)
    dx, dw, _ = sa.sol_attn_linear_bwd(dy, x, w, z if act != "none" else None, act)
    loss = lambda xx, ww: float((_np(dy) * bo.linear(_np(xx), _np(ww), None, act)[0]).sum())  # noqa: E731
    want = (loss(x + v, w) - loss(x - v, w)) / 2
    scale = float(np.sqrt((_np(dx) ** 2).sum() * (_np(v) ** 2).sum()))
    assert abs(float((_np(dx) * _np(v)).sum()) - want) <= 0.02 * scale
    dwv = 2.0 ** -8 * torch.randn((N, K), generator=g, device="cuda").double().cpu().numpy()
    lw = lambda s: float((_np(dy) * bo.linear(_np(x), _np(w) + s * dwv, None, act)[0]).sum())  # noqa: E731
    scale = float(np.sqrt((_np(dw) ** 2).sum() * (dwv ** 2).sum()))
    assert abs(float((_np(dw) * dwv).sum()) - (lw(1) - lw(-1)) / 2) <= 0.02 * scale


def test_nan_and_infinity_stay_in_their_rows_and_columns():
    for M in (5, 200):
        g = _gen(M, 8)
        x, w = ints(g, -2, 2, M, 72), ints(g, 1, 2, 136, 72)
        ref = sa.sol_attn_linear(x, w)
        x[3, 70] = float("nan")
        x[4, 0] = float("inf")
        out = sa.sol_attn_linear(x, w)
        keep = [i for i in range(M) if i not in (3, 4)]
        assert torch.equal(out[keep], ref[keep])
        assert out[3].isnan().all() and out[4].isinf().all()
        for act in ("gelu", "gelu_tanh", "silu"):  # large values of either sign: z or 0, never NaN
            big = torch.full((M, 8), 128.0, device="cuda", dtype=BF)
            o = sa.sol_attn_linear(big, torch.tensor([[24.0] * 8, [-24.0] * 8] * 4, device="cuda", dtype=BF), act=act)
            assert torch.equal(o[:, 0::2], torch.full_like(o[:, 0::2], 24576.0)) and not o[:, 1::2].any(), act


def test_values_past_the_rows_and_columns_stay():
    """Outputs inside a larger buffer: what lies behind them is not touched."""
    for M, N, K in ((3, 72, 64), (130, 72, 64), (200, 264, 72)):
        x, w = torch.ones((M, K), device="cuda", dtype=BF), torch.ones((N, K), device="cuda", dtype=BF)
        buf = torch.full((M * N + 4096,), 7.0, device="cuda", dtype=BF)
        out = buf[:M * N].view(M, N)
        sa.sol_attn_linear(x, w, out=out)
        assert bool((out == K).all()) and bool((buf[M * N:] == 7.0).all())


def test_leading_shape_and_empty_parts():
    x = torch.randn((2, 3, 64), device="cuda").to(BF)
    w = torch.randn((72, 64), device="cuda").to(BF)
    out = sa.sol_attn_linear(x, w)
    assert out.shape == (2, 3, 72) and torch.equal(out.view(6, 72), sa.sol_attn_linear(x.view(6, 64), w))
    dx, dw, db = sa.sol_attn_linear_bwd(out, x, w, want_dw=False, want_db=False)
    assert dx.shape == x.shape and dw is None and db is None
    dx, dw, db = sa.sol_attn_linear_bwd(out, x, w, want_dx=False)
    assert dx is None and dw.shape == w.shape and db.shape == (72,)


def test_more_elements_than_32_bits():
    M, K, N = 270_000, 8, 8000  # 2.16e9 outputs
    x = torch.zeros((M, K), device="cuda", dtype=BF)
    w = ints(_gen(9), -3, 3, N, K)
    rows = [0, 1, 134_217, 134_218, 268_435, 268_436, M - 1]
    x[rows] = ints(_gen(10), 1, 3, len(rows), K)
    out = sa.sol_attn_linear(x, w)
    assert torch.equal(out[rows], sa.sol_attn_linear(x[rows].contiguous(), w))
    assert not out[2:134_217].any() and not out[268_437:M - 1].any()
    del out
    z = torch.zeros((M, N), device="cuda", dtype=BF)
    dy = torch.zeros((M, N), device="cuda", dtype=BF)
    dy[rows] = ints(_gen(11), -4, 4, len(rows), N)
    dx, dw, db = sa.sol_attn_linear_bwd(dy, x, w, z, "silu")  # the slope at 0 is a half
    assert torch.equal(db, 0.5 * dy[rows].float().sum(0))
    rx, rw, _ = bo.linear_bwd(_np(dy[rows]) * 0.5, _np(x[rows]), _np(w))
    same_bits(dx[rows], rx, "dx")
    same_bits(dw, rw, "dw")


def test_same_bits_every_time_streams_and_graphs():
    g = _gen(12)
    M, N, K = 1000, 520, 264
    x = torch.randn((M, K), generator=g, device="cuda").to(BF)
    w = torch.randn((N, K), generator=g, device="cuda").to(BF)
    dy = torch.randn((M, N), generator=g, device="cuda").to(BF)

    def both(stream=None):
        out, z = sa.sol_attn_linear(x, w, act="gelu", want_z=True, stream=stream)
        few = sa.sol_attn_linear(x[:40], w, act="silu", stream=stream)
        return [out, z, few, *sa.sol_attn_linear_bwd(dy, x, w, z, "gelu", stream=stream)]
    ref = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, None):
        got = both(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(r, o) for r, o in zip(ref, got))
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs = both()
        graphs.append((gr, outs, torch.cuda.Stream()))
    for _ in range(3):
        for gr, _, st in graphs:
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for _, outs, _ in graphs:
        assert all(torch.equal(r, o) for r, o in zip(ref, outs))


def test_device_error_words():
    x, w = torch.ones((200, 64), device="cuda", dtype=BF), torch.ones((72, 64), device="cuda", dtype=BF)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for n in (3, 200):
        sa.sol_attn_linear(x[:n], w, workspace=ws)
        sa.sol_attn_check_device_error(ws)
    lib = sa.load_library()
    ws = torch.zeros(lib.sol_attn_linear_bwd_workspace_bytes(200, 72, 1), dtype=torch.uint8, device="cuda")
    dy = torch.ones((200, 72), device="cuda", dtype=BF)
    sa.sol_attn_linear_bwd(dy, x, w, dy, "gelu", workspace=ws)
    sa.sol_attn_check_device_error(ws)


def test_refusals():
    x, w = torch.ones((4, 64), device="cuda", dtype=BF), torch.ones((72, 64), device="cuda", dtype=BF)
    dy = torch.ones((4, 72), device="cuda", dtype=BF)
    for bad in (lambda: sa.sol_attn_linear(x.float(), w), lambda: sa.sol_attn_linear(x, w.half()),
                lambda: sa.sol_attn_linear(x, w, bias=torch.ones(72, device="cuda", dtype=BF)),
                lambda: sa.sol_attn_linear(x, w, residual=dy.float()), lambda: sa.sol_attn_linear(x, w.cpu())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sa.sol_attn_linear(x, w[:, :32]), lambda: sa.sol_attn_linear(x.t(), w),
                lambda: sa.sol_attn_linear(x, w, act="relu"), lambda: sa.sol_attn_linear(x, w, residual=dy[:2]),
                lambda: sa.sol_attn_linear(x, w, bias=torch.ones(71, device="cuda")),
                lambda: sa.sol_attn_linear(x[:, :32].contiguous(), w),
                lambda: sa.sol_attn_linear_bwd(dy, x[:2], w), lambda: sa.sol_attn_linear_bwd(dy, x, w, dy[:2], "gelu")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sa.sol_attn_linear(x[:, :12].contiguous(), w[:, :12].contiguous()),
                lambda: sa.sol_attn_linear(x, w[:5]), lambda: sa.sol_attn_linear(x[:0], w),
                lambda: sa.sol_attn_linear(x, w, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                lambda: sa.sol_attn_linear_bwd(dy, x, w, None, "gelu"), lambda: sa.sol_attn_linear_bwd(dy, x, w, dy, "none"),
                lambda: sa.sol_attn_linear_bwd(dy, x, w, want_dx=False, want_dw=False, want_db=False),
                lambda: sa.sol_attn_linear_bwd(dy, x, w, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(sa.SolAttnError):
            bad()
