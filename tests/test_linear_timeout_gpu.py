"""The linear layer's bounded device waits made to expire: a launch that leaves one copy out, so that its
consumer waits in vain, gives up after 0.2 s, lets everything in flight end and returns.

One case per kernel and tile: single CTAs of two widths, pairs of two widths, products split along the
reduction, the kernel for few rows with and without a cluster, and the two products of the gradient.
"""
import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
FIRST, SECOND, RESIDUAL = 2, 3, 4  # the CTA that leaves a slice of an operand out, or a chunk of the residual

# M, N, K
FEW = [(3, 4096, 4096), (100, 1024, 512), (16, 136, 264), (128, 40000, 256)]
ONE = [(300, 264, 136), (1000, 768, 768), (2000, 768, 768)]
PAIRS = [(8191, 768, 768), (4104, 4096, 136), (10000, 264, 2056)]
SPLIT = [(200, 4096, 4096), (300, 72, 8192), (1500, 264, 4104)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build
    build.build()
    sa.load_library()


def ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda").to(BF)


def operands(M, N, K):
    g = torch.Generator(device="cuda").manual_seed(M + 7 * N + 31 * K)
    return ints(g, -2, 2, M, K), ints(g, -2, 2, N, K), ints(g, -9, 9, M, N)


def words(M, N, K):
    return torch.zeros(sa.load_library().sol_attn_linear_workspace_bytes(M, N, K), dtype=torch.uint8, device="cuda")


def expires(mode, call, ws):
    """The call's results, with one of its copies left out; the wait for it is reported once."""
    sa.sol_attn_check_device_error(ws)
    sa.sol_attn_debug_drop_one_load(mode)
    got = call()
    with pytest.raises(sa.SolAttnError) as e:
        sa.sol_attn_check_device_error(ws)
    assert e.value.status == sa.SOL_ETIMEOUT
    sa.sol_attn_check_device_error(ws)
    return got


@pytest.mark.parametrize("mode", [FIRST, SECOND])
@pytest.mark.parametrize("M,N,K", FEW + ONE + PAIRS + SPLIT)
def test_a_lost_operand_is_reported_and_the_next_call_is_right(M, N, K, mode):
    x, w, res = operands(M, N, K)
    ws = words(M, N, K)
    want = sa.sol_attn_linear(x, w, residual=res, workspace=ws)
    expires(mode, lambda: sa.sol_attn_linear(x, w, residual=res, workspace=ws), ws)
    assert torch.equal(sa.sol_attn_linear(x, w, residual=res, workspace=ws), want)
    sa.sol_attn_check_device_error(ws)


@pytest.mark.parametrize("with_z", [False, True])
@pytest.mark.parametrize("M,N,K", ONE + PAIRS)
def test_a_lost_residual_leaves_no_sum_behind(M, N, K, with_z):
    """No output is formed from a staging buffer whose copy has not come: what the call writes is right or NaN."""
    x, w, res = operands(M, N, K)
    ws = words(M, N, K)
    want = sa.sol_attn_linear(x, w, residual=res, workspace=ws)
    out = torch.full_like(want, 7.5)  # no sum of whole numbers
    z = torch.full_like(want, 7.5) if with_z else None
    expires(RESIDUAL, lambda: sa.sol_attn_linear(x, w, residual=res, out=out, z=z, workspace=ws), ws)
    kept = (out == 7.5) | out.isnan()
    assert bool(kept.any()) and bool((kept | (out == want)).all())
    if with_z:
        plain = sa.sol_attn_linear(x, w, workspace=ws)
        assert bool(((z == 7.5) | z.isnan() | (z == plain)).all())
    again = res.clone()  # in place of the residual
    assert torch.equal(sa.sol_attn_linear(x, w, residual=again, out=again, workspace=ws), want)
    sa.sol_attn_check_device_error(ws)


@pytest.mark.parametrize("mode", [FIRST, SECOND])
@pytest.mark.parametrize("M,N,K,which", [(*s, p) for s in ((300, 264, 136), (4104, 4096, 136), (1000, 1024, 1024))
                                         for p in ("dx", "dw")] + [(3, 264, 520, "dx")])  # dw of 3 rows: one slice
def test_a_lost_operand_of_a_gradient_is_reported(M, N, K, which, mode):
    x, w, dy = operands(M, N, K)
    ws = torch.zeros(sa.load_library().sol_attn_linear_bwd_workspace_bytes(M, N, 0), dtype=torch.uint8, device="cuda")

    def call():
        return sa.sol_attn_linear_bwd(dy, x, w, want_dx=which == "dx", want_dw=which == "dw", want_db=False, workspace=ws)
    want = call()
    expires(mode, call, ws)
    got = call()
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
    sa.sol_attn_check_device_error(ws)


def right_or_nan(got, want, what):
    """Every value is the healthy call's or NaN, and some are NaN."""
    nan = got.isnan()
    assert bool(nan.any()), what
    bad = ~(nan | (got == want))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} wrong values, the first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("mode", [FIRST, SECOND])
@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,K", FEW + ONE + PAIRS + SPLIT)
def test_what_a_lost_operand_leaves_is_nan(M, N, K, act, mode):
    """On the default path, without error words, on outputs and a workspace that held other values before."""
    x, w, res = operands(M, N, K)
    bias = torch.arange(N, device="cuda").remainder(5).float()
    w = (w.float() / 64).to(BF)
    want, zz = sa.sol_attn_linear(x, w, bias, act, res, want_z=True)
    out, z = torch.full_like(want, 7.0), torch.full_like(want, 7.0)
    sa.sol_attn_debug_drop_one_load(mode)
    sa.sol_attn_linear(x, w, bias, act, res, out=out, z=z)
    torch.cuda.synchronize()
    right_or_nan(out, want, "out")
    right_or_nan(z, zz, "z")
    assert torch.equal(out.isnan(), z.isnan())
    again, za = sa.sol_attn_linear(x, w, bias, act, res, want_z=True)
    assert torch.equal(again, want) and torch.equal(za, zz)


@pytest.mark.parametrize("M,N,K", ONE + PAIRS)
def test_what_a_lost_residual_leaves_is_nan(M, N, K):
    x, w, res = operands(M, N, K)
    want, zz = sa.sol_attn_linear(x, w, residual=res, want_z=True)
    out, z = torch.full_like(want, 7.5), torch.full_like(want, 7.5)
    sa.sol_attn_debug_drop_one_load(RESIDUAL)
    sa.sol_attn_linear(x, w, residual=res, out=out, z=z)
    torch.cuda.synchronize()
    right_or_nan(out, want, "out")
    right_or_nan(z, zz, "z")


@pytest.mark.parametrize("mode", [FIRST, SECOND])
@pytest.mark.parametrize("which", ["dx", "dw"])
@pytest.mark.parametrize("M,N,K", [(300, 264, 136), (4104, 4096, 136), (1000, 1024, 1024)])
def test_what_a_lost_operand_of_a_gradient_leaves_is_nan(M, N, K, which, mode):
    x, w, dy = operands(M, N, K)

    def call():
        dx, dw, _ = sa.sol_attn_linear_bwd(dy, x, w, want_dx=which == "dx", want_dw=which == "dw", want_db=False)
        return dx if which == "dx" else dw
    want = call()
    sa.sol_attn_debug_drop_one_load(mode)
    right_or_nan(call(), want, which)
    assert torch.equal(call(), want)
