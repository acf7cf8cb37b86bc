"""Slopes of the activations over every finite bf16 value, against the float64 oracle.

db of one row is dy act'(z) unrounded, so it shows the fp32 slope itself. Its arithmetic is within 4 act_error(max(|z|, 1)) of
the magnitudes, the bound of tests/test_linear_gpu.py for products of four such factors, up to |z| = 16; beyond that every slope
is 0 or 1 to less than 1e-6 (the density of gelu at 16 is e^-128, silu's 16 e^-16 is 1.8e-6 and counted by the bound).
"""
import numpy as np
import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build
    build.build()
    sa.load_library()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_slopes_of_every_finite_value(act):
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16)
    z = bits.view(torch.bfloat16)
    z = z[torch.isfinite(z)]
    z = torch.cat((z, torch.zeros((-z.numel()) % 8, dtype=z.dtype)))[None].contiguous().cuda()
    dy, x = torch.ones_like(z), torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((z.shape[1], 8), dtype=torch.bfloat16, device="cuda")
    dx, dw, db = sa.sol_attn_linear_bwd(dy, x, w, z, act)
    v = z[0].double().cpu().numpy()
    a = np.clip(v, -700.0, 700.0)  # the oracle's exponentials are finite there and its slopes 0 or 1
    want = bo.activation_slope(a, act)
    m = np.minimum(np.maximum(np.abs(v), 1.0), 16.0)
    tol = 4 * 16 * U * m * (1 + 1.6 * m * (1 + 0.045 * m * m)) + U * np.abs(want)
    got = db.double().cpu().numpy()
    assert np.isfinite(got).all(), v[~np.isfinite(got)][:5]
    bad = np.abs(got - want) > tol
    assert not bad.any(), (v[bad][:5], got[bad][:5], want[bad][:5])
    assert not dx.isnan().any() and not dw.isnan().any()


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_nan_stays_nan(act):
    z = torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    z[0, 3] = float("nan")
    w = torch.zeros((8, 8), dtype=torch.bfloat16, device="cuda")
    _, _, db = sa.sol_attn_linear_bwd(torch.ones_like(z), z, w, z, act, want_dx=False, want_dw=False)
    assert db.isnan().tolist() == [i == 3 for i in range(8)]
