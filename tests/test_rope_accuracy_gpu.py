"""Cosine and sine of the rotary tables against 80-bit extended precision.

The bound, in units of 2^-24 and with a factor of 1. The angle is cut to 2^-32 of a turn twice: 0.1. Its remainder of at most
pi / 4 is converted to fp32, multiplied by a rounded constant, and rounded: three relative halves of 2^-23, so 3 pi / 4 = 2.4, which
a slope of at most 0.71 at that end (x cos x and x sin x are below 0.56 anywhere) carries as 1.7. The polynomial's last step rounds
a value below 1, its steps before that come in with a factor of at most q / 2 = 0.31 of one such rounding: 0.8 together; the factor's
multiplication rounds once more: 0.5. That is 3.1, held to 4. Farther out the rounding of frequency / 2 pi in 64 bits
counts: 0.16 * 1.5 * 2^-53 turns per position, 6.0 at 2^31, so 10 there.
"""
import numpy as np
import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build
    build.build()
    sa.load_library()


@pytest.mark.parametrize("first,step,bound", [(0, 1, 4), (1_000_003, 7, 4), (9_900_000, 1, 4), (-9_999_999, 3, 4), (2**31 - 40_000, 1, 10),
                                              (-2**31, 1, 10)])
def test_tables(first, step, bound):
    if np.finfo(np.longdouble).nmant < 63:
        pytest.skip("no extended precision on this machine")
    L = 30_000
    f, _ = sa.sol_attn_rope_inv_freq(128, device="cuda")
    pos = torch.arange(L, dtype=torch.int64) * step + first
    cos, sin = sa.sol_attn_rope_tables(pos.to(torch.int32).cuda(), f)
    angle = pos.numpy().astype(np.longdouble)[:, None] * f.cpu().numpy().astype(np.longdouble)
    for got, want in ((cos, np.cos(angle)), (sin, np.sin(angle))):
        err = np.abs(got.cpu().numpy().astype(np.longdouble) - want).max()
        assert err <= bound * 2.0 ** -24, float(err * 2 ** 24)
