"""Arguments that are missing or no tensors at all are refused by name, like wrong ones."""
import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build
    build.build()
    sa.load_library()


@pytest.mark.parametrize("bad", [None, 3.0, [1, 2]])
def test_missing_tensors(bad):
    x, w = torch.ones((4, 64), device="cuda", dtype=BF), torch.ones((72, 64), device="cuda", dtype=BF)
    dy, t = torch.ones((4, 72), device="cuda", dtype=BF), torch.ones((1, 4, 64), device="cuda", dtype=BF)
    q = torch.ones((1, 2, 8, 64), device="cuda", dtype=BF)
    f, _ = sa.sol_attn_rope_inv_freq(64, device="cuda")
    pos = torch.arange(8, dtype=torch.int32, device="cuda")
    calls = {"x": [lambda: sa.sol_attn_linear(bad, w), lambda: sa.sol_attn_linear_bwd(dy, bad, w), lambda: sa.sol_attn_residual_norm(bad),
                   lambda: sa.sol_attn_residual_norm_bwd(t, bad)],
             "w": [lambda: sa.sol_attn_linear(x, bad), lambda: sa.sol_attn_linear_bwd(dy, x, bad)],
             "dy": [lambda: sa.sol_attn_linear_bwd(bad, x, w)], "dh": [lambda: sa.sol_attn_residual_norm_bwd(bad, t)],
             "Q": [lambda: sa.sol_attn_rope(bad, None, pos, f)],
             "pos": [lambda: sa.sol_attn_rope(q, q, bad, f), lambda: sa.sol_attn_rope_tables(bad, f)],
             "inv_freq": [lambda: sa.sol_attn_rope(q, q, pos, bad), lambda: sa.sol_attn_rope(q, q, pos[None], bad),
                          lambda: sa.sol_attn_rope_tables(pos, bad), lambda: sa.sol_attn_rope_tables(pos[None], bad)]}
    for name, some in calls.items():
        for call in some:
            with pytest.raises(TypeError, match=name):
                call()
