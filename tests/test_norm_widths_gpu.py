"""Norm and its gradient just within and just past the widths at which fp32 rows leave the ring of asynchronous
copies (5120 channels of the gradient, 7680 of the forward), with enough rows for every block to take several.
Tolerances and references are those of tests/test_norm_gpu.py."""
import pytest
import torch
from test_norm_gpu import check_backward, check_forward, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_sparse_attention_41_b200 import build, sol_attn
    build.build()
    sol_attn.load_library()


@pytest.mark.parametrize("norm,post", [("layer", "none"), ("rms", "rms")])
@pytest.mark.parametrize("C", [5116, 5120, 5124])
def test_gradient(C, norm, post):
    check_backward(make(2, 450, C, "f32", post=post != "none"), "f32", norm, post)


@pytest.mark.parametrize("norm,post", [("layer", "layer"), ("rms", "none")])
@pytest.mark.parametrize("C", [7676, 7680, 7684])
def test_forward(C, norm, post):
    check_forward(make(2, 450, C, "f32", post=post != "none"), "f32", norm, post)
