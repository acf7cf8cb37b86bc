"""Pins of the float64 oracle of the dense operators: hand-worked values, library routines, and each
written-out gradient against central differences."""
import math

import numpy as np
import pytest
import torch

from oracle import block_oracle as bo


def _num_grad(f, a, eps=1e-6):
    """Central differences of the scalar f() with respect to every element of a (changed in place)."""
    g = np.zeros_like(a)
    for i in np.ndindex(a.shape):
        keep = a[i]
        a[i] = keep + eps
        hi = f()
        a[i] = keep - eps
        lo = f()
        a[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


def test_norms_by_hand():
    x = np.array([[[3.0, -1.0, 1.0, 1.0]]])
    # mean 1, variance (4 + 4 + 0 + 0) / 4 = 2; mean square 12 / 4 = 3
    assert np.allclose(bo.residual_norm(x, norm="layer", eps=1e-30)[1], [[[math.sqrt(2), -math.sqrt(2), 0, 0]]])
    assert np.allclose(bo.residual_norm(x, norm="rms", eps=1e-30)[1], np.array([[[3, -1, 1, 1]]]) / math.sqrt(3))


def test_residual_step_by_hand():
    # rms of y = (3, 4) is sqrt(12.5); x' = 2 x + gate post(y) gain
    x, y = np.array([[[1.0, 2.0]]]), np.array([[[3.0, 4.0]]])
    xo, h = bo.residual_norm(x, y, gate=np.array([[0.5, 2.0]]), scale=np.array([[1.0, 0.0]]),
                             shift=np.array([[0.0, 7.0]]), post_gain=np.array([1.0, 3.0]), norm="rms", post_norm="rms",
                             res_scale=2.0, eps=1e-30)
    want = np.array([2 + 0.5 * 3 / math.sqrt(12.5), 4 + 6 * 4 / math.sqrt(12.5)])
    assert np.allclose(xo[0, 0], want)
    r = math.sqrt((want ** 2).mean())
    assert np.allclose(h[0, 0], [2 * want[0] / r, want[1] / r + 7])


def test_norms_against_the_library():
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((2, 3, 17)) + 5, rng.standard_normal(17)
    t = torch.from_numpy(x)
    ln = torch.nn.functional.layer_norm(t, (17,), torch.from_numpy(g), None, 1e-5).numpy()
    assert np.allclose(bo.residual_norm(x, gain=g, norm="layer", eps=1e-5)[1], ln, atol=1e-13)
    rn = torch.nn.functional.rms_norm(t, (17,), torch.from_numpy(g), 1e-5).numpy()
    assert np.allclose(bo.residual_norm(x, gain=g, norm="rms", eps=1e-5)[1], rn, atol=1e-13)


@pytest.mark.parametrize("norm,post", [("layer", "none"), ("rms", "rms"), ("layer", "layer"), ("rms", "none")])
def test_residual_norm_gradients_against_differences(norm, post):
    rng = np.random.default_rng(7)
    B, T, C = 2, 3, 5
    a = {"x": rng.standard_normal((B, T, C)), "y": rng.standard_normal((B, T, C)), "gate": rng.standard_normal((B, C)),
         "gain": rng.standard_normal(C), "scale": rng.standard_normal((B, C)), "shift": rng.standard_normal((B, C))}
    if post != "none":
        a["post_gain"] = rng.standard_normal(C)
    dh, dxo = rng.standard_normal((B, T, C)), rng.standard_normal((B, T, C))
    kw = dict(norm=norm, post_norm=post, res_scale=0.7, eps=1e-3)

    def loss():
        xo, h = bo.residual_norm(**a, **kw)
        return float((dh * h).sum() + (dxo * xo).sum())
    got = bo.residual_norm_bwd(dh, dx_out=dxo, **{k: v for k, v in a.items() if k != "shift"}, **kw)
    assert set(got) == {"d" + k for k in a}
    for k, v in a.items():
        assert np.allclose(got["d" + k], _num_grad(loss, v), rtol=1e-6, atol=1e-7), k


def test_norm_gradient_without_a_branch_against_differences():
    rng = np.random.default_rng(8)
    x, dh = rng.standard_normal((1, 2, 6)), rng.standard_normal((1, 2, 6))
    got = bo.residual_norm_bwd(dh, x, norm="layer", eps=1e-3)
    assert set(got) == {"dx", "dshift"}
    assert np.allclose(got["dx"], _num_grad(lambda: float((dh * bo.residual_norm(x, norm="layer", eps=1e-3)[1]).sum()), x),
                       atol=1e-7)


def test_rope_by_hand_in_both_layouts():
    # one pair per axis of two; position (3, 1): angles 3 and 1
    cos, sin = bo.rope_tables(np.array([[3], [1]]), np.array([1.0, 1.0]), sections=(1, 1))
    x = np.array([1.0, 0.0, 0.0, 2.0, 9.0]).reshape(1, 1, 1, 5)
    inter = bo.rope(x, cos, sin)[0, 0, 0]
    assert np.allclose(inter, [math.cos(3), math.sin(3), -2 * math.sin(1), 2 * math.cos(1), 9.0])
    half = bo.rope(x, cos, sin, "half")[0, 0, 0]
    assert np.allclose(half, [math.cos(3), -2 * math.sin(1), math.sin(3), 2 * math.cos(1), 9.0])


@pytest.mark.parametrize("layout", ["interleaved", "half"])
def test_rope_scores_depend_on_distance_only_and_the_inverse_is_the_gradient(layout):
    rng = np.random.default_rng(3)
    f, m = bo.rope_inv_freq(8, scaling="yarn", factor=4.0, original_length=64.0)
    q, k = rng.standard_normal((2, 10))
    at = lambda v, p: bo.rope(v.reshape(1, 1, 1, 10), *bo.rope_tables(np.array([p]), f, None, m), layout)[0, 0, 0]  # noqa: E731
    assert np.isclose(at(q, 5) @ at(k, 2), at(q, 905) @ at(k, 902))
    cos, sin = bo.rope_tables(np.array([5]), f, None, m)
    dy = rng.standard_normal(10)
    num = _num_grad(lambda: float(at(q, 5) @ dy), q)
    assert np.allclose(bo.rope(dy.reshape(1, 1, 1, 10), cos, sin, layout, inverse=True)[0, 0, 0], num, atol=1e-8)


def test_rope_frequencies_of_long_contexts():
    plain, one = bo.rope_inv_freq(16)
    assert one == 1.0 and np.allclose(plain, 10000.0 ** (-np.arange(8) / 8))
    assert np.allclose(bo.rope_inv_freq(16, scaling="linear", factor=4.0)[0], plain / 4)
    ntk = bo.rope_inv_freq(16, scaling="ntk", factor=4.0)[0]
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], plain[-1] / 4)  # fastest kept, slowest stretched by the factor
    yarn, m = bo.rope_inv_freq(16, scaling="yarn", factor=4.0, original_length=1000.0, turns_low=1.0, turns_high=32.0)
    turns = 1000.0 * plain / (2 * math.pi)
    assert np.allclose(yarn[turns >= 32], plain[turns >= 32]) and np.allclose(yarn[turns <= 1], plain[turns <= 1] / 4)
    assert np.isclose(m, 0.1 * math.log(4.0) + 1)


@pytest.mark.parametrize("act", ["none", "gelu", "gelu_tanh", "silu"])
def test_linear_and_its_gradients(act):
    rng = np.random.default_rng(11)
    x, w, b, res = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), rng.standard_normal(5), rng.standard_normal((3, 5))
    t = torch.nn.functional.linear(torch.from_numpy(x), torch.from_numpy(w), torch.from_numpy(b))
    lib = {"none": lambda v: v, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
           "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](t).numpy() + res
    out, z = bo.linear(x, w, b, act, res)
    assert np.allclose(out, lib, atol=1e-12) and np.allclose(z, t.numpy())
    dy = rng.standard_normal((3, 5))
    dx, dw, db = bo.linear_bwd(dy, x, w, z, act)
    loss = lambda: float((dy * bo.linear(x, w, b, act, res)[0]).sum())  # noqa: E731
    for got, v in ((dx, x), (dw, w), (db, b)):
        assert np.allclose(got, _num_grad(loss, v), rtol=1e-6, atol=1e-7)
