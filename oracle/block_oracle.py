"""float64 oracle of the dense operators around the attention, in numpy: gated residual and norm,
rotary positions, linear layer, each with its gradients written out from the formula.

Test infrastructure only: it shares no code with the CUDA path. Definitions as in include/sol_attn.h.
"""
from __future__ import annotations

import math

import numpy as np


def _f64(*arrays):
    return tuple(None if a is None else np.asarray(a, dtype=np.float64) for a in arrays)


# ---- gated residual and norm ------------------------------------------------------------------------

def normalise(v, kind, eps):
    """Normalised rows of v and 1 / sqrt(mean square or variance + eps); kind "none" leaves v."""
    if kind == "none":
        return v, np.ones(v.shape[:-1] + (1,))
    if kind == "layer":
        v = v - v.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    return v * r, r


def normalise_back(w, n, r, kind):
    """Gradient of the rows from the gradient w of the normalised rows n."""
    if kind == "none":
        return w
    m = w.mean(-1, keepdims=True) if kind == "layer" else 0.0
    return r * (w - m - n * (w * n).mean(-1, keepdims=True))


def _rows(v):
    return 1.0 if v is None else v[:, None, :]


def residual_norm(x, y=None, gate=None, gain=None, scale=None, shift=None, post_gain=None, norm="layer",
                  post_norm="none", res_scale=1.0, eps=1e-6):
    """(x', h) of [B, T, C] inputs; gate, scale, shift [B, C]; gains [C]."""
    x, y, gate, gain, scale, shift, post_gain = _f64(x, y, gate, gain, scale, shift, post_gain)
    if y is not None:
        u, _ = normalise(y, post_norm, eps)
        if post_gain is not None:
            u = u * post_gain
        x = res_scale * x + _rows(gate) * u
    h, _ = normalise(x, norm, eps)
    if gain is not None:
        h = h * gain
    if scale is not None:
        h = h * (1.0 + scale[:, None, :])
    if shift is not None:
        h = h + shift[:, None, :]
    return x, h


def residual_norm_bwd(dh, x, y=None, gate=None, gain=None, scale=None, post_gain=None, dx_out=None, norm="layer",
                      post_norm="none", res_scale=1.0, eps=1e-6):
    """Gradients as a dict: dx, dy, dgate, dgain, dscale, dshift, dpost_gain (only those that exist)."""
    dh, x, y, gate, gain, scale, post_gain, dx_out = _f64(dh, x, y, gate, gain, scale, post_gain, dx_out)
    xo, _ = residual_norm(x, y, gate, None, None, None, post_gain, norm, post_norm, res_scale, eps)
    n, r = normalise(xo, norm, eps)
    out = {"dshift": dh.sum(1)}
    one = 1.0 if scale is None else 1.0 + scale[:, None, :]
    g = 1.0 if gain is None else gain
    if scale is not None:
        out["dscale"] = (dh * n * g).sum(1)
    if gain is not None:
        out["dgain"] = (dh * n * one).sum((0, 1))
    d = normalise_back(dh * g * one, n, r, norm)
    if dx_out is not None:
        d = d + dx_out
    if y is None:
        out["dx"] = d
        return out
    out["dx"] = res_scale * d
    ny, ry = normalise(y, post_norm, eps)
    pg = 1.0 if post_gain is None else post_gain
    if gate is not None:
        out["dgate"] = (d * ny * pg).sum(1)
    du = d * _rows(gate)
    if post_gain is not None:
        out["dpost_gain"] = (du * ny).sum((0, 1))
    out["dy"] = normalise_back(du * pg, ny, ry, post_norm)
    return out


# ---- rotary positions ---------------------------------------------------------------------------------

def rope_inv_freq(rot, base=10000.0, sections=None, scaling="none", factor=1.0, original_length=8192.0, turns_low=1.0,
                  turns_high=32.0):
    """Angular step of each pair and the factor on cosine and sine."""
    out = []
    for n in (sections if sections is not None else (rot // 2,)):
        for j in range(n):
            b = base * factor ** (n / (n - 1)) if scaling == "ntk" and n > 1 else base
            f = b ** (-j / n)
            if scaling == "linear":
                f /= factor
            if scaling == "yarn":
                wavelength = 2.0 * math.pi / f
                k = min(1.0, max(0.0, (original_length / wavelength - turns_low) / (turns_high - turns_low)))
                f = k * f + (1.0 - k) * f / factor
            out.append(f)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rope_tables(pos, inv_freq, sections=None, factor=1.0):
    """cos, sin float64 [..., L, rot / 2] of positions [..., axes, L] (or [L])."""
    pos = np.asarray(pos)
    if pos.ndim == 1:
        pos = pos[None]
    axis = np.repeat(np.arange(len(sections)), sections) if sections is not None else np.zeros(len(inv_freq), int)
    ang = np.moveaxis(pos.astype(np.float64)[..., axis, :], -2, -1) * np.asarray(inv_freq, dtype=np.float64)
    return factor * np.cos(ang), factor * np.sin(ang)


def rope(x, cos, sin, layout="interleaved", inverse=False):
    """Rows [B, H, L, d] turned by cos, sin [L, rot / 2] or [B, L, rot / 2]."""
    x = np.asarray(x, dtype=np.float64)
    half = cos.shape[-1]
    if cos.ndim == 3:
        cos, sin = cos[:, None], sin[:, None]
    if inverse:
        sin = -sin
    out = x.copy()
    ia, ib = (np.arange(half) * 2, np.arange(half) * 2 + 1) if layout == "interleaved" else \
        (np.arange(half), np.arange(half) + half)
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * cos - b * sin
    out[..., ib] = a * sin + b * cos
    return out


# ---- linear layer ---------------------------------------------------------------------------------------

_erf = np.vectorize(math.erf, otypes=[np.float64])


def activation(z, act):
    z = np.asarray(z, dtype=np.float64)
    if act == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1.0 + np.exp(-z))
    return z


def activation_slope(z, act):
    z = np.asarray(z, dtype=np.float64)
    if act == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        e = 1.0 / (1.0 + np.exp(-z))
        return e * (1.0 + z * (1.0 - e))
    return np.ones_like(z)


def linear(x, w, bias=None, act="none", residual=None):
    """(out, z): z = x w^T + bias, out = residual + act(z); x [M, K], w [N, K]."""
    x, w, bias, residual = _f64(x, w, bias, residual)
    z = x @ w.T
    if bias is not None:
        z = z + bias
    out = activation(z, act)
    return (out if residual is None else residual + out), z


def linear_bwd(dy, x, w, z=None, act="none"):
    """(dx, dw, db) from dy [M, N] and the forward's value z before the activation."""
    dy, x, w = _f64(dy, x, w)
    dz = dy if act == "none" else dy * activation_slope(z, act)
    return dz @ w, dz.T @ x, dz.sum(0)
