"""GPU parity of the gated residual and norm, and of its gradients, against the float64 oracle.

Tolerances. A stored bf16 value is off by at most half a step, 2^-8 of its size (fp32: 2^-24); the rest
is fp32 arithmetic, u = 2^-24 per operation. A row sum passes at most 16 additions in a thread and 10
in the shuffles, so with the handful of elementwise operations around it every intermediate is within
64 u of the sum of the magnitudes that enter it; a layer norm's mean is subtracted, so its error
counts relative to the row's mean magnitude. The gradients chain two norms: 256 u of the same kind of
sum. Column sums over rows add at most 200 terms in a row in one chain (64 per block, 37 per thread of
the second pass, 16 at the end): 512 u of the sum of magnitudes, terms included.
"""
import numpy as np
import pytest
import torch

from block_sparse_attention_41_b200 import sol_attn as sa
from oracle import block_oracle as bo

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-6
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
    return None if t is None else t.double().cpu().numpy()


def make(B, T, C, dtype, y=True, gate=True, gain=True, mod=True, post=False, seed=0, offset=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * C + T)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dt = DT[dtype]
    buf = r(B, 6, C) * 0.3
    return {"x": (r(B, T, C) + offset).to(dt), "y": (r(B, T, C) * 2).to(dt) if y else None,
            "gate": buf[:, 2] if y and gate else None, "gain": 1 + 0.1 * r(C) if gain else None,
            "scale": buf[:, 1] if mod else None, "shift": buf[:, 0] if mod else None,
            "post_gain": 1 + 0.1 * r(C) if post else None}


def bounds(a, norm, post, res_scale):
    """Oracle (x', h) and bounds of their fp32 errors."""
    v = {k: _np(t) for k, t in a.items()}
    xo, h = bo.residual_norm(**v, norm=norm, post_norm=post, res_scale=res_scale, eps=EPS)
    e = np.zeros_like(xo)
    if v["y"] is not None:
        ny, ry = bo.normalise(v["y"], post, EPS)
        k = np.abs(v["gate"][:, None]) if v["gate"] is not None else 1.0
        k = k * (np.abs(v["post_gain"]) if v["post_gain"] is not None else 1.0)
        mean = ry * np.abs(v["y"]).mean(-1, keepdims=True) if post == "layer" else 0.0
        e = 64 * U * (np.abs(res_scale * v["x"]) + k * (np.abs(ny) + mean))
    n, r = bo.normalise(xo, norm, EPS)
    en = r * e + r * e.mean(-1, keepdims=True) + np.abs(n) * (r * e * np.abs(n)).mean(-1, keepdims=True) + \
        64 * U * (np.abs(n) + (r * np.abs(xo).mean(-1, keepdims=True) if norm == "layer" else 0.0))
    k = np.abs(v["gain"]) if v["gain"] is not None else 1.0
    if v["scale"] is not None:
        k = k * np.abs(1 + v["scale"][:, None])
    eh = k * en + (64 * U * np.abs(v["shift"][:, None]) if v["shift"] is not None else 0.0)
    return xo, h, e, eh


def close(got, ref, extra, step, what):
    err = np.abs(_np(got) - ref)
    tol = step * np.abs(ref) + extra + 1e-30
    worst = float((err / tol).max())
    assert np.isfinite(_np(got)).all() and worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


def check_forward(a, dtype, norm, post="none", res_scale=1.0, **kw):
    xo, h = sa.sol_attn_residual_norm(**a, norm=norm, post_norm=post, res_scale=res_scale, eps=EPS, **kw)
    torch.cuda.synchronize()
    rx, rh, ex, eh = bounds(a, norm, post, res_scale)
    if a["y"] is None:
        assert xo is a["x"]
    else:
        close(xo, rx, ex, STEP[dtype], "x'")
    close(h, rh, eh, STEP[dtype], "h")
    return xo, h


SIZES = [(1, 1, 1), (1, 1, 8), (2, 3, 7), (3, 1, 64), (1, 5, 129), (2, 33, 256), (1, 9, 257), (2, 7, 768), (1, 3, 1023),
         (1, 4, 2048), (2, 5, 4096), (1, 3, 5120), (1, 3, 5119), (1, 2, 8184), (1, 2, 8191), (1, 2, 8192)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm,post", [("layer", "none"), ("rms", "rms"), ("layer", "layer"), ("rms", "none")])
@pytest.mark.parametrize("B,T,C", SIZES)
def test_forward(B, T, C, norm, post, dtype):
    check_forward(make(B, T, C, dtype, post=post != "none"), dtype, norm, post, res_scale=0.75)


@pytest.mark.parametrize("y,gate,gain,mod,post", [(False, False, False, False, "none"), (False, False, True, True, "none"),
                                                  (True, False, False, False, "none"), (True, True, False, False, "rms"),
                                                  (True, False, True, False, "layer"), (True, False, False, True, "rms")])
@pytest.mark.parametrize("C", [96, 203])
def test_absent_parts(y, gate, gain, mod, post, C):
    for dtype in ("bf16", "f32"):
        a = make(2, 5, C, dtype, y, gate, gain, mod, post=post == "rms")
        check_forward(a, dtype, "rms", post)
        check_backward(a, dtype, "layer", post, dxo=y)


def check_backward(a, dtype, norm, post="none", res_scale=1.0, dxo=True, seed=5):
    B, T, C = a["x"].shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    dh = torch.randn((B, T, C), generator=g, device="cuda").to(DT[dtype])
    dx_out = torch.randn((B, T, C), generator=g, device="cuda").to(DT[dtype]) if dxo else None
    given = {k: v for k, v in a.items() if k != "shift"}
    got = sa.sol_attn_residual_norm_bwd(dh, dx_out=dx_out, norm=norm, post_norm=post, res_scale=res_scale, eps=EPS, **given)
    torch.cuda.synchronize()
    v = {k: _np(t) for k, t in given.items()}
    ref = bo.residual_norm_bwd(_np(dh), dx_out=_np(dx_out), norm=norm, post_norm=post, res_scale=res_scale, eps=EPS, **v)
    want = {"dx", "dy"} & set(ref) | {"d" + k for k in ("gate", "gain", "scale", "post_gain") if a[k] is not None}
    if a["scale"] is not None:
        want.add("dshift")
    assert {k for k, t in got.items() if t is not None} == want
    # magnitudes that enter each value
    xo, _ = bo.residual_norm(v["x"], v["y"], v["gate"], None, None, None, v["post_gain"], norm, post, res_scale, EPS)
    n, r = bo.normalise(xo, norm, EPS)
    off = 1.0 + (r * np.abs(xo).mean(-1, keepdims=True) if norm == "layer" else 0.0)  # what a subtracted mean costs
    k = (np.abs(v["gain"]) if v["gain"] is not None else 1.0) * (np.abs(1 + v["scale"][:, None]) if v["scale"] is not None else 1.0)
    w = np.abs(_np(dh)) * k
    mean = lambda q: q.mean(-1, keepdims=True)  # noqa: E731
    m = off * r * (w + mean(w) + (np.abs(n) + off) * mean(w * (np.abs(n) + off)))
    if dx_out is not None:
        m = m + np.abs(_np(dx_out))
    close(got["dx"], ref["dx"], 256 * U * np.abs(res_scale) * m, STEP[dtype], "dx")
    P = np.abs(_np(dh)) * (np.abs(n) + off)
    if "dshift" in want:
        close(got["dshift"], ref["dshift"], 512 * U * np.abs(_np(dh)).sum(1), U, "dshift")
        close(got["dscale"], ref["dscale"], 512 * U * P.sum(1) * (np.abs(v["gain"]) if v["gain"] is not None else 1), U, "dscale")
    if "dgain" in want:
        s = np.abs(1 + v["scale"][:, None]) if v["scale"] is not None else 1.0
        close(got["dgain"], ref["dgain"], 512 * U * (P * s).sum((0, 1)), U, "dgain")
    if "dy" in want:
        ny, ry = bo.normalise(v["y"], post, EPS)
        offy = 1.0 + (ry * mean(np.abs(v["y"])) if post == "layer" else 0.0)
        ay = np.abs(ny) + (offy if post != "none" else 0.0)
        gate = np.abs(v["gate"][:, None]) if v["gate"] is not None else 1.0
        pg = np.abs(v["post_gain"]) if v["post_gain"] is not None else 1.0
        du = m * gate * pg
        md = du if post == "none" else offy * ry * (du + mean(du) + ay * mean(du * ay))
        close(got["dy"], ref["dy"], 256 * U * md, STEP[dtype], "dy")
        if "dgate" in want:
            close(got["dgate"], ref["dgate"], 512 * U * (m * ay * pg).sum(1), U, "dgate")
        if "dpost_gain" in want:
            close(got["dpost_gain"], ref["dpost_gain"], 512 * U * (m * gate * ay).sum((0, 1)), U, "dpost_gain")
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm,post", [("layer", "none"), ("rms", "rms"), ("layer", "layer"), ("rms", "none")])
@pytest.mark.parametrize("B,T,C", SIZES + [(1, 1500, 128), (3, 700, 320), (5, 1, 512), (2, 1200, 1024)])
def test_backward(B, T, C, norm, post, dtype):
    check_backward(make(B, T, C, dtype, post=post != "none"), dtype, norm, post, res_scale=0.75)


def test_backward_has_the_same_bits_every_time():
    a = make(2, 3000, 640, "bf16", post=True)
    one = check_backward(a, "bf16", "rms", "rms")
    two = check_backward(a, "bf16", "rms", "rms")
    for k in one:
        assert torch.equal(one[k], two[k]), k


def test_rows_of_zeros_and_constants_give_the_shift():
    a = make(1, 4, 512, "f32", y=False)
    a["x"][0, 0] = 0.0
    a["x"][0, 1] = 12345.0
    _, h = sa.sol_attn_residual_norm(**a, norm="layer", eps=EPS)
    assert torch.equal(h[0, 0], a["shift"][0]) and torch.equal(h[0, 1], a["shift"][0])
    _, h = sa.sol_attn_residual_norm(**a, norm="rms", eps=EPS)
    assert torch.equal(h[0, 0], a["shift"][0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [1, 5, 8, 31, 72, 100, 128, 200, 256, 300, 511, 512, 1000, 1032])
def test_many_rows_of_few_channels(C, dtype):
    # full blocks: as many rows side by side as threads, barriers and shared memory allow
    T = 30_000 if C <= 300 else 6000
    a = make(2, T, C, dtype, post=True)
    check_forward(a, dtype, "rms", "rms")
    check_backward(make(1, T // 4, C, dtype, post=True), dtype, "layer", "rms")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [4104, 5376, 6144, 6145, 7680, 7684, 7688, 8184, 8191])
def test_long_ragged_rows(C, dtype):
    # around the sizes where the gradient or the forward changes its threads or leaves the ring out
    a = make(1, 400, C, dtype, post=True)
    check_forward(a, dtype, "layer", "layer")
    check_backward(a, dtype, "rms", "rms")


def test_a_large_common_offset_keeps_its_digits():
    # rows at 1000 with a deviation of 1: a difference of moments in fp32 would lose the variance's digits
    a = make(1, 6, 2048, "f32", y=False, offset=1000.0)
    check_forward(a, "f32", "layer")


def test_a_row_of_nan_stays_a_row():
    a = make(1, 9, 256, "bf16", post=True)
    ref = sa.sol_attn_residual_norm(**a, norm="rms", post_norm="rms")
    a["y"][0, 3, 17] = float("nan")
    a["x"][0, 5, 0] = float("inf")
    got = sa.sol_attn_residual_norm(**a, norm="rms", post_norm="rms")
    for r, g in zip(ref, got):
        keep = [i for i in range(9) if i not in (3, 5)]
        assert torch.equal(g[0, keep], r[0, keep])
        assert g[0, 3].isnan().all()


def test_in_place_and_given_outputs():
    a = make(2, 50, 384, "bf16")
    rx, rh = sa.sol_attn_residual_norm(**a, norm="layer")
    h = torch.full_like(rh, float("nan"))
    x = a["x"].clone()
    gx, gh = sa.sol_attn_residual_norm(**{**a, "x": x}, norm="layer", x_out=x, h=h)
    assert gx is x and gh is h and torch.equal(gx, rx) and torch.equal(gh, rh)


def test_one_shared_row_of_modulation():
    a = make(3, 4, 128, "f32")
    for k in ("gate", "scale", "shift"):
        a[k] = a[k][:1].expand(3, 128)
    check_forward(a, "f32", "layer")
    check_backward(a, "f32", "layer")


def test_more_elements_than_32_bits():
    B, T, C = 1, 420_000, 5120  # 2.15e9 values
    x = torch.zeros((B, T, C), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 209_714, 209_716, T - 2, T - 1]
    x[0, rows] = torch.randn((len(rows), C), device="cuda").to(torch.bfloat16)
    _, h = sa.sol_attn_residual_norm(x, norm="rms")
    _, want = sa.sol_attn_residual_norm(x[:, rows].contiguous(), norm="rms")
    assert torch.equal(h[0, rows], want[0])
    del h
    dh = torch.ones_like(x)
    g = sa.sol_attn_residual_norm_bwd(dh, x, norm="rms")
    small = sa.sol_attn_residual_norm_bwd(dh[:, rows].contiguous(), x[:, rows].contiguous(), norm="rms")
    assert torch.equal(g["dx"][0, rows], small["dx"][0])


def test_streams_and_graphs():
    a = make(2, 300, 640, "bf16", post=True)
    dh = torch.randn_like(a["x"])
    given = {k: v for k, v in a.items() if k != "shift"}

    def both(stream=None):
        xo, h = sa.sol_attn_residual_norm(**a, norm="rms", post_norm="rms", stream=stream)
        g = sa.sol_attn_residual_norm_bwd(dh, dx_out=h, norm="rms", post_norm="rms", stream=stream, **given)
        return [xo, h] + [g[k] for k in sorted(g)]
    ref = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = both(stream)
        s.synchronize()
        assert all(torch.equal(r, g) for r, g in zip(ref, got))
    # two captured graphs replayed at once on two streams: no workspace is shared
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = both()
        graphs.append((g, outs, torch.cuda.Stream()))
    for _ in range(3):
        for g, _, st in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, outs, _ in graphs:
        assert all(torch.equal(r, o) for r, o in zip(ref, outs))


def test_refusals():
    a = make(2, 4, 64, "bf16")
    with pytest.raises(ValueError):
        sa.sol_attn_residual_norm(**{**a, "x": a["x"].transpose(0, 1)})
    with pytest.raises(ValueError):
        sa.sol_attn_residual_norm(**{**a, "y": a["y"][:1]})
    with pytest.raises(TypeError):
        sa.sol_attn_residual_norm(**{**a, "y": a["y"].float()})
    with pytest.raises(TypeError):
        sa.sol_attn_residual_norm(**{**a, "gain": a["gain"].bfloat16()})
    with pytest.raises(ValueError):
        sa.sol_attn_residual_norm(**{**a, "gate": a["gate"][:1]})
    with pytest.raises(ValueError):
        sa.sol_attn_residual_norm(**a, norm="group")
    with pytest.raises(TypeError):
        sa.sol_attn_residual_norm(a["x"].half())
    with pytest.raises(sa.SolAttnError):
        sa.sol_attn_residual_norm(a["x"], gate=a["gate"])
    with pytest.raises(sa.SolAttnError):
        sa.sol_attn_residual_norm(torch.empty((1, 0, 64), device="cuda"))
    with pytest.raises(sa.SolAttnError):
        sa.sol_attn_residual_norm(torch.empty((1, 1, 8200), device="cuda"))
    with pytest.raises(sa.SolAttnError):
        sa.sol_attn_residual_norm_bwd(a["x"], a["x"], a["y"], gate=a["gate"],
                                      workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(sa.SolAttnError):
        sa.sol_attn_residual_norm_bwd(a["x"], a["x"], dx_out=a["x"])
