"""A whole video-transformer block out of the library's calls, as a user strings them together:
modulation from the timestep, norm, projection, rotary positions, attention, output projection, gated
residual and norm, MLP onto the residual stream; and the backward pass of its dense half.

Against float64 from the same weights. Between input and output a value is stored in bf16 twelve times
(h, qkv, q and k, o, attention's p, its projection, x', h', the MLP's middle, its product, the sum), each time off
by at most 2^-8 of it; norms, attention and products carry an error on in the proportion in which
they carry the value. So 12 x 2^-8 bounds the relative error in the 2-norm, and the gradients, which pass eight
such roundings beside the forward's, are held to 20 x 2^-8.
"""
import math

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


def weights(B, T, H, d, seed=0):
    C = H * d
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s, a=1.0, dt=BF):
        return (torch.randn(s, generator=g, device="cuda") * a).to(dt)
    f, _ = sa.sol_attn_rope_inv_freq(d, sections=(d // 2 - 2 * (d // 6), d // 6, d // 6), device="cuda")
    t = torch.arange(T, device="cuda")
    return {"x": r(B, T, C), "t": r(B, C), "w_mod": r(6 * C, C, a=0.3 * C ** -0.5), "b_mod": r(6 * C, a=0.1, dt=torch.float32),
            "w_qkv": r(3 * C, C, a=C ** -0.5), "b_qkv": r(3 * C, a=0.1, dt=torch.float32), "w_o": r(C, C, a=C ** -0.5),
            "w_1": r(4 * C, C, a=C ** -0.5), "b_1": r(4 * C, a=0.1, dt=torch.float32), "w_2": r(C, 4 * C, a=(4 * C) ** -0.5),
            "f": f, "sections": (d // 2 - 2 * (d // 6), d // 6, d // 6),
            "pos": torch.stack((t // 64, t // 8 % 8, t % 8)).to(torch.int32)}


def block(p, H, tau):
    B, T, C = p["x"].shape
    d = C // H
    mod = sa.sol_attn_linear(p["t"], p["w_mod"], p["b_mod"]).float().view(B, 6, C)
    _, h = sa.sol_attn_residual_norm(p["x"], shift=mod[:, 0], scale=mod[:, 1])
    qkv = sa.sol_attn_linear(h, p["w_qkv"], p["b_qkv"]).view(B, T, 3 * H, d).transpose(1, 2)
    q, k = sa.sol_attn_rope(qkv[:, :H], qkv[:, H:2 * H], p["pos"], p["f"], sections=p["sections"])
    o, _, _ = sa.sol_attn(q, k, qkv[:, 2 * H:].contiguous(), [tau] * H)
    y = sa.sol_attn_linear(o.transpose(1, 2).reshape(B, T, C), p["w_o"])
    x1, h1 = sa.sol_attn_residual_norm(p["x"], y, gate=mod[:, 2], shift=mod[:, 3], scale=mod[:, 4])
    m, z = sa.sol_attn_linear(h1, p["w_1"], p["b_1"], act="gelu_tanh", want_z=True)
    out = sa.sol_attn_linear(m, p["w_2"], residual=x1)
    return {"mod": mod, "y": y, "x1": x1, "h1": h1, "m": m, "z": z, "out": out}


def norm64(v):
    return (v - v.mean(-1, keepdim=True)) / torch.sqrt(v.var(-1, correction=0, keepdim=True) + 1e-6)


def dense_half64(p, mod, y, x):
    x1 = x + mod[:, 2, None] * y
    h1 = norm64(x1) * (1 + mod[:, 4, None]) + mod[:, 3, None]
    m = torch.nn.functional.gelu(h1 @ p["w_1"].double().T + p["b_1"].double(), approximate="tanh")
    return x1 + m @ p["w_2"].double().T


def block64(p, H):
    B, T, C = p["x"].shape
    d = C // H
    mod = (p["t"].double() @ p["w_mod"].double().T + p["b_mod"].double()).view(B, 6, C)
    x = p["x"].double()
    h = norm64(x) * (1 + mod[:, 1, None]) + mod[:, 0, None]
    qkv = (h @ p["w_qkv"].double().T + p["b_qkv"].double()).view(B, T, 3 * H, d).transpose(1, 2)
    axis = torch.repeat_interleave(torch.arange(3), torch.tensor(p["sections"])).cuda()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), p["pos"].double()[axis].T * p["f"])
    q, k = (torch.view_as_real(torch.view_as_complex(v.reshape(B, H, T, d // 2, 2).contiguous()) * turn).flatten(-2)
            for v in (qkv[:, :H], qkv[:, H:2 * H]))
    o = torch.softmax(q @ k.transpose(-1, -2) / math.sqrt(d), -1) @ qkv[:, 2 * H:]
    y = o.transpose(1, 2).reshape(B, T, C) @ p["w_o"].double().T
    return dense_half64(p, mod, y, x)


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("B,T,H,d", [(1, 700, 4, 64), (2, 515, 2, 128), (1, 129, 6, 64)])
def test_block_against_64_bits(B, T, H, d):
    p = weights(B, T, H, d)
    got = block(p, H, math.inf)
    assert rel(got["out"], block64(p, H)) <= 12 * 2.0 ** -8


def backward(p, f, dout):
    """Gradient of the block's dense half from that of its output: dx1 reaches the stream twice."""
    dm, dw2, _ = sa.sol_attn_linear_bwd(dout, f["m"], p["w_2"], want_db=False)
    dh1, dw1, db1 = sa.sol_attn_linear_bwd(dm, f["h1"], p["w_1"], f["z"], "gelu_tanh")
    mod = f["mod"]
    g = sa.sol_attn_residual_norm_bwd(dh1, p["x"], f["y"], gate=mod[:, 2], scale=mod[:, 4], dx_out=dout)
    return {"w_1": dw1, "b_1": db1, "w_2": dw2, "x": g["dx"], "y": g["dy"], "gate": g["dgate"], "scale": g["dscale"],
            "shift": g["dshift"]}


def test_backward_of_the_dense_half_against_64_bits():
    p = weights(2, 515, 2, 128, seed=3)
    f = block(p, 2, 1.5)
    dout = torch.randn_like(p["x"])
    got = backward(p, f, dout)
    leaf = {k: p[k].double().requires_grad_(True) for k in ("w_1", "b_1", "w_2", "x")}
    y, mod = f["y"].double().requires_grad_(True), f["mod"].double().requires_grad_(True)
    out = dense_half64({**p, **leaf}, mod, y, leaf["x"])
    out.backward(dout.double())
    want = {**{k: v.grad for k, v in leaf.items()}, "y": y.grad, "gate": mod.grad[:, 2], "shift": mod.grad[:, 3], "scale": mod.grad[:, 4]}
    for k in want:
        assert got[k].shape == want[k].shape, k
        assert rel(got[k], want[k]) <= 20 * 2.0 ** -8, (k, rel(got[k], want[k]))


def test_a_captured_block_repeats_on_new_inputs():
    """Forward and backward captured once, replayed on other inputs, against an eager run; another graph
    of the same calls is replayed beside it, and an eager graph of the same leaves lives meanwhile."""
    p = weights(1, 300, 4, 64, seed=5)
    dout = torch.randn_like(p["x"])

    def step():
        f = block(p, 4, 1.0)
        return {**{k: f[k] for k in ("out", "x1")}, **backward(p, f, dout)}
    leaf = p["w_2"].detach().requires_grad_(True)
    alive = (leaf.float() * 2).sum()  # an autograd graph over the same memory
    step()
    side = torch.cuda.Stream()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = step()
        graphs.append((g, o))
    for seed in (7, 8):
        new = weights(1, 300, 4, 64, seed=seed)
        for k in ("x", "t", "w_1"):
            p[k].copy_(new[k])
        torch.cuda.synchronize()
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        torch.cuda.synchronize()
        want = step()
        for _, o in graphs:
            for k, v in want.items():
                assert torch.equal(v, o[k]), k
    alive.backward()
    assert bool((leaf.grad == 2).all())


def test_two_streams_at_once():
    ps = [weights(1, 600, 4, 64, seed=s) for s in (11, 12)]
    want = [block(p, 4, 1.0)["out"] for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[], []]
    for _ in range(5):
        for i, (p, s) in enumerate(zip(ps, streams)):
            with torch.cuda.stream(s):
                got[i].append(block(p, 4, 1.0)["out"])
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)
