"""The dense operators around the sparse attention of a video diffusion transformer block: what is
measured of them, on which cases, with their plain forms.

Three operators, each in every direction that it has:

* residual norm: ``x' = a x + gate * post(y)`` and ``h = norm(x') * gain * (1 + scale) + shift``, the
  step between two halves of a block, and its gradients;
* rotary positions of queries and keys (both pair layouts, part of the head, several position
  axes, scaled frequencies), its inverse (the gradient), and the cosine and sine tables;
* linear layer ``residual + act(x w^T + bias)``, and its gradients.

``own`` chooses between the plain forms (elementary torch operations in 32 bits, rounded once at
the end) and the library's entry points. ``exact`` states each operator in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------------------------

def _norm_case(name, op, B, T, C, dtype, norm, post="none", y=True, gate=True, gain=False, mod=True):
    return {"name": name, "op": op, "B": B, "T": T, "C": C, "dtype": dtype, "norm": norm, "post": post, "y": y,
            "gate": gate, "gain": gain, "mod": mod}


def _rope_case(name, B, Hq, Hk, L, d, rot, dtype, layout, axes, scaling="none", factor=1.0, start=0, inverse=False):
    return {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hk": Hk, "L": L, "d": d, "rot": rot, "dtype": dtype,
            "layout": layout, "axes": axes, "scaling": scaling, "factor": factor, "start": start, "inverse": inverse}


def _linear_case(name, op, M, K, N, act, bias=True, residual=False):
    return {"name": name, "op": op, "M": M, "K": K, "N": N, "act": act, "bias": bias, "residual": residual}


def listed():
    return [
        # between attention and MLP of the 720p video (40 heads of 128): gated residual, layer norm, modulation
        _norm_case("norm_720p", "norm", 1, 75600, 5120, "bf16", "layer"),
        # one conditioning token of each of four requests: latency
        _norm_case("norm_token", "norm", 4, 1, 4096, "bf16", "rms", post="rms", gain=True),
        # training step of the joint text and video block with a guidance pair (32 heads of 128), norms on both sides
        _norm_case("norm_bwd_cfg", "norm_bwd", 2, 33272, 4096, "bf16", "rms", post="rms", gain=True),
        # training step of the small video transformer (12 heads of 64) in fp32
        _norm_case("norm_bwd_small_f32", "norm_bwd", 1, 8192, 768, "f32", "layer"),
        # queries and keys of the 720p video out of the token-major projection, three position axes
        _rope_case("rope_720p", 1, 40, 40, 75600, 128, 128, "bf16", "interleaved", 3),
        # gradient of the half layout on half of each head, positions stretched over a long context, fp32
        _rope_case("rope_bwd_partial_f32", 2, 32, 32, 33272, 128, 64, "f32", "half", 1, "yarn", 8.0, 0, True),
        # one new token per request far into a long context: latency
        _rope_case("rope_token", 2, 40, 8, 1, 128, 128, "bf16", "half", 1, "linear", 4.0, 1000003),
        # cosine and sine tables of the 1080p video, the input of the fused norm and rotary pass
        {"name": "rope_tables_1080p", "op": "rope_tables", "L": 252960, "rot": 128, "axes": 3, "scaling": "none",
         "factor": 1.0, "start": 0},
        # first matrix of the MLP of the joint text and video block
        _linear_case("linear_mlp_gelu", "linear", 33272, 4096, 16384, "gelu_tanh"),
        # output projection of the small video transformer onto its residual, ragged token count
        _linear_case("linear_out_residual", "linear", 8191, 768, 768, "none", residual=True),
        # six modulation vectors of the 720p block from one timestep token of a guidance pair
        _linear_case("linear_modulation", "linear", 2, 5120, 30720, "none"),
        # training step of a square projection of the joint text and video block
        _linear_case("linear_bwd_gelu", "linear_bwd", 33272, 4096, 4096, "gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "rope", "rope", "rope_tables", "linear", "linear", "linear_bwd"])
    if op in ("norm", "norm_bwd"):
        B, dtype = rng.randint(1, 4), rng.choice(["bf16", "bf16", "f32"])
        C = _log(rng, 64, 8192)
        if rng.random() < 0.75:
            C = max(8, C // 8 * 8)
        most = 75600 * 5120 // (B * C * (1 if dtype == "bf16" else 2) * (1 if op == "norm" else 2))
        T = _log(rng, 1, max(2, min(75600, most)))
        y = rng.random() < 0.8
        c = _norm_case("", op, B, T, C, dtype, rng.choice(["layer", "rms"]),
                       post=rng.choice(["none", "layer", "rms"]) if y else "none", y=y,
                       gate=y and rng.random() < 0.7, gain=rng.random() < 0.5, mod=rng.random() < 0.7)
    elif op == "rope":
        B, d, dtype = rng.randint(1, 2), rng.choice([64, 96, 128, 256]), rng.choice(["bf16", "bf16", "f32"])
        Hk = rng.choice([1, 2, 4, 8, 12])
        Hq = Hk * rng.choice([1, 1, 2, 4])
        axes = rng.choice([1, 3])
        rot = rng.choice([d, d, d // 2, 2 * rng.randint(3, d // 2)])
        most = 75600 * 80 * 128 // (B * (Hq + Hk) * d * (1 if dtype == "bf16" else 2))
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        c = _rope_case("", B, Hq, Hk, _log(rng, 1, max(2, min(75600, most))), d, rot, dtype,
                       rng.choice(["interleaved", "half"]), axes, scaling,
                       1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                       rng.choice([0, 0, _log(rng, 1000, 1000000)]), rng.random() < 0.4)
    elif op == "rope_tables":
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        c = {"op": op, "L": _log(rng, 1, 252960), "rot": 2 * rng.randint(3, 64), "axes": rng.choice([1, 3]),
             "scaling": scaling, "factor": 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
             "start": rng.choice([0, _log(rng, 1000, 1000000)])}
    else:
        K, N = 8 * _log(rng, 8, 1024), 8 * _log(rng, 8, 2048)
        M = _log(rng, 1, max(2, min(33272, 33272 * 4096 * 16384 // (K * N * (2 if op == "linear_bwd" else 1)))))
        c = _linear_case("", op, M, K, N, rng.choice(["none", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.8,
                         residual=op == "linear" and rng.random() < 0.4)
    c.pop("name", None)
    return c


# ---- inputs --------------------------------------------------------------------------------------

def _sections(half, axes):
    """Pairs per position axis: all on one, or split over (t, y, x) with the remainder on t."""
    if axes == 1:
        return (half,)
    n = half // 3
    return (half - 2 * n, n, n)


def _frequencies(rot, axes, scaling, factor, base=10000.0, original=8192):
    """float64 [rot / 2] angular step of each pair per position, and the factor on cosine and sine."""
    out = []
    for n in _sections(rot // 2, axes):
        if n == 0:
            continue
        j = np.arange(n, dtype=np.float64)
        b = base * factor ** (n / (n - 1)) if scaling == "ntk" and n > 1 else base
        f = b ** (-j / n)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            turns = original * f / (2 * math.pi)
            keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
            f = f * keep + f / factor * (1.0 - keep)
        out.append(f)
    return np.concatenate(out), (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def _positions(L, axes, start):
    """int32 [axes, L]: consecutive tokens, or a row-major (t, y, x) grid of 40-wide, 24-high frames."""
    i = np.arange(L, dtype=np.int64)
    p = [i + start] if axes == 1 else [i // 960 + start, i // 40 % 24, i % 40]
    return torch.from_numpy(np.stack(p).astype(np.int32)).to(DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape, scale=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).mul_(scale).to(dtype)

    s = {"case": case}
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        B, T, C, dt = case["B"], case["T"], case["C"], DTYPES[case["dtype"]]
        spread = torch.exp(rand(C, scale=0.5))  # channels of a residual stream differ in size
        s["x"] = (rand(B, T, C) * spread + rand(C, scale=0.3)).to(dt)
        s["y"] = (rand(B, T, C) * spread).to(dt) if case["y"] else None
        mod = rand(B, 6, C, scale=0.3)  # the block's six modulation vectors, one buffer
        s["shift"], s["scale"] = (mod[:, 0], mod[:, 1]) if case["mod"] else (None, None)
        s["gate"] = mod[:, 2] if case["gate"] else None
        s["gain"] = 1.0 + rand(C, scale=0.1) if case["gain"] else None
        s["post_gain"] = 1.0 + rand(C, scale=0.1) if case["post"] != "none" else None
        if op == "norm_bwd":
            s["dh"] = rand(B, T, C).to(dt)
            s["dx_out"] = rand(B, T, C).to(dt) if case["y"] else None
    elif op == "rope":
        B, Hq, Hk, L, d = (case[k] for k in ("B", "Hq", "Hk", "L", "d"))
        dt = DTYPES[case["dtype"]]
        f, s["factor"] = _frequencies(case["rot"], case["axes"], case["scaling"], case["factor"])
        s["inv_freq"] = torch.from_numpy(f).to(DEV)
        s["sections"] = _sections(case["rot"] // 2, case["axes"])
        s["pos"] = _positions(L, case["axes"], case["start"])
        if case["inverse"]:  # gradients come head-major, as the attention has them
            s["q"], s["k"] = rand(B, Hq, L, d, dtype=dt), rand(B, Hk, L, d, dtype=dt)
        else:  # queries, keys and values come token-major out of one projection
            qkv = rand(B, L, Hq + 2 * Hk, d, dtype=dt)
            s["q"], s["k"] = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
    elif op == "rope_tables":
        f, s["factor"] = _frequencies(case["rot"], case["axes"], case["scaling"], case["factor"])
        s["inv_freq"] = torch.from_numpy(f).to(DEV)
        s["sections"] = _sections(case["rot"] // 2, case["axes"])
        # another seed is another crop of the video
        s["pos"] = _positions(case["L"], case["axes"], case["start"] + seed % 1000)
    else:
        M, K, N = case["M"], case["K"], case["N"]
        bf = torch.bfloat16
        s["x"], s["w"] = rand(M, K, dtype=bf), rand(N, K, scale=K ** -0.5, dtype=bf)
        s["bias"] = rand(N, scale=0.3) if case["bias"] else None
        s["residual"] = rand(M, N, dtype=bf) if case["residual"] else None
        if op == "linear_bwd":
            s["dy"] = rand(M, N, dtype=bf)
            # what the forward pass kept: its value before the activation
            s["z"] = rand(M, N, dtype=bf) if case["act"] != "none" else None
    return s


# ---- one pass ------------------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from block_sparse_attention_41_b200 import sol_attn as sa

    c = s["case"]
    op = c["op"]
    if op == "norm":
        x, h = sa.sol_attn_residual_norm(s["x"], s["y"], gate=s["gate"], gain=s["gain"], scale=s["scale"],
                                         shift=s["shift"], post_gain=s["post_gain"], norm=c["norm"],
                                         post_norm=c["post"], eps=EPS)
        return {"x": x, "h": h} if c["y"] else {"h": h}
    if op == "norm_bwd":
        g = sa.sol_attn_residual_norm_bwd(s["dh"], s["x"], s["y"], gate=s["gate"], gain=s["gain"], scale=s["scale"],
                                          post_gain=s["post_gain"], dx_out=s["dx_out"], norm=c["norm"],
                                          post_norm=c["post"], eps=EPS)
        return {k: v for k, v in g.items() if v is not None}
    if op == "rope":
        kw = {}
        if c["inverse"]:  # into the token-major gradient of the projection
            B, Hq, Hk, L, d = (c[k] for k in ("B", "Hq", "Hk", "L", "d"))
            dqkv = torch.empty((B, L, Hq + 2 * Hk, d), dtype=s["q"].dtype, device=DEV)
            kw = {"Q_out": dqkv[:, :, :Hq].transpose(1, 2), "K_out": dqkv[:, :, Hq:Hq + Hk].transpose(1, 2)}
        return sa.sol_attn_rope(s["q"], s["k"], s["pos"], s["inv_freq"], layout=c["layout"], sections=s["sections"],
                                attn_factor=s["factor"], inverse=c["inverse"], **kw)
    if op == "rope_tables":
        return sa.sol_attn_rope_tables(s["pos"], s["inv_freq"], sections=s["sections"], attn_factor=s["factor"])
    if op == "linear":
        return sa.sol_attn_linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"])
    dx, dw, db = sa.sol_attn_linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], act=c["act"], want_db=c["bias"])
    return {"dx": dx, "dw": dw, "db": db} if c["bias"] else {"dx": dx, "dw": dw}


# ---- plain forms: 32 bits, rounded once at the end --------------------------------------------------

def _center(v, kind):
    return v - v.mean(-1, keepdim=True) if kind == "layer" else v


def _normed(v, kind):
    """The normalised rows and the reciprocal of their root mean square."""
    v = _center(v, kind)
    r = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * r, r


def _norm_back(w, n, r, kind):
    """Gradient of the rows, from the gradient w of the normalised rows n."""
    return r * (_center(w, kind) - n * (w * n).mean(-1, keepdim=True))


def _norm_forward(s):
    """x' and what leads to it: post(y) before its gain, its reciprocal deviation, post(y), the gate."""
    c = s["case"]
    x = s["x"].float()
    if s["y"] is None:
        return x, None, None, None, None
    n, r = (s["y"].float(), None) if c["post"] == "none" else _normed(s["y"].float(), c["post"])
    u = n if c["post"] == "none" else n * s["post_gain"]
    gate = s["gate"][:, None] if s["gate"] is not None else None
    return x + (u if gate is None else gate * u), n, r, u, gate


def _angles(s, pos):
    """float64 [L, rot / 2]: position times frequency, each pair on its own axis."""
    parts, at = [], 0
    for a, n in enumerate(s["sections"]):
        parts.append(pos[a].double()[:, None] * s["inv_freq"][at:at + n])
        at += n
    return torch.cat(parts, 1)


def _rotate(x, cos, sin, layout, rot):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if layout == "interleaved" else (x[..., :rot // 2], x[..., rot // 2:rot])
    p, q = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((p, q), -1).flatten(-2) if layout == "interleaved" else torch.cat((p, q), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1.0 + torch.exp(-z)) if act == "silu" else z


def _act_slope(z, act):
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * k * (1.0 + 3.0 * 0.044715 * z * z)
    e = 1.0 / (1.0 + torch.exp(-z))
    return e * (1.0 + z * (1.0 - e))


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        x = _norm_forward(s)[0]
        h = _normed(x, c["norm"])[0]
        if s["gain"] is not None:
            h = h * s["gain"]
        if s["scale"] is not None:
            h = h * (1.0 + s["scale"][:, None]) + s["shift"][:, None]
        dt = s["x"].dtype
        return {"x": x.to(dt), "h": h.to(dt)} if c["y"] else {"h": h.to(dt)}
    if op == "norm_bwd":
        dt = s["x"].dtype
        x, ny, ry, u, gate = _norm_forward(s)
        n, r = _normed(x, c["norm"])
        dh = s["dh"].float()
        out = {}
        p = (dh * n).sum(1)  # [B, C]
        gain = s["gain"] if s["gain"] is not None else 1.0
        if s["scale"] is not None:
            out["dscale"], out["dshift"] = gain * p, dh.sum(1)
        if s["gain"] is not None:
            out["dgain"] = (p if s["scale"] is None else p * (1.0 + s["scale"])).sum(0)
        w = dh * gain if s["scale"] is None else dh * gain * (1.0 + s["scale"][:, None])
        dx = _norm_back(w, n, r, c["norm"])
        if s["dx_out"] is not None:
            dx = dx + s["dx_out"].float()
        out["dx"] = dx.to(dt)
        if c["y"]:
            if gate is not None:
                out["dgate"] = (dx * u).sum(1)
            du = dx if gate is None else dx * gate
            if c["post"] != "none":
                out["dpost_gain"] = (du * ny).sum((0, 1))
                du = _norm_back(du * s["post_gain"], ny, ry, c["post"])
            out["dy"] = du.to(dt)
        return out
    if op in ("rope", "rope_tables"):
        a = _angles(s, s["pos"])
        cos, sin = (s["factor"] * torch.cos(a)).float(), (s["factor"] * torch.sin(a)).float()
        if op == "rope_tables":
            return cos, sin
        if c["inverse"]:
            sin = -sin
        return tuple(_rotate(v, cos, sin, c["layout"], c["rot"]).to(v.dtype) for v in (s["q"], s["k"]))
    if op == "linear":
        z = s["x"].float() @ s["w"].float().T
        if s["bias"] is not None:
            z = z + s["bias"]
        z = _act(z, c["act"])
        if s["residual"] is not None:
            z = s["residual"].float() + z
        return z.to(torch.bfloat16)
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_slope(s["z"].float(), c["act"])
    out = {"dx": (dz @ s["w"].float()).to(torch.bfloat16), "dw": (dz.T @ s["x"].float()).to(torch.bfloat16)}
    if c["bias"]:
        out["db"] = dz.sum(0)
    return out


# ---- what a pass cannot do without ----------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        B, T, C = case["B"], case["T"], case["C"]
        e = 2 if case["dtype"] == "bf16" else 4
        one = B * T * C
        vectors = B * C * ((2 if case["mod"] else 0) + (1 if case["gate"] else 0)) + \
            C * ((1 if case["gain"] else 0) + (1 if case["post"] != "none" else 0))
        if op == "norm":  # x, y in and x', h out, or x in and h out
            return {"bytes": e * one * (4 if case["y"] else 2) + 4 * vectors, "flops": 12 * one}
        # x, dh in, dx out; with a branch also y and the gradient of x' in, dy out
        return {"bytes": e * one * (6 if case["y"] else 3) + 8 * vectors, "flops": 30 * one}
    if op == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["B"] * (case["Hq"] + case["Hk"]) * case["L"]
        return {"bytes": 2 * e * n * case["d"] + 4 * case["axes"] * case["L"] + 4 * case["rot"],
                "flops": 3 * n * case["rot"]}
    if op == "rope_tables":
        return {"bytes": 4 * case["L"] * (case["rot"] + case["axes"]) + 4 * case["rot"], "flops": 20 * case["L"] * case["rot"]}
    M, K, N = case["M"], case["K"], case["N"]
    if op == "linear":
        return {"bytes": 2 * (M * K + N * K + M * N * (2 if case["residual"] else 1)) + (4 * N if case["bias"] else 0),
                "flops": 2 * M * K * N}
    return {"bytes": 2 * (2 * M * K + 2 * N * K + M * N * (1 if case["act"] == "none" else 2)) + (4 * N if case["bias"] else 0),
            "flops": 4 * M * K * N}


# ---- the definitions in 64 bits ---------------------------------------------------------------------

def _exact_norm(v, kind):
    if kind == "layer":
        var, mean = torch.var_mean(v, -1, correction=0, keepdim=True)
        return (v - mean) / torch.sqrt(var + EPS)
    return v / torch.sqrt(v.square().mean(-1, keepdim=True) + EPS)


def _exact_act(z, act):
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        v = {k: (t.double() if isinstance(t, torch.Tensor) else None) for k, t in s.items() if k != "case"}
        back = op == "norm_bwd"
        given = [k for k in ("x", "y", "gate", "gain", "scale", "shift", "post_gain") if v[k] is not None]
        for k in given:
            v[k].requires_grad_(back)
        x = v["x"]
        if v["y"] is not None:
            u = v["y"] if case["post"] == "none" else _exact_norm(v["y"], case["post"]) * v["post_gain"]
            x = x + (u if v["gate"] is None else u * v["gate"].unsqueeze(1))
        h = _exact_norm(x, case["norm"])
        if v["gain"] is not None:
            h = h * v["gain"]
        if v["scale"] is not None:
            h = torch.addcmul(v["shift"].unsqueeze(1), h, 1.0 + v["scale"].unsqueeze(1))
        if not back:
            return {"x": x, "h": h} if case["y"] else {"h": h}
        outs, grads = ([h], [v["dh"]]) if v["dx_out"] is None else ([h, x], [v["dh"], v["dx_out"]])
        return {"d" + k: g for k, g in zip(given, torch.autograd.grad(outs, [v[k] for k in given], grads))}
    if op in ("rope", "rope_tables"):
        axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=DEV),
                                       torch.tensor(s["sections"], device=DEV))
        turn = torch.polar(torch.full((), float(s["factor"]), dtype=torch.float64, device=DEV).expand(1, 1),
                           s["pos"].double()[axis].T * s["inv_freq"])
        if op == "rope_tables":
            return turn.real.contiguous(), turn.imag.contiguous()
        if case["inverse"]:
            turn = turn.conj()
        h = case["rot"] // 2
        out = []
        for x in (s["q"].double(), s["k"].double()):
            y = x.clone()
            at = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if case["layout"] == "interleaved" else \
                (slice(0, h), slice(h, 2 * h))
            z = torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous()) * turn
            y[..., at[0]], y[..., at[1]] = z.real, z.imag
            out.append(y)
        return tuple(out)
    x, w = s["x"].double(), s["w"].double()
    if op == "linear":
        z = torch.nn.functional.linear(x, w, None if s["bias"] is None else s["bias"].double())
        z = _exact_act(z, case["act"])
        return z if s["residual"] is None else z + s["residual"].double()
    dy = s["dy"].double()
    if case["act"] != "none":
        z = s["z"].double().requires_grad_(True)
        dy, = torch.autograd.grad(_exact_act(z, case["act"]), z, dy)
    out = {"dx": torch.mm(dy, w), "dw": torch.mm(dy.t(), x)}
    if case["bias"]:
        out["db"] = dy.sum(0)
    return out
