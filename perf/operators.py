"""The layer operators around the sparse attention, as a user's program calls them.

A video transformer's layer makes Q, K, V from its activations (a projection that writes
[heads][N][D]), norms Q and K per head and rotates them by their grid position, runs the
sparse attention, and takes O back (a projection that reads [heads][N][D], adds the residual).
Four operators: the per-head norm with the rotation and its gradients, the projection with
bias, activation and residual in its epilogue and its gradients.

`run` computes them with elementary torch operations in 32 bits, or (`own`) with the
framework's calls.  `exact` computes them in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(name, op, T, H, W, heads, D, dtype, layout, pairing, dims, **more):
    return {"name": name, "op": op, "T": T, "H": H, "W": W, "heads": heads, "D": D, "dtype": dtype, "layout": layout,
            "pairing": pairing, "dt": dims[0], "dh": dims[1], "dw": dims[2], **more}


def _linear(name, op, M, K, N, in_heads=0, out_heads=0, act="none", bias=True, residual=False, out="bf16", **more):
    return {"name": name, "op": op, "M": M, "K": K, "N": N, "in_heads": in_heads, "out_heads": out_heads, "act": act,
            "bias": bias, "residual": residual, "out": out, **more}


def listed():
    return [
        # Q and K of one sequence-parallel rank's 5 of 40 heads at the 2K grid, from a fused projection
        _norm("norm_rope_72x88x160_5heads", "norm_rope", 72, 88, 160, 5, 128, "bf16", "fused", "adjacent", (44, 42, 42)),
        # every head of a 92,160-token layer, from a projection that wrote head-major
        _norm("norm_rope_24x48x80", "norm_rope", 24, 48, 80, 40, 128, "bf16", "heads", "halves", (44, 42, 42)),
        # a second branch's 1,001 audio tokens on a 1-D axis
        _norm("norm_rope_audio_1001", "norm_rope", 1001, 1, 1, 40, 64, "bf16", "fused", "halves", (64, 0, 0)),
        # the gradients of that layer: fp32 dQ, dK from the attention's backward
        _norm("norm_rope_grad_24x48x80", "norm_rope_grad", 24, 48, 80, 40, 128, "bf16", "fused", "adjacent",
              (44, 42, 42), grad="f32"),
        # the smallest grid, fp32 throughout, half of each head rotated
        _norm("norm_rope_grad_8x16x16", "norm_rope_grad", 8, 16, 16, 2, 64, "f32", "heads", "halves", (16, 8, 8),
              grad="f32"),
        # Q, K and V of 92,160 tokens in one product, written head-major for the plan
        _linear("qkv_92160", "linear", 92160, 5120, 15360, out_heads=120),
        # the attention's O back to the residual stream, read head-major
        _linear("out_residual_92160", "linear", 92160, 5120, 5120, in_heads=40, residual=True, out="f32"),
        # the first feed-forward product of a ragged clip, its pre-activation kept for the backward
        _linear("ffn_gelu_9973", "linear", 9973, 5120, 20480, act="gelu_tanh", pre=True),
        # the modulation of a layer from one time embedding: a single token against all the weights
        _linear("modulation_1", "linear", 1, 5120, 30720, act="none", out="f32"),
        # a few tokens of a short prompt
        _linear("few_tokens_13", "linear", 13, 5120, 5120, act="silu", residual=True),
        # the gradients of the output projection: dO written head-major for the attention's backward
        _linear("out_grad_92160", "linear_grad", 92160, 5120, 5120, in_heads=40, out="bf16", dw="f32"),
        # the gradients of a feed-forward product through its activation, ragged rows
        _linear("ffn_gelu_grad_2477", "linear_grad", 2477, 5120, 20480, act="gelu_tanh", dw="bf16"),
    ]


def _log(rng, a, b):
    return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "linear", "linear", "linear_grad", "linear_grad"])
    if op.startswith("norm"):
        D = rng.choice([64, 128])
        if rng.random() < 0.3:
            T, H, W = _log(rng, 1, 20000), 1, 1
            dims = (D, 0, 0)
        else:
            T, H, W = _log(rng, 1, 72), _log(rng, 1, 88), _log(rng, 1, 160)
            dims = rng.choice([(44, 42, 42), (32, 48, 48), (16, 24, 24)] if D == 128 else [(24, 20, 20), (16, 24, 24), (16, 8, 8)])
        heads = max(1, min(_log(rng, 1, 48), 471_859_200 // (T * H * W * D)))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        case = _norm("", op, T, H, W, heads, D, dtype, rng.choice(["fused", "heads"]), rng.choice(["adjacent", "halves"]), dims)
        if op == "norm_rope_grad":
            case["grad"] = rng.choice(["bf16", "f32"])
    else:
        M = _log(rng, 1, 100) if rng.random() < 0.35 else _log(rng, 100, 92160)
        in_heads = rng.choice([0, 0, _log(rng, 1, 40)])
        K = in_heads * rng.choice([64, 128]) if in_heads else _log(rng, 64, 8192)
        out_heads = rng.choice([0, 0, _log(rng, 1, 120)])
        N = out_heads * rng.choice([64, 128]) if out_heads else _log(rng, 64, 20480)
        while M * K * N > 92160 * 5120 * 5120:
            M = M * 2 // 3
        case = _linear("", op, M, K, N, in_heads, out_heads, rng.choice(["none", "gelu", "gelu_tanh", "silu"]), rng.random() < 0.7,
                       op == "linear" and rng.random() < 0.5, rng.choice(["bf16", "f32"]) if op == "linear" else "bf16")
        if op == "linear":
            case["pre"] = case["act"] != "none" and rng.random() < 0.5
        else:
            # through an activation dz is rounded to the operands' 16 bits: the weights' gradient keeps no more
            case["dw"] = rng.choice(["bf16", "f32"]) if case["act"] == "none" else "bf16"
    del case["name"]
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    return out.normal_(0.0, scale, generator=g)


def _angles(c):
    """Rotation angles [N, pairs] in 64 bits: pair p of an axis with d channels turns by position / THETA^(2p/d)."""
    pos = torch.arange(c["T"] * c["H"] * c["W"], device="cuda")
    out = []
    for axis, d in ((pos // (c["H"] * c["W"]), c["dt"]), (pos // c["W"] % c["H"], c["dh"]), (pos % c["W"], c["dw"])):
        f = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / max(d, 1))
        out.append(axis.double()[:, None] * f)
    return torch.cat(out, 1)


def _pairs(c):
    """The two channels of every pair, in the order of _angles' columns."""
    a, b, base = [], [], 0
    for d in (c["dt"], c["dh"], c["dw"]):
        for p in range(d // 2):
            a.append(base + (2 * p if c["pairing"] == "adjacent" else p))
            b.append(base + (2 * p + 1 if c["pairing"] == "adjacent" else p + d // 2))
        base += d
    return torch.tensor(a, device="cuda"), torch.tensor(b, device="cuda")


def _norm_inputs(c, seed):
    g, N, dt = _gen(seed), c["T"] * c["H"] * c["W"], DTYPES[c["dtype"]]
    s = {}
    if c["layout"] == "fused":
        qkv = _randn(g, (N, 3, c["heads"], c["D"]), dt)
        s["q"], s["k"] = qkv[:, 0].transpose(0, 1), qkv[:, 1].transpose(0, 1)
    else:
        s["q"], s["k"] = (_randn(g, (c["heads"], N, c["D"]), dt) for _ in range(2))
    s["wq"], s["wk"] = (1 + _randn(g, (c["D"],), torch.float32, 0.2) for _ in range(2))
    if c["op"] == "norm_rope_grad":
        s["dq"], s["dk"] = (_randn(g, (c["heads"], N, c["D"]), DTYPES[c["grad"]]) for _ in range(2))
    return s


def _linear_inputs(c, seed):
    g, M, K, N = _gen(seed), c["M"], c["K"], c["N"]
    s = {"x": _randn(g, (c["in_heads"], M, K // c["in_heads"]) if c["in_heads"] else (M, K), torch.bfloat16),
         "W": _randn(g, (N, K), torch.bfloat16, K ** -0.5),
         "b": _randn(g, (N,), torch.float32, 0.1) if c["bias"] else None}
    shape = (c["out_heads"], M, N // c["out_heads"]) if c["out_heads"] else (M, N)
    if c["op"] == "linear":
        s["r"] = _randn(g, shape, DTYPES[c["out"]]) if c["residual"] else None
    else:
        s["dy"] = _randn(g, shape, DTYPES[c["out"]])
        s["pre"] = _randn(g, shape, torch.bfloat16) if c["act"] != "none" else None
    return s


def prepare(case, seed):
    c = dict(case)
    if c["op"].startswith("norm"):
        s = _norm_inputs(c, seed)
        if own:
            from dynamic_block_sparse_indicator_b200 import _lib
            pairing = _lib.PRISM_PAIR_ADJACENT if c["pairing"] == "adjacent" else _lib.PRISM_PAIR_HALVES
            s["rope"] = _lib.make_rope(c["T"], c["H"], c["W"], (c["dt"], c["dh"], c["dw"]), theta=THETA, pairing=pairing)
        else:
            ang = _angles(c)
            s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
            s["a"], s["b"] = _pairs(c)
    else:
        s = _linear_inputs(c, seed)
        if own:
            from dynamic_block_sparse_indicator_b200 import _lib
            s["act"] = {"none": _lib.PRISM_ACT_NONE, "gelu": _lib.PRISM_ACT_GELU, "gelu_tanh": _lib.PRISM_ACT_GELU_TANH,
                        "silu": _lib.PRISM_ACT_SILU}[c["act"]]
            s["status"] = torch.zeros(4, dtype=torch.int32, device="cuda")
    s["case"] = c
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(u, cos, sin, a, b):
    out = u.clone()
    ua, ub = u[..., a], u[..., b]
    out[..., a] = ua * cos - ub * sin
    out[..., b] = ua * sin + ub * cos
    return out


def _plain_norm_rope(x, w, s):
    x32 = x.float()
    u = x32 * torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS) * w
    return _rotate(u, s["cos"], s["sin"], s["a"], s["b"]).to(x.dtype)


def _plain_norm_rope_grad(gy, x, w, s):
    x32 = x.float()
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    n = x32 * r
    v = _rotate(gy.float(), s["cos"], -s["sin"], s["a"], s["b"])
    dw = (v * n).sum((0, 1))
    v = v * w
    return (r * (v - n * (v * n).mean(-1, keepdim=True))).to(x.dtype), dw


def _tokens(x):
    """[heads, M, D] as [M, heads D]; [M, K] as it is."""
    return x.transpose(0, 1).reshape(x.shape[1], -1) if x.dim() == 3 else x


def _heads(y, heads):
    return y.reshape(y.shape[0], heads, -1).transpose(0, 1).contiguous() if heads else y


def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    sg = 1 / (1 + torch.exp(-z))
    return sg * (1 + z * (1 - sg))


def _plain_linear(c, s):
    z = _tokens(s["x"].float()) @ s["W"].float().t()
    if c["bias"]:
        z = z + s["b"]
    y = _heads(_act(z, c["act"]), c["out_heads"])
    if c["residual"]:
        y = y + s["r"].float()
    y = y.to(DTYPES[c["out"]])
    return {"y": y, "pre": _heads(z, c["out_heads"]).to(torch.bfloat16)} if c.get("pre") else {"y": y}


def _plain_linear_grad(c, s):
    dz = _tokens(s["dy"].float())
    if c["act"] != "none":
        dz = dz * _act_grad(_tokens(s["pre"].float()), c["act"])
    out = {"dx": _heads(dz @ s["W"].float(), c["in_heads"]).to(torch.bfloat16),
           "dW": (dz.t() @ _tokens(s["x"].float())).to(DTYPES[c["dw"]])}
    if c["bias"]:
        out["db"] = dz.sum(0)
    return out


def run(s):
    c = s["case"]
    if own:
        from dynamic_block_sparse_indicator_b200 import _lib
        if c["op"] == "norm_rope":
            q, k = _lib.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["rope"], eps=EPS)
            return {"q": q, "k": k}
        if c["op"] == "norm_rope_grad":
            dq, dk, dwq, dwk = _lib.qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["rope"], eps=EPS)
            return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
        if c["op"] == "linear":
            y, pre, _ = _lib.linear(s["x"], s["W"], s["b"], s["r"], activation=s["act"], out_dtype=DTYPES[c["out"]],
                                    out_heads=c["out_heads"], want_pre=bool(c.get("pre")), status=s["status"])
            return {"y": y, "pre": pre} if c.get("pre") else {"y": y}
        dx, dW, db, _ = _lib.linear_bwd(s["dy"], s["x"], s["W"], s["pre"], activation=s["act"], dw_dtype=DTYPES[c["dw"]],
                                        want_db=c["bias"], status=s["status"])
        return {"dx": dx, "dW": dW, "db": db} if c["bias"] else {"dx": dx, "dW": dW}
    if c["op"] == "norm_rope":
        return {"q": _plain_norm_rope(s["q"], s["wq"], s), "k": _plain_norm_rope(s["k"], s["wk"], s)}
    if c["op"] == "norm_rope_grad":
        dq, dwq = _plain_norm_rope_grad(s["dq"], s["q"], s["wq"], s)
        dk, dwk = _plain_norm_rope_grad(s["dk"], s["k"], s["wk"], s)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    return _plain_linear(c, s) if c["op"] == "linear" else _plain_linear_grad(c, s)


def work(case):
    c = case
    if c["op"].startswith("norm"):
        e = 2 * c["T"] * c["H"] * c["W"] * c["heads"] * c["D"]
        size = 2 if c["dtype"] == "bf16" else 4
        weights = 2 * 4 * c["D"]
        if c["op"] == "norm_rope":
            return {"bytes": 2 * e * size + weights, "flops": 8 * e}
        return {"bytes": e * (2 * size + (2 if c["grad"] == "bf16" else 4)) + 2 * weights, "flops": 16 * e}
    M, K, N = c["M"], c["K"], c["N"]
    out = 2 if c["out"] == "bf16" else 4
    if c["op"] == "linear":
        more = (out * M * N if c["residual"] else 0) + (2 * M * N if c.get("pre") else 0) + (4 * N if c["bias"] else 0)
        return {"bytes": 2 * (M * K + N * K) + out * M * N + more, "flops": 2 * M * K * N}
    more = (2 * M * N if c["act"] != "none" else 0) + (4 * N if c["bias"] else 0)
    return {"bytes": out * M * N + 2 * (M * K + N * K) + 2 * M * K + (2 if c["dw"] == "bf16" else 4) * N * K + more,
            "flops": 4 * M * K * N}


# ------------------------------------------------------------------ 64 bits
def _exact_norm_rope(c, x, w):
    """Every head by itself; the rotation as a product of complex numbers."""
    a, b = _pairs(c)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), _angles(c))
    rows = []
    for h in range(x.shape[0]):
        u = x[h].double()
        u = u / ((u ** 2).sum(1, keepdim=True) / c["D"] + EPS).sqrt() * w.double()
        z = torch.complex(u[:, a], u[:, b]) * turn
        u = u.index_copy(1, a, z.real).index_copy(1, b, z.imag)
        rows.append(u)
    return torch.stack(rows)


def _exact_act(z, act):
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * torch.sigmoid(z) if act == "silu" else z


def exact(case, seed):
    c = case
    if c["op"] == "norm_rope":
        s = _norm_inputs(c, seed)
        return {"q": _exact_norm_rope(c, s["q"], s["wq"]), "k": _exact_norm_rope(c, s["k"], s["wk"])}
    if c["op"] == "norm_rope_grad":
        s, out = _norm_inputs(c, seed), {}
        for n in "qk":
            dx, dw = [], torch.zeros(c["D"], dtype=torch.float64, device="cuda")
            for h in range(c["heads"]):  # one head at a time: the graph of all would not fit
                x = s[n][h:h + 1].double().requires_grad_()
                w = s["w" + n].double().requires_grad_()
                y = _exact_norm_rope(c, x, w)
                gx, gw = torch.autograd.grad(y, (x, w), s["d" + n][h:h + 1].double())
                dx.append(gx[0])
                dw += gw
            out["d" + n], out["dw" + n] = torch.stack(dx), dw
        return out
    s = _linear_inputs(c, seed)
    D, E = (c["K"] // c["in_heads"] if c["in_heads"] else 0), (c["N"] // c["out_heads"] if c["out_heads"] else 0)
    W = s["W"].double()
    x = s["x"].double()
    if c["op"] == "linear":
        z = torch.einsum("hmd,nhd->mn", x, W.reshape(c["N"], c["in_heads"], D)) if D else torch.einsum("mk,nk->mn", x, W)
        if c["bias"]:
            z += s["b"].double()
        if E:
            z = torch.stack([z[:, E * h:E * h + E] for h in range(c["out_heads"])])
        y = _exact_act(z, c["act"])
        if c["residual"]:
            y = y + s["r"].double()
        return {"y": y, "pre": z} if c.get("pre") else {"y": y}
    dz = s["dy"].double()
    if c["act"] != "none":
        z = s["pre"].double().requires_grad_()
        dz, = torch.autograd.grad(_exact_act(z, c["act"]), z, dz)
    if E:
        dz = torch.cat([dz[h] for h in range(c["out_heads"])], 1)
    if D:
        out = {"dx": torch.einsum("mn,nhd->hmd", dz, W.reshape(c["N"], c["in_heads"], D)),
               "dW": torch.einsum("mn,hmd->nhd", dz, x).reshape(c["N"], c["K"])}
    else:
        out = {"dx": torch.einsum("mn,nk->mk", dz, W), "dW": torch.einsum("mn,mk->nk", dz, x)}
    if c["bias"]:
        out["db"] = dz.sum(0)
    return out
