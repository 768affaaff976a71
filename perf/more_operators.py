"""What the dense feed-forward block's operators are measured on, and their plain forms.

The five operators of the training step of a dense feed-forward block: layer
norm (forward, backward with the sums for its weight and bias), the gated
projections H = act(X Wg^T) * (X Wu^T) as one product (forward, backward down to
the gradients of both projections), and the orthogonalised update of a weight
from its gradient by Newton-Schulz products.

``own`` False: elementary torch operations in 32 bits.  ``own`` True: the
library's entry points.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# (hidden, ffn) of the layer sets in workloads.py
BLOCKS = ((576, 1536), (2304, 5760))
# (rows, cols) of their weights
WEIGHTS = ((576, 576), (192, 576), (1536, 576), (576, 1536), (2304, 2304), (5760, 2304), (2304, 5760))
LN_EPS = 1e-5
ORTH_EPS = 1e-7
# the quintic of the update: x -> a x + b x^3 + c x^5 on every singular value
QUINTIC = (3.4445, -4.7750, 2.0315)


def _norm(name, op, T, d, dtype="bf16", out="bf16", bias=True, res=False):
    """bias: the norm has one; out (backward): type of the weight's and the bias's gradients; res (backward): the
    residual stream's gradient is added to the input's."""
    return {"name": name, "op": op, "T": T, "d": d, "dtype": dtype, "out": out, "bias": bias, "res": res}


def _gated(name, op, T, d, f, act="silu", dtype="bf16", keep=True):
    """keep: forward, both projections are stored beside their product (training); backward, the product is computed
    again beside the gradients (for the down projection's weight gradient)."""
    return {"name": name, "op": op, "T": T, "d": d, "f": f, "act": act, "dtype": dtype, "keep": keep}


def _orth(name, batch, rows, cols, dtype="bf16", out="bf16", steps=5, rank=16, scale=1.0):
    """`batch` gradients [rows, cols], each of a strong part of this rank beside noise."""
    return {"name": name, "op": "orth", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype, "out": out,
            "steps": steps, "rank": rank, "scale": scale}


def listed():
    return [
        # a few rows of the 135M-class hidden size: a short prompt's tail, latency
        _norm("ln_fwd_few_rows", "ln_fwd", 8, 576, dtype="f16"),
        # a 16K-token micro-batch of the 2B-class hidden size
        _norm("ln_fwd_16k", "ln_fwd", 16384, 2304),
        # the same block's backward at 8K tokens, with the residual stream's gradient, FP32 sums for the weights
        _norm("ln_bwd_8k", "ln_bwd", 8192, 2304, out="f32", res=True),
        # an FP32 norm of an odd micro-batch of the 135M-class size, no bias
        _norm("ln_bwd_2k_f32", "ln_bwd", 2047, 576, dtype="f32", out="f32", bias=False),
        # one token through the 2B-class block: the two weights are read, nothing is kept
        _gated("gated_fwd_1_token", "gated_fwd", 1, 2304, 5760, keep=False),
        # a training micro-batch of the 2B-class block
        _gated("gated_fwd_4k", "gated_fwd", 4096, 2304, 5760),
        # an odd micro-batch of the 135M-class block, GELU, fp16
        _gated("gated_fwd_1k_gelu", "gated_fwd", 1001, 576, 1536, act="gelu", dtype="f16"),
        # their backward passes
        _gated("gated_bwd_4k", "gated_bwd", 4096, 2304, 5760),
        _gated("gated_bwd_1k_gelu", "gated_bwd", 1001, 576, 1536, act="gelu", dtype="f16"),
        # the key projection of one 135M-class layer: latency
        _orth("orth_1_small", 1, 192, 576),
        # the query and output projections of twelve 135M-class layers, FP32 momentum
        _orth("orth_24_square", 24, 576, 576, dtype="f32"),
        # the gate and up projections of two 2B-class layers
        _orth("orth_4_tall", 4, 5760, 2304, scale=0.3),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("ln_fwd", "ln_bwd", "gated_fwd", "gated_bwd", "orth"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op in ("ln_fwd", "ln_bwd"):
        d = rng.choice((576, 2304, 5760, _log(rng, 64, 8192), _log(rng, 64, 8192)))
        T = min(_log(rng, 1, 16384), 16384 * 2304 // d)
        dtype = rng.choice((dtype, dtype, "f32"))
        c = _norm("", op, T, d, dtype, rng.choice((dtype, "f32")), rng.random() < 0.7, op == "ln_bwd" and rng.random() < 0.5)
    elif op in ("gated_fwd", "gated_bwd"):
        d, f = rng.choice(BLOCKS) if rng.random() < 0.6 else (_log(rng, 64, 4096), _log(rng, 64, 6144))
        T = max(1, min(_log(rng, 1, 4096), 4096 * 2304 * 5760 // (d * f)))
        c = _gated("", op, T, d, f, rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu")), dtype, rng.random() < 0.7)
    else:
        rows, cols = rng.choice(WEIGHTS) if rng.random() < 0.6 else (_log(rng, 16, 3000), _log(rng, 16, 3000))
        cost = rows * cols * min(rows, cols)
        batch = max(1, min(_log(rng, 1, 32), 4 * 5760 * 2304 * 2304 // cost))
        out = rng.choice(("bf16", "bf16", "f16"))
        c = _orth("", batch, rows, cols, rng.choice((dtype, "f32")), out, rng.choice((5, 5, 5, 3, 6)),
                  rng.choice((4, 16, 64)), rng.choice((1.0, 0.2)))
    del c["name"]
    return c


def _randn(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def prepare(case, seed):
    """Values as in inputs.py: activations N(0, 1), weights N(0, 0.02), output gradients N(0, 0.01)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)
    op, dt = case["op"], TYPES[case["dtype"]]
    s = {"op": op}
    if op == "orth":
        b, rows, cols, r = case["batch"], case["rows"], case["cols"], case["rank"]
        left = torch.randn((b, rows, r), generator=g, device="cuda") * 0.8 ** torch.arange(r, device="cuda")
        G = left @ torch.randn((b, r, cols), generator=g, device="cuda")
        s["G"] = (0.01 * G + torch.randn((b, rows, cols), generator=g, device="cuda") * 0.003).to(dt)
        s["O"] = torch.empty((b, rows, cols), dtype=TYPES[case["out"]], device="cuda")
        s["steps"], s["scale"] = case["steps"], case["scale"]
        return s
    T, d = case["T"], case["d"]
    if op in ("ln_fwd", "ln_bwd"):
        # channels of different means and sizes, a few of them far out
        size = torch.exp(0.5 * torch.randn(d, generator=g, device="cuda"))
        X = torch.randn((T, d), generator=g, device="cuda").mul_(size).add_(0.5 * torch.randn(d, generator=g, device="cuda"))
        s["X"] = X.to(dt)
        s["w"] = (1 + _randn(g, (d,), 0.1, torch.float32)).to(dt)
        s["b"] = _randn(g, (d,), 0.1, dt) if case["bias"] else None
        stats = {k: torch.empty(T, device="cuda") for k in ("mean", "rstd")}
        if op == "ln_fwd":
            s["outs"] = {"Y": torch.empty_like(s["X"]), **stats}
            return s
        wide = s["X"].double()
        s["mean"] = stats["mean"].copy_(wide.mean(1))
        s["rstd"] = stats["rstd"].copy_(torch.rsqrt((wide - wide.mean(1, keepdim=True)).square().mean(1) + LN_EPS))
        s["dY"] = _randn(g, (T, d), 0.01, dt)
        s["dR"] = _randn(g, (T, d), 0.01, dt) if case["res"] else None
        wt = TYPES[case["out"]]
        s["outs"] = {"dX": torch.empty_like(s["X"]), "dw": torch.empty(d, dtype=wt, device="cuda")}
        if case["bias"]:
            s["outs"]["db"] = torch.empty(d, dtype=wt, device="cuda")
        return s
    f = case["f"]
    s["act"] = case["act"]
    if op == "gated_fwd":
        s["X"], s["W"] = _randn(g, (T, d), 1.0, dt), _randn(g, (2 * f, d), 0.02, dt)  # gate rows, then up rows
        s["outs"] = {"H": torch.empty((T, f), dtype=dt, device="cuda")}
        if case["keep"]:
            s["outs"]["GU"] = torch.empty((T, 2 * f), dtype=dt, device="cuda")
    else:
        s["dY"], s["W"] = _randn(g, (T, d), 0.01, dt), _randn(g, (d, f), 0.02, dt)  # the down projection
        s["GU"] = _randn(g, (T, 2 * f), 0.02 * math.sqrt(d), dt)
        s["outs"] = {"dGU": torch.empty((T, 2 * f), dtype=dt, device="cuda")}
        if case["keep"]:
            s["outs"]["H"] = torch.empty((T, f), dtype=dt, device="cuda")
    return s


def _act(kind, x):
    """The activation and its derivative."""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-x))
        return x * p, p * (1 + x * (1 - p))
    if kind == "gelu":
        p = 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
        return x * p, p + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    if kind == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (x + 0.044715 * x * x * x))
        return 0.5 * x * (1 + t), 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * k * (1 + 3 * 0.044715 * x * x)
    return torch.clamp(x, min=0), (x > 0).float()


def _plain(s):
    op, o = s["op"], s.get("outs")
    if op == "orth":
        X = s["G"].float()
        X = X / (X.square().sum((1, 2), keepdim=True).sqrt() + ORTH_EPS)
        tall = X.shape[1] > X.shape[2]
        if tall:
            X = X.transpose(1, 2)
        a, b, c = QUINTIC
        for _ in range(s["steps"]):
            A = torch.bmm(X, X.transpose(1, 2))
            X = a * X + torch.bmm(b * A + c * torch.bmm(A, A), X)
        return s["O"].copy_(s["scale"] * (X.transpose(1, 2) if tall else X))
    if op == "ln_fwd":
        X = s["X"].float()
        mean = X.mean(1)
        dev = X - mean[:, None]
        rstd = torch.rsqrt(dev.square().mean(1) + LN_EPS)
        Y = dev * rstd[:, None] * s["w"].float()
        if s["b"] is not None:
            Y = Y + s["b"].float()
        return {"Y": o["Y"].copy_(Y), "mean": o["mean"].copy_(mean), "rstd": o["rstd"].copy_(rstd)}
    if op == "ln_bwd":
        dY, rstd = s["dY"].float(), s["rstd"][:, None]
        n = (s["X"].float() - s["mean"][:, None]) * rstd
        q = dY * s["w"].float()
        dX = rstd * (q - q.mean(1, keepdim=True) - n * (q * n).mean(1, keepdim=True))
        if s["dR"] is not None:
            dX = dX + s["dR"].float()
        r = {"dX": o["dX"].copy_(dX), "dw": o["dw"].copy_((dY * n).sum(0))}
        if s["b"] is not None:
            r["db"] = o["db"].copy_(dY.sum(0))
        return r
    if op == "gated_fwd":
        P = s["X"].float() @ s["W"].float().t()
        f = P.shape[1] // 2
        r = {"H": o["H"].copy_(_act(s["act"], P[:, :f])[0] * P[:, f:])}
        if "GU" in o:
            r["GU"] = o["GU"].copy_(P)
        return r
    dH = s["dY"].float() @ s["W"].float()
    f = dH.shape[1]
    G, U = s["GU"][:, :f].float(), s["GU"][:, f:].float()
    A, dA = _act(s["act"], G)
    r = {"dGU": o["dGU"].copy_(torch.cat((dH * U * dA, dH * A), 1))}
    if "H" in o:
        r["H"] = o["H"].copy_(A * U)
    return r


def run(state):
    if not own:
        return _plain(state)
    import gemms_linear_layers_gb300 as tg
    s, op = state, state["op"]
    if op == "orth":
        return tg.tg_orthogonalize(s["G"], O=s["O"], steps=s["steps"], coeffs=QUINTIC, scale=s["scale"], eps=ORTH_EPS)
    if op == "ln_fwd":
        return tg.tg_layer_norm_fwd(s["X"], s["w"], b=s["b"], eps=LN_EPS, outs=s["outs"])
    if op == "ln_bwd":
        return tg.tg_layer_norm_bwd(s["dY"], s["X"], s["w"], s["mean"], s["rstd"], dR=s["dR"], bias=s["b"] is not None,
                                    outs=s["outs"])
    if op == "gated_fwd":
        return tg.tg_gated_fwd(s["X"], s["W"], act=s["act"], keep="GU" in s["outs"], outs=s["outs"])
    return tg.tg_gated_bwd(s["dY"], s["W"], s["GU"], act=s["act"], keep="H" in s["outs"], outs=s["outs"])


_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def work(case):
    op, e = case["op"], _BYTES[case["dtype"]]
    if op == "orth":
        b, n = case["batch"], case["rows"] * case["cols"]
        m, k = min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # A = X X^T and A A are symmetric: half of each
        flops = case["steps"] * (m * (m + 1) * k + m * (m + 1) * m + 2 * m * m * k)
        return {"bytes": b * n * (e + _BYTES[case["out"]]), "flops": b * flops}
    T, d = case["T"], case["d"]
    if op == "ln_fwd":
        return {"bytes": 2 * T * d * e + (2 if case["bias"] else 1) * d * e + 8 * T, "flops": 8 * T * d}
    if op == "ln_bwd":
        sums = (2 if case["bias"] else 1) * d * _BYTES[case["out"]]
        return {"bytes": (4 if case["res"] else 3) * T * d * e + d * e + sums + 8 * T, "flops": 14 * T * d}
    f = case["f"]
    if op == "gated_fwd":
        return {"bytes": e * (T * d + 2 * f * d + (3 if case["keep"] else 1) * T * f), "flops": 4 * T * d * f + 8 * T * f}
    return {"bytes": e * (T * d + f * d + (5 if case["keep"] else 4) * T * f), "flops": 2 * T * d * f + 16 * T * f}


def exact(case, seed):
    """The definitions in 64 bits: gradients through autograd, the update through the matrices' own polynomial."""
    s = prepare(case, seed)
    op = s["op"]
    up = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "orth":
        outs = []
        a, b, c = QUINTIC
        for G in up["G"]:
            X = G / (torch.linalg.vector_norm(G) + ORTH_EPS)
            eye = torch.eye(min(G.shape), dtype=torch.float64, device="cuda")
            for _ in range(case["steps"]):
                A = X.T @ X if G.shape[0] > G.shape[1] else X @ X.T
                Q = torch.addmm(a * eye + b * A, A, A, alpha=c)
                X = X @ Q if G.shape[0] > G.shape[1] else Q @ X
            outs.append(X * case["scale"])
        return torch.stack(outs)
    if op == "ln_fwd":
        var, mean = torch.var_mean(up["X"], 1, correction=0)
        rstd = (var + LN_EPS) ** -0.5
        Y = torch.einsum("td,t,d->td", up["X"] - mean[:, None], rstd, up["w"])
        return {"Y": Y + up["b"] if "b" in up else Y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        # dX = rstd (I - 1 1^T / d - n n^T / d) (w dY)
        xc = up["X"] - up["mean"][:, None]
        q = up["dY"] * up["w"]
        along = (q * xc).sum(1) * up["rstd"] ** 2 / case["d"]
        dX = (q - (q.sum(1) / case["d"])[:, None] - xc * along[:, None]) * up["rstd"][:, None]
        r = {"dX": dX + up["dR"] if "dR" in up else dX, "dw": torch.einsum("td,td,t->d", up["dY"], xc, up["rstd"])}
        if case["bias"]:
            r["db"] = up["dY"].sum(0)
        return r
    F = torch.nn.functional
    act = {"silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda x: F.gelu(x, approximate="tanh"), "relu": F.relu}[case["act"]]
    f = case["f"]
    if op == "gated_fwd":
        G, U = (torch.einsum("td,fd->tf", up["X"], w) for w in up["W"].split(f))
        r = {"H": act(G) * U}
        if case["keep"]:
            r["GU"] = torch.cat((G, U), 1)
        return r
    GU = up["GU"].requires_grad_()
    H = act(GU[:, :f]) * GU[:, f:]
    (dGU,) = torch.autograd.grad(H, GU, torch.einsum("td,df->tf", up["dY"], up["W"]))
    return {"dGU": dGU, "H": H.detach()} if case["keep"] else {"dGU": dGU}
