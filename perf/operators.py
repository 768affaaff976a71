"""What the expert-block operators are measured on, and their plain forms.

The six operators of the training step of an expert block: the three products
of a linear layer whose rows are grouped by expert (forward, input gradient,
weight gradient), the norms after and before a block with its gate and
residual scale (forward, backward), and the clipping of many gradient tensors
by their global norm.

``own`` False: elementary torch operations in 32 bits.  ``own`` True: the
library's entry points.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# (d_in, d_out) of the layer sets in workloads.py: hidden 576 (135M-class) and hidden 2,304 (2B-class)
LAYERS = ((576, 192), (576, 576), (576, 1536), (1536, 576), (2304, 2304), (2304, 5760), (5760, 2304))
EPS = 1e-6


def _group(name, op, T, E, d_in, d_out, zipf=0.5, empty=0.0, spare=0, dtype="bf16", out="bf16", route=1):
    """One product over E experts. Expert shares fall as rank^-zipf; a share `empty` of the experts has no
    rows; the last `spare` of the T rows belong to no expert (a buffer of fixed size that is not full)."""
    return {"name": name, "op": op, "T": T, "E": E, "d_in": d_in, "d_out": d_out, "zipf": zipf, "empty": empty,
            "spare": spare, "dtype": dtype, "out": out, "route": route}


def _norm(name, op, T, d, gate, dtype="bf16", res="bf16", out="bf16", scale=1.0):
    """gate: none, channel [d], token [T, 1] or full [T, d]; res: type of the residual stream; out (backward):
    type of the weights' and the broadcast gate's gradients."""
    return {"name": name, "op": op, "T": T, "d": d, "gate": gate, "dtype": dtype, "res": res, "out": out, "scale": scale}


def _clip(name, hidden, ffn, layers, rank, dtype, kind, max_norm):
    """Gradients of `layers` decoder layers: the seven projections, or (rank > 0) their rank-r LoRA factors.
    kind "same": every tensor of `dtype`; "mixed": every third tensor FP32 (norms and biases kept in FP32)."""
    return {"name": name, "op": "clip", "hidden": hidden, "ffn": ffn, "layers": layers, "rank": rank, "dtype": dtype,
            "kind": kind, "max_norm": max_norm}


def listed():
    return [
        # a few rows through small experts: launch latency and the experts' weights
        _group("fwd_few_rows", "fwd", 48, 8, 576, 1536, zipf=1.0, empty=0.25),
        # a 16K-token micro-batch over 64 experts of the 2B-class up projection: the largest product
        _group("fwd_16k_64_experts", "fwd", 16384, 64, 2304, 5760, spare=101),
        # the gradient for the up projection's input at 4,096 tokens, uneven groups
        _group("dgrad_4k_8_experts", "dgrad", 4096, 8, 2304, 5760, zipf=1.0, dtype="f16", out="f16", route=3),
        # the 135M-class down projection over many small experts (about 30 rows each)
        _group("dgrad_1k_32_experts", "dgrad", 1000, 32, 1536, 576, empty=0.1, route=4),
        # weight gradients of the 2B-class down projection, 8 experts
        _group("wgrad_4k_8_experts", "wgrad", 4096, 8, 5760, 2304, zipf=1.0, route=5),
        # weight gradients in FP32 for many experts with few rows each: bound by writing them
        _group("wgrad_2k_64_experts", "wgrad", 2047, 64, 576, 1536, empty=0.1, out="f32", route=6),
        # the smallest step: a handful of rows of the 135M-class hidden size
        _norm("norm_fwd_few_rows", "norm_fwd", 8, 576, "none"),
        # a large micro-batch of the 2B-class hidden size, element-wise gate
        _norm("norm_fwd_16k", "norm_fwd", 16384, 2304, "full", scale=0.5),
        # router probability as the gate of each token, 2B-class, FP32 residual stream
        _norm("norm_bwd_8k", "norm_bwd", 8192, 2304, "token", res="f32"),
        # 135M-class hidden size, learned gate for each channel, FP32 gradients of the weights
        _norm("norm_bwd_2k", "norm_bwd", 2048, 576, "channel", dtype="f16", res="f16", out="f32", scale=0.7),
        # LoRA factors' gradients of four 135M-class layers: many small tensors
        _clip("clip_lora", 576, 1536, 4, 16, "f32", "same", 1.0),
        # the projections' gradients of eight 2B-class layers
        _clip("clip_2b", 2304, 5760, 8, 0, "bf16", "mixed", 1.0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("fwd", "dgrad", "wgrad", "norm_fwd", "norm_bwd", "clip"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    if op == "clip":
        rank = rng.choice((0, 0, 16))
        hidden, ffn = rng.choice(((576, 1536), (2304, 5760), (_log(rng, 64, 2304), _log(rng, 64, 5760))))
        layers = rng.randint(1, 8 if rank == 0 else 4)
        c = _clip("", hidden, ffn, layers, rank, rng.choice(("bf16", "f16", "f32")) if rank or hidden < 2304 else dtype,
                  rng.choice(("same", "mixed")), rng.choice((0.5, 1.0, 1e6)))
    elif op in ("norm_fwd", "norm_bwd"):
        T = _log(rng, 1, 16384)
        d = rng.choice((576, 2304, 5760, _log(rng, 64, 8192), _log(rng, 64, 8192)))
        T = min(T, 16384 * 2304 // d)
        c = _norm("", op, T, d, rng.choice(("none", "channel", "token", "full")), dtype, rng.choice((dtype, dtype, "f32")),
                  rng.choice((dtype, "f32")), rng.choice((1.0, 1.0, 0.5)))
    else:
        T, E = _log(rng, 1, 16384), _log(rng, 1, 64)
        d_in, d_out = rng.choice(LAYERS) if rng.random() < 0.7 else (_log(rng, 64, 4096), _log(rng, 64, 4096))
        T = max(1, min(T, int(16384 * 2304 * 5760 // (d_in * d_out))))
        c = _group("", op, T, E, d_in, d_out, rng.choice((0.0, 0.5, 1.0)), rng.choice((0.0, 0.0, 0.3)),
                   rng.choice((0, 0, T // 10)), dtype, rng.choice((dtype, dtype, "f32")), rng.randint(1, 9999))
    del c["name"]
    return c


def _sizes(case):
    """Rows of each expert, from the case alone."""
    E, T = case["E"], case["T"] - case["spare"]
    rng = random.Random(case["route"])
    w = [(r + 1.0) ** -case["zipf"] for r in range(E)]
    rng.shuffle(w)
    live = [e for e in range(E) if rng.random() >= case["empty"]] or [0]
    w = [w[e] if e in set(live) else 0.0 for e in range(E)]
    n = [int(T * x / sum(w)) for x in w]
    n[live[0]] += T - sum(n)
    return n


def _clip_shapes(case):
    h, f, r = case["hidden"], case["ffn"], case["rank"]
    proj = [(h, h)] * 4 + [(f, h)] * 2 + [(h, f)]
    shapes = [s for o, i in proj for s in ((r, i), (o, r))] if r else proj
    shapes = shapes * case["layers"]
    types = [TYPES["f32"] if case["kind"] == "mixed" and k % 3 == 2 else TYPES[case["dtype"]] for k in range(len(shapes))]
    return shapes, types


def _randn(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def prepare(case, seed):
    """Values as in inputs.py: activations N(0, 1), weights N(0, 0.02), output gradients N(0, 0.01)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    op = case["op"]
    s = {"op": op}
    if op == "clip":
        shapes, types = _clip_shapes(case)
        s["grads"] = [_randn(g, sh, 0.01, t) for sh, t in zip(shapes, types)]
        s["outs"] = [torch.empty_like(x) for x in s["grads"]]
        s["max_norm"] = case["max_norm"]
        s["norm"] = torch.empty(1, device="cuda")
        if own:
            import gemms_linear_layers_gb300 as tg
            # the gradient buffers stay where they are for the whole run: their list is laid out once
            s["grads"], s["outs"] = tg.tg_tensor_list(s["grads"]), tg.tg_tensor_list(s["outs"])
        return s
    dt = TYPES[case["dtype"]]
    if op in ("norm_fwd", "norm_bwd"):
        T, d, res = case["T"], case["d"], TYPES[case["res"]]
        s["B"] = _randn(g, (T, d), 1.0, dt)
        s["w_post"], s["w_pre"] = (1 + _randn(g, (d,), 0.1, torch.float32)).to(dt), (1 + _randn(g, (d,), 0.1, torch.float32)).to(dt)
        shape = {"none": None, "channel": (d,), "token": (T, 1), "full": (T, d)}[case["gate"]]
        s["gate"] = None if shape is None else torch.rand(shape, generator=g, device="cuda").to(dt)
        s["scale"] = case["scale"]
        H = _randn(g, (T, d), 1.5, res)
        if op == "norm_fwd":
            s["H"] = H
            s["outs"] = {"H": torch.empty_like(H), "N": torch.empty_like(s["B"]),
                         "rstd_b": torch.empty(T, device="cuda"), "rstd_h": torch.empty(T, device="cuda")}
        else:
            s["H_out"] = H
            s["rstd_b"] = torch.rsqrt(s["B"].float().square().mean(1) + EPS)
            s["rstd_h"] = torch.rsqrt(H.float().square().mean(1) + EPS)
            s["dH_out"], s["dN"] = _randn(g, (T, d), 0.01, res), _randn(g, (T, d), 0.01, dt)
            wt = TYPES[case["out"]]
            s["outs"] = {"dB": torch.empty_like(s["B"]), "dH": torch.empty_like(H),
                         "dw_post": torch.empty(d, dtype=wt, device="cuda"), "dw_pre": torch.empty(d, dtype=wt, device="cuda")}
            if shape is not None:
                s["outs"]["dgate"] = torch.empty(shape, dtype=dt if case["gate"] == "full" else wt, device="cuda")
        return s
    T, E, d_in, d_out = case["T"], case["E"], case["d_in"], case["d_out"]
    n = _sizes(case)
    s["most"] = max(n)
    s["offsets"] = torch.tensor([0] + n, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    out = TYPES[case["out"]]
    if op != "dgrad":
        s["X"] = _randn(g, (T, d_in), 1.0, dt)
    if op != "fwd":
        s["dY"] = _randn(g, (T, d_out), 0.01, dt)
    if op != "wgrad":
        s["W"] = _randn(g, (E, d_out, d_in), 0.02, dt)
    s["out"] = torch.empty({"fwd": (T, d_out), "dgrad": (T, d_in), "wgrad": (E, d_out, d_in)}[op], dtype=out, device="cuda")
    return s


def _by_expert(x, offsets, most):
    """[T, d] -> [E, most, d] in FP32, rows past an expert's own left zero."""
    lo, hi = offsets[:-1, None].long(), offsets[1:, None].long()
    at = lo + torch.arange(most, device=x.device)
    return torch.where((at < hi)[..., None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)


def _from_expert(y, offsets, T):
    """[E, most, d] -> [T, d], rows of no expert zero."""
    t = torch.arange(T, device=y.device)
    e = torch.searchsorted(offsets[1:].long(), t, right=True)
    here = (e < y.shape[0]) & (t >= offsets[0])
    e = e.clamp(max=y.shape[0] - 1)
    at = (t - offsets[:-1].long()[e]).clamp(min=0, max=y.shape[1] - 1)
    return torch.where(here[:, None], y[e, at], 0.0)


def _plain(s):
    op = s["op"]
    if op == "fwd":
        y = torch.bmm(_by_expert(s["X"], s["offsets"], s["most"]), s["W"].float().transpose(1, 2))
        return s["out"].copy_(_from_expert(y, s["offsets"], s["X"].shape[0]))
    if op == "dgrad":
        y = torch.bmm(_by_expert(s["dY"], s["offsets"], s["most"]), s["W"].float())
        return s["out"].copy_(_from_expert(y, s["offsets"], s["dY"].shape[0]))
    if op == "wgrad":
        dY, X = _by_expert(s["dY"], s["offsets"], s["most"]), _by_expert(s["X"], s["offsets"], s["most"])
        return s["out"].copy_(torch.bmm(dY.transpose(1, 2), X))
    if op == "clip":
        norm = torch.stack([x.float().square().sum(dtype=torch.float64) for x in s["grads"]]).sum().sqrt()
        c = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0).float()
        return {"norm": s["norm"].copy_(norm), "grads": [o.copy_(x.float() * c) for x, o in zip(s["grads"], s["outs"])]}
    o = s["outs"]
    gate = 1.0 if s["gate"] is None else s["gate"].float()
    B, w_post, w_pre = s["B"].float(), s["w_post"].float(), s["w_pre"].float()
    if op == "norm_fwd":
        rstd_b = torch.rsqrt(B.square().mean(1) + EPS)
        H = s["scale"] * s["H"].float() + gate * (B * rstd_b[:, None] * w_post)
        rstd_h = torch.rsqrt(H.square().mean(1) + EPS)
        return {"H": o["H"].copy_(H), "N": o["N"].copy_(H * rstd_h[:, None] * w_pre),
                "rstd_b": o["rstd_b"].copy_(rstd_b), "rstd_h": o["rstd_h"].copy_(rstd_h)}
    rb, rh = s["rstd_b"][:, None], s["rstd_h"][:, None]
    dN, hn, bn = s["dN"].float(), s["H_out"].float() * rh, B * rb
    g1 = dN * w_pre
    dh = s["dH_out"].float() + rh * (g1 - hn * (g1 * hn).mean(1, keepdim=True))
    du = gate * dh
    g2 = du * w_post
    r = {"dB": o["dB"].copy_(rb * (g2 - bn * (g2 * bn).mean(1, keepdim=True))), "dH": o["dH"].copy_(s["scale"] * dh),
         "dw_post": o["dw_post"].copy_((du * bn).sum(0)), "dw_pre": o["dw_pre"].copy_((dN * hn).sum(0))}
    if s["gate"] is not None:
        dg = dh * bn * w_post
        dg = dg if s["gate"].dim() == 2 and s["gate"].shape[1] != 1 else dg.sum(1, keepdim=True) if s["gate"].dim() == 2 else dg.sum(0)
        r["dgate"] = o["dgate"].copy_(dg)
    return r


def run(state):
    if not own:
        return _plain(state)
    import gemms_linear_layers_gb300 as tg
    s, op = state, state["op"]
    if op == "fwd":
        return tg.tg_grouped_fwd(s["X"], s["W"], s["offsets"], Y=s["out"])
    if op == "dgrad":
        return tg.tg_grouped_dgrad(s["dY"], s["W"], s["offsets"], dX=s["out"])
    if op == "wgrad":
        return tg.tg_grouped_wgrad(s["dY"], s["X"], s["offsets"], dW=s["out"])
    if op == "clip":
        norm = tg.tg_grad_clip(s["grads"], s["max_norm"], outs=s["outs"], norm=s["norm"])
        return {"norm": norm, "grads": s["outs"].tensors}
    if op == "norm_fwd":
        return tg.tg_norm_residual_fwd(s["B"], s["H"], s["w_post"], s["w_pre"], gate=s["gate"], res_scale=s["scale"],
                                       eps=EPS, outs=s["outs"])
    return tg.tg_norm_residual_bwd(s["dH_out"], s["dN"], s["B"], s["H_out"], s["w_post"], s["w_pre"], s["rstd_b"],
                                   s["rstd_h"], gate=s["gate"], res_scale=s["scale"], outs=s["outs"])


_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def work(case):
    op = case["op"]
    if op == "clip":
        shapes, types = _clip_shapes(case)
        n = [a * b for a, b in shapes]
        # each gradient read once and written once
        return {"bytes": 2 * sum(k * (4 if t == torch.float32 else 2) for k, t in zip(n, types)) + 4, "flops": 3 * sum(n)}
    e = _BYTES[case["dtype"]]
    if op in ("norm_fwd", "norm_bwd"):
        T, d, r, w = case["T"], case["d"], _BYTES[case["res"]], _BYTES[case["out"]]
        gate = {"none": 0, "channel": d, "token": T, "full": T * d}[case["gate"]]
        if op == "norm_fwd":
            return {"bytes": T * d * (2 * e + 2 * r) + 2 * d * e + gate * e + 8 * T, "flops": 9 * T * d}
        dgate = gate * (e if case["gate"] == "full" else w)
        return {"bytes": T * d * (3 * e + 3 * r) + 2 * d * (e + w) + gate * e + dgate + 8 * T, "flops": 24 * T * d}
    n, d_in, d_out = _sizes(case), case["d_in"], case["d_out"]
    rows, live, o = sum(n), sum(x > 0 for x in n), _BYTES[case["out"]]
    if op == "fwd":
        b = rows * d_in * e + live * d_in * d_out * e + case["T"] * d_out * o
    elif op == "dgrad":
        b = rows * d_out * e + live * d_in * d_out * e + case["T"] * d_in * o
    else:
        b = rows * (d_in + d_out) * e + case["E"] * d_in * d_out * o
    return {"bytes": b + 4 * (case["E"] + 1), "flops": 2 * rows * d_in * d_out}


def exact(case, seed):
    """The definitions in 64 bits, expert by expert, tensor by tensor and with the norms written as functions."""
    s = prepare(case, seed)
    op = s["op"]
    if op in ("fwd", "dgrad", "wgrad"):
        ends = s["offsets"].tolist()
        shape = tuple(s["out"].shape)
        r = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for e, (a, b) in enumerate(zip(ends, ends[1:])):
            if op == "fwd":
                r[a:b] = torch.einsum("ti,oi->to", s["X"][a:b].double(), s["W"][e].double())
            elif op == "dgrad":
                r[a:b] = torch.einsum("to,oi->ti", s["dY"][a:b].double(), s["W"][e].double())
            else:
                r[e] = torch.einsum("to,ti->oi", s["dY"][a:b].double(), s["X"][a:b].double())
        return r
    if op == "clip":
        tensors = [g.double() for g in s["grads"]]
        norm = math.sqrt(math.fsum(float(torch.dot(g.flatten(), g.flatten())) for g in tensors))
        c = min(1.0, s["max_norm"] / (norm + 1e-6))
        return {"norm": torch.full((1,), norm, dtype=torch.float64, device="cuda"), "grads": [g.mul_(c) for g in tensors]}
    d = case["d"]
    up = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    gate = up.get("gate", torch.ones((), dtype=torch.float64, device="cuda"))
    if op == "norm_fwd":
        rb = ((up["B"] ** 2).sum(1) / d + EPS) ** -0.5
        H = torch.addcmul(s["scale"] * up["H"], gate, torch.einsum("td,t,d->td", up["B"], rb, up["w_post"]))
        rh = ((H ** 2).sum(1) / d + EPS) ** -0.5
        return {"H": H, "N": torch.einsum("td,t,d->td", H, rh, up["w_pre"]), "rstd_b": rb, "rstd_h": rh}

    def through_norm(x, r, w, dy):
        """Gradients of y = x r(x) w, r = rsqrt(mean(x^2) + eps) given as `r`, for x and w."""
        dxn = dy * w
        dx = dxn * r[:, None] - x * (r ** 3 * (dxn * x).sum(1) / d)[:, None]
        return dx, torch.einsum("td,td,t->d", dy, x, r)

    dx, dw_pre = through_norm(up["H_out"], up["rstd_h"], up["w_pre"], up["dN"])
    dh = dx + up["dH_out"]
    dB, dw_post = through_norm(up["B"], up["rstd_b"], up["w_post"], gate * dh)
    r = {"dB": dB, "dH": s["scale"] * dh, "dw_post": dw_post, "dw_pre": dw_pre}
    if case["gate"] != "none":
        dg = torch.einsum("td,td,t,d->td", dh, up["B"], up["rstd_b"], up["w_post"])
        r["dgate"] = {"full": dg, "token": dg.sum(1, keepdim=True), "channel": dg.sum(0)}[case["gate"]]
    return r
