"""Plain 64-bit definitions of the expert-block operators, with the error scales their tolerances use.

Tolerances are derived, not fitted.  U = 2^-24 is FP32's half step.  An output
of a 16-bit type is off by at most half a step of that type beyond the FP32
error: `half_step`.
"""
import torch

U = 2.0 ** -24
PRODUCT = 1e-5  # FP32 accumulation on the tensor cores, relative to the sum of |a b|


def half_step(ref, dtype):
    """Half a unit of dtype at ref's values (zero for FP32: counted with the FP32 error)."""
    if dtype == torch.float32:
        return torch.zeros_like(ref)
    t = ref.abs() * (torch.finfo(dtype).eps / 2)
    return t.clamp(min=2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134)  # subnormals: steps of 2^-24, 2^-133


def check(got, ref, err, what):
    """|got - ref| <= err (FP32 part) + half a step of got's type (of a value that is itself off by err)."""
    g = got.detach().double().to(ref.device)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    bound = err + half_step(ref.abs() + err, got.dtype)
    off = (g - ref).abs()
    bad = ~(off <= bound)
    if bad.any():
        k = int(torch.argmax(torch.where(bad, off / bound.clamp(min=1e-300), torch.zeros_like(off)).flatten()))
        i = torch.unravel_index(torch.tensor(k), ref.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; worst at {[int(x) for x in i]}: got "
                             f"{float(g[i])} want {float(ref[i])} bound {float(bound[i])}")


# ------------------------------------------------------------ grouped products
def groups(offsets):
    o = [int(x) for x in offsets]
    return list(enumerate(zip(o, o[1:])))


def grouped_fwd(X, W, offsets):
    X, W = X.double(), W.double()
    Y = torch.zeros(X.shape[0], W.shape[1], dtype=torch.float64, device=X.device)
    S = torch.zeros_like(Y)
    for e, (a, b) in groups(offsets):
        Y[a:b] = X[a:b] @ W[e].T
        S[a:b] = X[a:b].abs() @ W[e].abs().T
    return Y, S


def grouped_dgrad(dY, W, offsets):
    return grouped_fwd(dY, W.transpose(1, 2), offsets)


def grouped_wgrad(dY, X, offsets):
    dY, X = dY.double(), X.double()
    C = torch.zeros(len(offsets) - 1, dY.shape[1], X.shape[1], dtype=torch.float64, device=X.device)
    S = torch.zeros_like(C)
    for e, (a, b) in groups(offsets):
        C[e] = dY[a:b].T @ X[a:b]
        S[e] = dY[a:b].abs().T @ X[a:b].abs()
    return C, S


# ---------------------------------------------------------- norms with residual
def norm_fwd(B, H, w_post, w_pre, gate, scale, eps):
    """{name: (value, FP32 error)}.  A row's sum of squares has only positive
    terms: at most d / 32 + 10 additions in a row, halved by the square root."""
    B, H, w_post, w_pre = (t.double() for t in (B, H, w_post, w_pre))
    gate = torch.ones((), dtype=torch.float64, device=B.device) if gate is None else gate.double()
    n = (B.shape[1] / 32 + 24) * U
    rb = (B.square().mean(1) + eps).rsqrt()
    u = gate * B * rb[:, None] * w_post
    Ho = scale * H + u
    size = (scale * H).abs() + u.abs()
    rh = (Ho.square().mean(1) + eps).rsqrt()
    # an error of n * size in the elements moves the row's norm by at most the norm of that error
    drift = (size.square().mean(1)).sqrt() * rh
    eh = n * size
    en = n * (size * rh[:, None] * w_pre.abs() + (Ho * rh[:, None] * w_pre).abs() * (1 + drift)[:, None])
    return {"H": (Ho, eh), "N": (Ho * rh[:, None] * w_pre, en), "rstd_b": (rb, n * rb),
            "rstd_h": (rh, n * rh * (1 + drift))}


def norm_bwd(dHo, dN, B, Ho, w_post, w_pre, rb, rh, gate, scale):
    """{name: (value, FP32 error)}: the formulas on values, and on magnitudes for the error scale."""
    T, d = B.shape
    kind = None if gate is None else tuple(gate.shape)
    args = [t.double() for t in (dHo, dN, B, Ho, w_post, w_pre)]
    rb, rh = rb.double()[:, None], rh.double()[:, None]
    g = torch.ones((), dtype=torch.float64, device=B.device) if gate is None else gate.double()

    def formulas(dHo, dN, B, Ho, w_post, w_pre, g, sign):
        hn, bn, g1 = Ho * rh, B * rb, dN * w_pre
        dh = dHo + rh * (g1 - sign * hn * (g1 * hn).mean(1, keepdim=True))
        g2 = g * dh * w_post
        r = {"dB": rb * (g2 - sign * bn * (g2 * bn).mean(1, keepdim=True)), "dH": scale * dh if sign > 0 else abs(scale) * dh,
             "dw_post": (g * dh * bn).sum(0), "dw_pre": (dN * hn).sum(0)}
        dg = dh * bn * w_post
        if kind is not None:
            r["dgate"] = dg if kind == (T, d) else dg.sum(1, keepdim=True) if kind == (T, 1) else dg.sum(0)
        return r

    v = formulas(*args, g, 1.0)
    m = formulas(*[t.abs() for t in args], g.abs(), -1.0)
    # roundings along the longest chain: two row sums (d / 32 + 10 additions each), a column sum (T), about 30 more
    n = (2 * (d / 32 + 10) + T + 30) * U
    return {k: (v[k], n * m[k]) for k in v}


# ------------------------------------------------------------------- clipping
def clip(grads, max_norm):
    s = sum(float(g.double().square().sum()) for g in grads)
    norm = s ** 0.5
    c = min(1.0, max_norm / (norm + 1e-6)) if norm == norm else float("nan")
    return norm, c, [g.double() * c for g in grads]
