"""Plain 64-bit definitions of the dense feed-forward block's operators, with the error scales their tolerances use.

Tolerances are derived, not fitted: every function returns values and an FP32 error bound; expert_ref.check adds half a
step of the output's type.  U = 2^-24 is FP32's half step.  SUM bounds the additions that a value passes through in a
row's sums (24 in a thread, 5 + 5 in shuffles, the products before and after: fewer than 64 roundings).
"""
import math

import torch

from expert_ref import PRODUCT, U, check, half_step  # noqa: F401  (for the tests)

SUM = 64 * U
# The activations' own error: e^x to within 2 + 1.2 |x| units (|x| < 26 where the logistic function is not 0 or 1 in
# 16 bits) and a divide of 2: below 2^-18.  GELU's tail is off by 1.1e-6 and by the rounding of its exponent,
# x^2 / 2 twice, which is x^2 2^-24: `act` returns that beside the values.
ACT = 2.0 ** -18


def layer_norm_fwd(X, w, b, eps):
    """({Y, mean, rstd}, their FP32 errors)."""
    X, w = X.double(), w.double()
    mean = X.mean(1)
    dev = X - mean[:, None]
    rstd = (dev.square().mean(1) + eps) ** -0.5
    Y = dev * rstd[:, None] * w
    size = X.abs().mean(1)
    e_mean = SUM * size
    # squares are of distances from means that are each off by e_mean: 2 e_mean / sigma of them, half of that in rstd
    e_rstd = rstd * (2 * SUM + 2 * e_mean * rstd)
    e_Y = ((dev.abs() * (e_rstd + 4 * U * rstd)[:, None] + (rstd * e_mean)[:, None] + U * rstd[:, None] * X.abs()) * w.abs()
           + 2 * U * Y.abs())
    if b is not None:
        Y = Y + b.double()
        e_Y = e_Y + U * Y.abs()
    return {"Y": Y, "mean": mean, "rstd": rstd}, {"Y": e_Y, "mean": e_mean, "rstd": e_rstd}


def layer_norm_bwd(dY, X, w, mean, rstd, dR):
    """({dX, dw, db}, their FP32 errors) for the given mean and rstd."""
    dY, X, w, mean, rstd = (t.double() for t in (dY, X, w, mean[:, None], rstd[:, None]))
    n = (X - mean) * rstd
    q = dY * w
    m1, m2 = q.mean(1, keepdim=True), (q * n).mean(1, keepdim=True)
    dX = rstd * (q - m1 - n * m2)
    e_dX = rstd.abs() * (8 * U * (q.abs() + m1.abs() + (n * m2).abs())
                         + SUM * (q.abs().mean(1, keepdim=True) + n.abs() * (q * n).abs().mean(1, keepdim=True)))
    if dR is not None:
        dX = dX + dR.double()
    e_dX = e_dX + U * dX.abs()
    rows = SUM + U * X.shape[0] / 100  # a thread adds the rows of its team, 1 of 152 or more; then teams and CTAs
    return ({"dX": dX, "dw": (dY * n).sum(0), "db": dY.sum(0)},
            {"dX": e_dX, "dw": rows * (dY * n).abs().sum(0), "db": rows * dY.abs().sum(0)})


def act(kind, x):
    """(value, derivative, scale of the derivative's error, relative error) of an activation in 64 bits."""
    if kind == "silu":
        p = torch.sigmoid(x)
        return x * p, p * (1 + x * (1 - p)), p * (1 + x.abs()), ACT
    if kind == "gelu":
        p = 0.5 * torch.special.erfc(-x * math.sqrt(0.5))
        d = torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
        return x * p, p + x * d, p + x.abs() * d, ACT + x * x * U
    if kind == "gelu_tanh":
        k = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(k * (x + 0.044715 * x ** 3))
        d = p * (1 - p) * k * (1 + 3 * 0.044715 * x * x)
        return x * p, p + x * d, p + x.abs() * d, ACT
    return x.clamp(min=0), (x > 0).double(), torch.zeros_like(x), 0.0


def gated_fwd(X, W, kind):
    """({H, GU}, their FP32 errors)."""
    X, W = X.double(), W.double()
    P, e = X @ W.T, PRODUCT * (X.abs() @ W.abs().T)
    f = W.shape[0] // 2
    G, Up, eg, eu = P[:, :f], P[:, f:], e[:, :f], e[:, f:]
    A, _, _, ea = act(kind, G)
    # no activation here is steeper than 1.13
    eh = 1.13 * eg * (Up.abs() + eu) + A.abs() * eu + (ea + 2 * U) * (A * Up).abs()
    return {"H": A * Up, "GU": P}, {"H": eh, "GU": e}


def gated_bwd(dY, W_down, GU, kind):
    """({dGU, H}, their FP32 errors)."""
    dY, W, GU = dY.double(), W_down.double(), GU.double()
    dH, e = dY @ W, PRODUCT * (dY.abs() @ W.abs())
    f = W.shape[1]
    G, Up = GU[:, :f], GU[:, f:]
    A, dA, s, ea = act(kind, G)
    dG, dU = dH * Up * dA, dH * A
    edG = e * (Up * dA).abs() + (dH * Up).abs() * 2 * ea * s + 3 * U * dG.abs()
    edU = e * A.abs() + (ea + U) * dU.abs()
    return {"dGU": torch.cat((dG, dU), 1), "H": A * Up}, {"dGU": torch.cat((edG, edU), 1), "H": (ea + U) * (A * Up).abs()}


def orthogonalize(G, coeffs, scale, eps, out):
    """(O, bound on |O' - O| in the Frobenius norm before O' is rounded to `out`) of one matrix.

    X and what is made of it are held to 2^-17, each product has two such factors.  For a step of X with largest
    singular value s that is at most 2^-17 |X| (a + 3 b s^2 + 9 c s^4) (A: 2 factors and itself; A A: 2 of 3 and
    itself, and 2 more in Q X); later steps enlarge it by at most max |p'| and |p(s) / s| of theirs on [0, s].
    The last step of a bf16 result has X, D = A - I and E in one fp16 part in its products, u = 2^-11: with
    e = 2 u s |X| + u |D| in D, it is s ((|b + 2 c| + 2 |c| |D|_2) e + u |E|) + |E|_2 u |X|."""
    X = G.double()
    X = X / (torch.linalg.vector_norm(X) + eps)
    noise = 0.0
    fro = lambda M: float(torch.linalg.vector_norm(M))  # noqa: E731
    for i, (a, b, c) in enumerate(coeffs):
        A = X @ X.T if X.shape[0] <= X.shape[1] else X.T @ X
        eye = torch.eye(A.shape[0], dtype=torch.float64, device=X.device)
        finite = bool(torch.isfinite(A).all())
        squares = torch.linalg.eigvalsh(A.cpu()).clamp(min=0) if finite else torch.zeros(1, dtype=torch.float64)
        s = math.sqrt(float(squares.max()))
        grid = torch.linspace(0, 1, 401, dtype=torch.float64) * s
        steep = max(float((a + 3 * b * grid ** 2 + 5 * c * grid ** 4).abs().max()),
                    float((a + b * grid ** 2 + c * grid ** 4).abs().max()))
        here = 2.0 ** -17 * fro(X) * (abs(a) + 3 * abs(b) * s ** 2 + 9 * abs(c) * s ** 4)
        if out == torch.bfloat16 and i > 0 and i + 1 == len(coeffs) and abs(b + 2 * c) + abs(c) <= 3:
            u, D, d = 2.0 ** -11, A - eye, squares - 1
            E = (b + 2 * c) * D + c * D @ D
            e = 2 * u * s * fro(X) + u * fro(D)
            here += (s * ((abs(b + 2 * c) + 2 * abs(c) * float(d.abs().max())) * e + u * fro(E))
                     + float(((b + 2 * c) * d + c * d ** 2).abs().max()) * u * fro(X))
        noise = noise * steep + here
        Q = a * eye + b * A + c * A @ A
        X = Q @ X if X.shape[0] <= X.shape[1] else X @ Q
    return scale * X, abs(scale) * noise
