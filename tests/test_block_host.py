"""Host-side checks of the dense block's operators (no GPU): arguments that the C entry points refuse before any device
work, and the binding's own checks."""
import ctypes

import pytest
import torch

import gemms_linear_layers_gb300 as tg
from gemms_linear_layers_gb300 import _binding as B
from gemms_linear_layers_gb300 import build

BF = torch.bfloat16
NULL, EVEN, ODD, HALF = (ctypes.c_void_p(x) for x in (0, 0x1000, 0x1001, 0x1002))
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def test_layer_norm_refuses(lib):
    def fwd(x=EVEN, w=EVEN, b=NULL, y=EVEN, stat=NULL, T=4, d=8, eps=1e-5, din=B.TG_BF16):
        return lib.tg_layer_norm_fwd(x, w, b, y, stat, stat, T, d, eps, din, NULL)

    for bad in ({"T": -1}, {"T": 1 << 31}, {"d": -8}, {"d": 16385}, {"eps": -1e-5}, {"eps": NAN}, {"eps": INF}, {"x": NULL},
                {"w": NULL}, {"y": NULL}):
        assert fwd(**bad) == 1, bad
    for bad in ({"din": 3}, {"din": -1}):
        assert fwd(**bad) == 2, bad
    for bad in ({"x": ODD}, {"w": ODD}, {"b": ODD}, {"y": HALF, "din": B.TG_F32}, {"b": HALF, "din": B.TG_F32}, {"stat": HALF}):
        assert fwd(**bad) == 3, bad

    def bwd(g=EVEN, x=EVEN, w=EVEN, stat=EVEN, r=NULL, dx=EVEN, dw=EVEN, db=NULL, T=4, d=8, din=B.TG_BF16, out=B.TG_BF16):
        return lib.tg_layer_norm_bwd(g, x, w, stat, stat, r, dx, dw, db, T, d, din, out, NULL, 0, NULL)

    for bad in ({"T": -1}, {"d": 16385}, {"g": NULL}, {"x": NULL}, {"w": NULL}, {"stat": NULL}, {"dx": NULL}, {"dw": NULL}):
        assert bwd(**bad) == 1, bad
    for bad in ({"din": 9}, {"out": B.TG_F16}, {"din": B.TG_F32, "out": B.TG_BF16}):
        assert bwd(**bad) == 2, bad
    for bad in ({"g": ODD}, {"r": ODD}, {"stat": HALF}, {"dw": HALF, "out": B.TG_F32}, {"db": HALF, "out": B.TG_F32}):
        assert bwd(**bad) == 3, bad


@pytest.mark.parametrize("fn", ["tg_gated_fwd", "tg_gated_bwd"])
def test_gated_refuses(lib, fn):
    def call(a=EVEN, w=EVEN, gu=EVEN, h=EVEN, T=4, f=8, d=8, act=0, din=B.TG_BF16):
        if fn == "tg_gated_fwd":
            return lib.tg_gated_fwd(a, w, h, gu, T, f, d, act, din, NULL, 0, NULL)
        return lib.tg_gated_bwd(a, w, gu, gu, h, T, f, d, act, din, NULL, 0, NULL)

    for bad in ({"T": -1}, {"f": -1}, {"d": -1}, {"T": (1 << 31) - 1}, {"f": (1 << 31) - 1}, {"d": 1 << 31}, {"act": 4},
                {"act": -1}, {"a": NULL}, {"w": NULL}, {"T": 1 << 30, "f": 1 << 10}, {"f": 1 << 20, "d": 1 << 20},
                {"h": NULL} if fn == "tg_gated_fwd" else {"gu": NULL}):
        assert call(**bad) == 1, bad
    for bad in ({"din": B.TG_F32}, {"din": 5}):
        assert call(**bad) == 2, bad
    for bad in ({"a": ODD}, {"w": ODD}, {"gu": ODD}, {"h": ODD}):
        assert call(**bad) == 3, bad


def test_orthogonalize_refuses(lib):
    def call(g=EVEN, o=EVEN, batch=1, rows=8, cols=8, coeffs=(3.4, -4.8, 2.0), steps=1, scale=1.0, eps=1e-7, din=B.TG_F32,
             out=B.TG_BF16):
        c = None if coeffs is None else (ctypes.c_double * len(coeffs))(*coeffs)
        return lib.tg_orthogonalize(g, o, batch, rows, cols, c, steps, scale, eps, din, out, NULL, 0, NULL)

    for bad in ({"batch": -1}, {"rows": -1}, {"cols": -1}, {"batch": (1 << 20) + 1}, {"rows": (1 << 20) + 1},
                {"cols": (1 << 20) + 1}, {"batch": 1 << 20, "rows": 1 << 10, "cols": 1 << 10}, {"steps": 0}, {"steps": 65},
                {"coeffs": None}, {"coeffs": (NAN, 0.0, 0.0)}, {"coeffs": (1.0, INF, 0.0)}, {"coeffs": (1.0, 0.0, 1e300)},
                {"scale": INF}, {"scale": NAN}, {"eps": -1.0}, {"eps": NAN}, {"g": NULL}, {"o": NULL}):
        assert call(**bad) == 1, bad
    for bad in ({"out": B.TG_F32}, {"din": 4}, {"out": 7}):
        assert call(**bad) == 2, bad
    for bad in ({"g": HALF}, {"o": ODD}):
        assert call(**bad) == 3, bad


def test_workspace_sizes_of_what_is_refused(lib):
    for op, dims, din, out in ((19, (4, 16385, 0, 0), 0, 0), (20, (1 << 31, 8, 8, 0), 0, 0), (21, (8, 8, 8, 0), 2, 2),
                               (22, (8, 1 << 20, 1 << 20, 0), 0, 0), (23, (1 << 20, 1 << 10, 1 << 10, 0), 2, 0),
                               (23, (1, 8, 8, 0), 2, 2), (19, (-1, 8, 0, 0), 0, 0)):
        assert lib.tg_workspace_size(op, *dims, din, out) == B.SIZE_MAX, (op, dims)


class OnDevice(torch.Tensor):
    is_cuda = True


def test_the_binding_refuses():
    x, w = torch.zeros(4, 8), torch.zeros(16, 8)
    for call in (lambda: tg.tg_layer_norm_fwd(x, x[0]), lambda: tg.tg_layer_norm_bwd(x, x, x[0], x[:, 0], x[:, 0]),
                 lambda: tg.tg_gated_fwd(x, w), lambda: tg.tg_gated_bwd(x, x, x), lambda: tg.tg_orthogonalize(x),
                 lambda: tg.tg_orthogonalize(x[0]), lambda: tg.tg_orthogonalize(None)):
        with pytest.raises(ValueError):
            call()


def test_arguments_that_the_binding_looks_at():
    assert B._act("gelu_tanh") == 2 and B._act(3) == 3
    for bad in ("swish", 4, None, -1):
        with pytest.raises(ValueError):
            B._act(bad)
    array, n = B._orth_coeffs((1.0, 2.0, 3.0), None)
    assert n == 5 and list(array) == [1.0, 2.0, 3.0] * 5
    array, n = B._orth_coeffs(((1.0, 2.0, 3.0), (4.0, 5.0, 6.0)), None)
    assert n == 2 and list(array) == [1.0, 2.0, 3.0, 4.0, 5.0, 6.0]
    for bad, steps in (((1.0, 2.0), None), (((1.0, 2.0, 3.0),), 2), (((1.0, 2.0), (3.0, 4.0, 5.0)), None), ((), None)):
        with pytest.raises(ValueError):
            B._orth_coeffs(bad, steps)


@pytest.mark.parametrize("steps", (0, -1, 65, 10 ** 15, 2.5))
def test_steps_are_looked_at_before_they_are_laid_out(steps):
    with pytest.raises(ValueError):
        B._orth_coeffs((1.0, 2.0, 3.0), steps)


def test_exported():
    import gemms_linear_layers_gb300 as pkg
    for n in B.SIGNATURES:
        if n.startswith(("tg_layer_norm", "tg_gated", "tg_orth")):
            assert n in pkg.__all__, n
