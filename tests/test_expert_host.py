"""Host-side checks of the expert-block operators (no GPU): arguments that the C entry points refuse before any
device work, and the binding's own checks."""
import contextlib
import ctypes
import threading

import pytest
import torch
from torch.multiprocessing.reductions import StorageWeakRef

import gemms_linear_layers_gb300 as tg
from gemms_linear_layers_gb300 import _binding as B
from gemms_linear_layers_gb300 import build, expert_step

BF = torch.bfloat16
NULL, EVEN, ODD, HALF = (ctypes.c_void_p(x) for x in (0, 0x1000, 0x1001, 0x1002))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


@pytest.mark.parametrize("fn", ["tg_grouped_fwd", "tg_grouped_dgrad", "tg_grouped_wgrad"])
def test_grouped_products_refuse(lib, fn):
    f = getattr(lib, fn)

    def call(a=EVEN, b=EVEN, off=EVEN, c=EVEN, T=8, E=2, o=8, i=8, din=B.TG_BF16, dout=B.TG_BF16):
        return f(a, b, off, c, T, E, o, i, din, dout, NULL, 0, NULL)

    for bad in ({"T": -1}, {"E": -1}, {"o": -8}, {"i": 1 << 31}, {"T": (1 << 31) - 1},
                {"E": 1 << 30, "o": 1 << 30, "i": 1 << 30}, {"E": 1 << 20, "o": 1 << 20, "i": 512}):
        assert call(**bad) == 1, bad
    for bad in ({"a": NULL}, {"b": NULL}, {"off": NULL}, {"c": NULL}):
        assert call(**bad) == 1, bad
    for bad in ({"din": B.TG_F32, "dout": B.TG_F32}, {"din": 7}, {"dout": B.TG_F16}):
        assert call(**bad) == 2, bad
    for bad in ({"a": ODD}, {"b": ODD}, {"c": ODD}, {"off": HALF}, {"c": HALF, "dout": B.TG_F32}):
        assert call(**bad) == 3, bad


def test_norms_refuse(lib):
    def fwd(B_=EVEN, H=EVEN, w=EVEN, gate=NULL, kind=0, out=EVEN, rstd=EVEN, T=4, d=8, scale=1.0, eps=1e-6,
            din=B.TG_BF16, res=B.TG_BF16):
        return lib.tg_norm_residual_fwd(B_, H, w, w, gate, kind, out, out, rstd, rstd, T, d, scale, eps, din, res, NULL)

    for bad in ({"T": -1}, {"d": -8}, {"d": 16385}, {"scale": float("nan")}, {"scale": float("inf")}, {"eps": -1e-6},
                {"eps": float("nan")}, {"kind": 4}, {"kind": -1}, {"kind": 1}, {"B_": NULL}, {"H": NULL}, {"w": NULL},
                {"out": NULL}):
        assert fwd(**bad) == 1, bad
    for bad in ({"din": 5}, {"res": B.TG_F16}, {"din": B.TG_F32, "res": B.TG_BF16}):
        assert fwd(**bad) == 2, bad
    for bad in ({"B_": ODD}, {"H": HALF, "res": B.TG_F32}, {"rstd": HALF}, {"kind": 2, "gate": ODD}):
        assert fwd(**bad) == 3, bad

    def bwd(g=EVEN, w=EVEN, gate=NULL, kind=0, rstd=EVEN, dx=EVEN, dw=EVEN, dgate=NULL, T=4, d=8, scale=1.0,
            din=B.TG_BF16, res=B.TG_BF16, out=B.TG_BF16):
        return lib.tg_norm_residual_bwd(g, g, g, g, w, w, gate, kind, rstd, rstd, dx, dx, dw, dw, dgate, T, d, scale, din,
                                        res, out, NULL, 0, NULL)

    for bad in ({"T": -1}, {"d": 16385}, {"scale": float("inf")}, {"kind": 9}, {"g": NULL}, {"rstd": NULL}, {"dx": NULL},
                {"dw": NULL}, {"kind": 3, "gate": EVEN}, {"kind": 3, "dgate": EVEN}):
        assert bwd(**bad) == 1, bad
    for bad in ({"din": 9}, {"res": B.TG_F16}, {"out": B.TG_F16}):
        assert bwd(**bad) == 2, bad
    for bad in ({"g": ODD}, {"rstd": HALF}, {"dw": HALF, "out": B.TG_F32}, {"kind": 1, "gate": EVEN, "dgate": ODD}):
        assert bwd(**bad) == 3, bad


def test_clipping_refuses(lib):
    def call(p=0x1000, o=0x1000, n=5, dt=B.TG_F32, count=1, max_norm=1.0, norm=EVEN, outs=True):
        ps, os, ns, ds = (ctypes.c_void_p * 1)(p), (ctypes.c_void_p * 1)(o), (ctypes.c_int64 * 1)(n), (ctypes.c_int32 * 1)(dt)
        return lib.tg_grad_clip(ps, os if outs else NULL, ns, ds, count, max_norm, norm, NULL, 0, NULL)

    for bad in ({"count": -1}, {"count": (1 << 20) + 1}, {"max_norm": -1.0}, {"max_norm": float("nan")}, {"norm": NULL},
                {"p": 0}, {"o": 0}, {"n": -1}, {"n": 1 << 41}, {"outs": False}):
        assert call(**bad) == 1, bad
    assert call(dt=3) == 2 and call(dt=-1) == 2
    for bad in ({"p": 0x1002}, {"o": 0x1001, "dt": B.TG_BF16, "p": 0x1000}, {"norm": HALF}):
        assert call(**bad) == 3, bad
    assert lib.tg_grad_norm(NULL, NULL, NULL, 1, EVEN, NULL, 0, NULL) == 1


def test_the_binding_takes_cuda_tensors_only():
    x, w, o = torch.zeros(4, 8), torch.zeros(2, 8, 8), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        tg.tg_grouped_fwd(x, w, o)
    with pytest.raises(ValueError):
        tg.tg_grouped_wgrad(x, x, o)
    with pytest.raises(ValueError):
        tg.tg_norm_residual_fwd(x, x, x[0], x[0])
    with pytest.raises(ValueError):
        tg.tg_tensor_list([x])


def test_exported():
    import gemms_linear_layers_gb300 as pkg
    for n in B.SIGNATURES:
        if n.startswith(("tg_grouped", "tg_norm", "tg_grad")):
            assert n in pkg.__all__, n


class OnDevice(torch.Tensor):
    is_cuda = True


class Sizes:
    """Stands for the library in `_scratch`: workspaces of the given sizes, one after the other."""

    def __init__(self, *sizes):
        self.sizes = list(sizes)

    def tg_workspace_size(self, *_):
        return self.sizes.pop(0) if len(self.sizes) > 1 else self.sizes[0]


def scratch(monkeypatch, *sizes):
    monkeypatch.setattr(B, "_lib", Sizes(*sizes))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return lambda raw=7, stream=None: B._scratch(B.TG_OP_NORM_RESIDUAL_BWD, (1, 1, 0, 0), 0, 0, None, torch.device("cpu"),
                                                 stream, raw)


def test_threads_on_one_stream_have_workspaces_of_their_own(monkeypatch):
    """A call's launches pass data through its workspace, and another thread's launches on the same stream may land
    between them."""
    take = scratch(monkeypatch, 4096)
    here, there = take(), []
    t = threading.Thread(target=lambda: there.append(take()))
    t.start()
    t.join()
    assert here[0] != there[0][0]
    assert take()[0] == here[0]  # the same thread's next call on the stream: the same buffer
    assert take(raw=8)[0] != here[0]


def test_a_workspace_outlives_its_replacement_by_a_larger_one(monkeypatch):
    """The buffer goes with the call until its launches are queued, whatever replaces it among the kept ones."""
    take = scratch(monkeypatch, 4096, 4 << 20)
    address, size, buf = take()
    assert size >= 4096 and buf.data_ptr() == address
    assert take()[0] != address


def test_memory_of_a_call_on_a_given_stream_is_that_streams(monkeypatch):
    """What a call on the caller's own stream allocates comes from that stream's memory: the current stream's may
    still be read by work queued there, which the other stream does not wait for."""
    current, taken = ["current"], []

    class Buffer:
        def __init__(self):
            self.used_on = []

        def data_ptr(self):
            return 0x1000

        def record_stream(self, s):
            self.used_on.append(s)

    @contextlib.contextmanager
    def enter(s):
        current.append(s)
        yield
        current.pop()

    def empty(*_, **__):
        taken.append(current[-1])
        return Buffer()

    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: current[-1])
    monkeypatch.setattr(torch, "empty", empty)
    take = scratch(monkeypatch, 4096)
    take(stream="side")
    assert taken.pop() == "side"
    res = {}
    B._result(res, None, "dB", (2, 3), BF, torch.device("cpu"), "side")
    assert taken.pop() == "side" and res["dB"].used_on == ["current"]  # where the caller may go on with it
    B._result(res, None, "dH", (2, 3), BF, torch.device("cpu"), None)
    assert taken.pop() == "current" and res["dH"].used_on == []


@pytest.mark.parametrize("fn", ["tg_grouped_fwd", "tg_grouped_dgrad", "tg_grouped_wgrad"])
def test_grouped_products_refuse_what_their_tiles_cannot_count(lib, fn):
    """Widths within a tile of 2^31 (the tile counts are 32-bit) and tensors of more than 2^38 elements; sizes at
    the limits pass the checks of sizes (and end at the missing device or at a tensor's address)."""
    def call(T=1, E=1, o=8, i=8):
        return getattr(lib, fn)(EVEN, EVEN, EVEN, ODD, T, E, o, i, B.TG_BF16, B.TG_BF16, NULL, 0, NULL)

    top = (1 << 31) - 1024
    for bad in ({"o": top + 1}, {"i": top + 1}, {"o": (1 << 31) - 1}, {"i": (1 << 31) - 1}, {"T": top + 1},
                {"E": 1 << 20, "o": 1 << 10, "i": (1 << 8) + 1}, {"T": 1 << 20, "o": (1 << 18) + 1},
                {"T": 1 << 20, "i": (1 << 18) + 1}):
        assert call(**bad) == 1, bad
    for good in ({"o": top}, {"i": top}, {"T": top}, {"E": 1 << 20, "o": 1 << 10, "i": 1 << 8}, {"T": 1 << 20, "o": 1 << 18},
                 {"T": 1 << 20, "i": 1 << 18}):
        assert call(**good) == 3, good


def test_a_list_whose_tensors_moved_is_refused():
    """A laid-out list holds addresses: a tensor that was given other memory since is an error, not a write to where
    it used to be, and that memory is held meanwhile."""
    a, b = (torch.zeros(n).as_subclass(OnDevice) for n in (5, 3))
    laid_out = tg.tg_tensor_list([a, b])
    memory = StorageWeakRef(b.untyped_storage())
    b.data = torch.ones(3).as_subclass(OnDevice)
    assert not memory.expired()
    for call in (lambda: tg.tg_grad_norm(laid_out), lambda: tg.tg_grad_clip(laid_out, 1.0),
                 lambda: tg.tg_grad_clip(tg.tg_tensor_list([a, b]), 1.0, outs=laid_out)):
        with pytest.raises(ValueError, match="tensor 1 "):
            call()


@pytest.mark.parametrize("given", ["dw_post", "dw_pre", "dgate"])
def test_the_type_of_summed_gradients_follows_any_given_output(monkeypatch, given):
    """One FP32 output given among those summed over rows: the others come in FP32 too; one that is None is new."""
    class Library:
        def tg_workspace_size(self, *_):
            return 0

        def tg_norm_residual_bwd(self, *args):
            self.out_type = args[20]  # after dtypes in, res
            return 0

    library = Library()
    monkeypatch.setattr(B, "_lib", library)
    monkeypatch.setattr(B, "_raw_stream", lambda *_: 0)
    dev = lambda *shape, dtype=BF: torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)
    x, w, r = dev(4, 8), dev(8), dev(4, dtype=torch.float32)
    outs = {"dw_post": None, "dw_pre": None, "dgate": None, given: dev(8, dtype=torch.float32)}
    got = tg.tg_norm_residual_bwd(x, x, x, x, w, w, r, r, gate=w, outs=outs)
    assert library.out_type == B.TG_F32 and got[given] is outs[given]
    assert all(got[k].dtype == torch.float32 for k in ("dw_post", "dw_pre", "dgate")) and got["dB"].dtype == BF
    full = tg.tg_norm_residual_bwd(x, x, x, x, w, w, r, r, gate=x, outs={"dgate": dev(4, 8)})  # of B's type
    assert full["dw_pre"].dtype == BF
    with pytest.raises(ValueError):
        tg.tg_norm_residual_bwd(x, x, x, x, w, w, r, r, gate=w, outs={**outs, "dw_post": dev(8), "dw_pre": r[:0]})


def test_the_examples_gradient_is_that_of_its_loss():
    g = torch.Generator().manual_seed(3)
    out, target = torch.randn(7, 24, generator=g, dtype=torch.float64), torch.randn(7, 24, generator=g, dtype=torch.float64)
    loss, grad = expert_step.loss_and_gradient(out, target)
    assert grad.dtype == out.dtype
    for k in range(3):  # quadratic: its central difference is the derivative, but for roundings
        D = torch.randn(7, 24, generator=g, dtype=torch.float64)
        up, down = (expert_step.loss_and_gradient(out + s * D, target)[0] for s in (0.5, -0.5))
        assert float((grad * D).sum()) == pytest.approx(float(up - down), rel=1e-4)  # FP32: sums of 168 terms
    assert float(loss) > 0
