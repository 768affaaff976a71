"""The dense feed-forward block's operators against their 64-bit definitions: layer norm, the gated projections and
their backward, the orthogonalised update."""
import math

import pytest
import torch

import gemms_linear_layers_gb300 as tg
from gemms_linear_layers_gb300 import inputs
import block_ref as R

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ("silu", "gelu", "gelu_tanh", "relu")
QUINTIC = (3.4445, -4.7750, 2.0315)


def randn(shape, std, dtype, tag):
    return inputs.normal(shape, std, dtype, inputs.seed_for("block", *shape, str(dtype), tag)).cuda()


def off16(t):
    """The same values at an address that is no multiple of 16 bytes."""
    b = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)[1:].view(t.shape)
    assert b.data_ptr() % 16
    return b.copy_(t)


def same(t):
    return t


# ----------------------------------------------------------------- layer norm
LN_SIZES = [(1, 1), (1, 8), (2, 7), (5, 31), (3, 33), (17, 64), (8, 576), (301, 576), (2, 2304), (700, 2304), (1, 2301),
            (333, 2301), (40, 1003), (64, 4100), (5, 5760), (9, 8191), (7, 8200), (3, 12289), (2, 16384), (400, 10240),
            (5001, 576), (5001, 577), (3101, 2304), (3101, 2302), (1231, 5124)]  # teams of several rows: two at a time


def ln_inputs(T, d, dtype, place=same):
    X = randn((T, d), 1.0, F32, "x") * torch.exp(0.5 * randn((d,), 1.0, F32, "size")) + randn((d,), 0.5, F32, "mean")
    t = {"X": X.to(dtype), "w": (1 + randn((d,), 0.1, F32, "w")).to(dtype), "b": randn((d,), 0.1, dtype, "b"),
         "dY": randn((T, d), 0.01, dtype, "dY"), "dR": randn((T, d), 0.01, dtype, "dR")}
    return {k: place(v) for k, v in t.items()}


def check_all(got, ref, err, what, keys=None):
    for k in keys or got:
        R.check(got[k], ref[k], err[k], f"{what} {k}")


@pytest.mark.parametrize("dtype", (BF, HF, F32))
@pytest.mark.parametrize("T,d", LN_SIZES)
def test_layer_norm_forward(T, d, dtype):
    t = ln_inputs(T, d, dtype)
    for b in (t["b"], None):
        got = tg.tg_layer_norm_fwd(t["X"], t["w"], b=b, eps=1e-5)
        check_all(got, *R.layer_norm_fwd(t["X"], t["w"], b, 1e-5), f"{T}x{d} {dtype}")


@pytest.mark.parametrize("dtype", (BF, HF, F32))
@pytest.mark.parametrize("T,d", LN_SIZES)
def test_layer_norm_backward(T, d, dtype):
    t = ln_inputs(T, d, dtype)
    stat = R.layer_norm_fwd(t["X"], t["w"], None, 1e-5)[0]
    mean, rstd = stat["mean"].float(), stat["rstd"].float()
    for dR, bias, out in ((None, True, F32), (t["dR"], True, dtype), (t["dR"], False, F32)):
        got = tg.tg_layer_norm_bwd(t["dY"], t["X"], t["w"], mean, rstd, dR=dR, bias=bias, out_dtype=out)
        assert set(got) == {"dX", "dw"} | ({"db"} if bias else set()) and got["dw"].dtype == out
        check_all(got, *R.layer_norm_bwd(t["dY"], t["X"], t["w"], mean, rstd, dR), f"{T}x{d} {dtype} {out}")


@pytest.mark.parametrize("dtype", (BF, F32))
@pytest.mark.parametrize("T,d", [(5, 576), (301, 33), (3, 9000), (2, 15000)])
def test_layer_norm_off_16_bytes(T, d, dtype):
    t = ln_inputs(T, d, dtype, off16)
    got = tg.tg_layer_norm_fwd(t["X"], t["w"], b=t["b"], outs={"Y": off16(t["X"])})
    ref, err = R.layer_norm_fwd(t["X"], t["w"], t["b"], 1e-5)
    check_all(got, ref, err, f"{T}x{d} {dtype}")
    m, r = got["mean"], got["rstd"]
    got = tg.tg_layer_norm_bwd(t["dY"], t["X"], t["w"], m, r, dR=t["dR"])
    check_all(got, *R.layer_norm_bwd(t["dY"], t["X"], t["w"], m, r, t["dR"]), f"{T}x{d} {dtype}")


@pytest.mark.parametrize("T,d", [(19, 576), (40, 2301), (3, 12289)])
def test_layer_norm_far_from_zero(T, d):
    """A mean a thousand times the deviation: the bound (e_mean / sigma) allows 1e-2 of rstd, squares of X itself would
    leave nothing of the variance."""
    X = randn((T, d), 1.0, F32, "far") + 1000.0
    w, b = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    got = tg.tg_layer_norm_fwd(X, w, b=b, eps=0.0)
    ref, err = R.layer_norm_fwd(X, w, b, 0.0)
    assert float((err["rstd"] / ref["rstd"]).max()) < 0.01
    check_all(got, ref, err, f"{T}x{d}")


@pytest.mark.parametrize("T,d", [(70, 1003), (3333, 2304), (5001, 577)])
def test_layer_norm_in_place_and_rows_apart(T, d):
    t = ln_inputs(T, d, BF)
    stat = tg.tg_layer_norm_fwd(t["X"], t["w"], b=t["b"])
    X = t["X"].clone()
    assert torch.equal(tg.tg_layer_norm_fwd(X, t["w"], b=t["b"], outs={"Y": X})["Y"], stat["Y"])
    want = tg.tg_layer_norm_bwd(t["dY"], t["X"], t["w"], stat["mean"], stat["rstd"], dR=t["dR"])
    for k in ("dY", "dR", "X"):
        a = {n: v.clone() for n, v in t.items()}
        got = tg.tg_layer_norm_bwd(a["dY"], a["X"], a["w"], stat["mean"], stat["rstd"], dR=a["dR"], outs={"dX": a[k]})
        assert all(torch.equal(got[n], want[n]) for n in want), k
    # values that are not numbers stay in their row
    bad = t["X"].clone()
    bad[5, 3], bad[9, 0] = math.inf, math.nan
    got = tg.tg_layer_norm_fwd(bad, t["w"], b=t["b"])["Y"]
    rows = [i for i in range(T) if i not in (5, 9)]
    assert torch.equal(got[rows], stat["Y"][rows]) and got[9].isnan().all()


def test_layer_norm_empty():
    for T, d in ((0, 64), (4, 0)):
        X, w = torch.empty(T, d, dtype=BF, device="cuda"), torch.ones(d, dtype=BF, device="cuda")
        tg.tg_layer_norm_fwd(X, w, b=w)
        z = torch.zeros(T, device="cuda")
        got = tg.tg_layer_norm_bwd(X, X, w, z, z, out_dtype=F32)
        assert not got["dw"].any() and not got["db"].any()


def test_layer_norm_gradient_by_differences():
    t = ln_inputs(6, 40, F32)
    X, w, b, g = (t[k].double().cpu() for k in ("X", "w", "b", "dY"))

    def loss(X, w, b):
        return float((R.layer_norm_fwd(X, w, b, 1e-5)[0]["Y"] * g).sum())

    f = tg.tg_layer_norm_fwd(t["X"], t["w"], b=t["b"])
    got = tg.tg_layer_norm_bwd(t["dY"], t["X"], t["w"], f["mean"], f["rstd"])
    h = 1e-5  # the difference is off by h^2 f''' / 6 and 2^-52 |loss| / h, below 1e-8
    for i, j in ((0, 0), (3, 17), (5, 39)):
        d = torch.zeros_like(X)
        d[i, j] = h
        assert abs((loss(X + d, w, b) - loss(X - d, w, b)) / (2 * h) - float(got["dX"][i, j])) < 1e-7
    for j in (0, 21):
        d = torch.zeros_like(w)
        d[j] = h
        assert abs((loss(X, w + d, b) - loss(X, w - d, b)) / (2 * h) - float(got["dw"][j])) < 1e-6
        assert abs((loss(X, w, b + d) - loss(X, w, b - d)) / (2 * h) - float(got["db"][j])) < 1e-6


# ----------------------------------------------------------- the gated block
GATED_SIZES = [(1, 8, 8), (1, 64, 576), (3, 7, 5), (16, 1536, 576), (5, 200, 2304), (33, 130, 1501), (64, 1000, 3000),
               (100, 5760, 2304), (31, 33, 65), (127, 200, 72), (128, 128, 64),
               (129, 130, 129), (256, 256, 128), (257, 1000, 999), (300, 1536, 576), (1001, 321, 200), (513, 5760, 2304)]


def gated_inputs(T, f, d, dtype, place=same):
    t = {"X": randn((T, d), 1.0, dtype, "X"), "W": randn((2 * f, d), 1.2 / math.sqrt(d), dtype, "W"),
         "dY": randn((T, d), 0.1, dtype, "dY"), "Wd": randn((d, f), 0.05, dtype, "Wd"),
         "GU": randn((T, 2 * f), 1.5, dtype, "GU")}
    return {k: place(v) for k, v in t.items()}


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,f,d", GATED_SIZES)
def test_gated(T, f, d, act):
    dtype = HF if (T + f + d + len(act)) % 2 else BF
    t = gated_inputs(T, f, d, dtype)
    ref, err = R.gated_fwd(t["X"], t["W"], act)
    got = tg.tg_gated_fwd(t["X"], t["W"], act=act, keep=True)
    check_all(got, ref, err, f"{T}x{f}x{d} {act} {dtype}")
    alone = tg.tg_gated_fwd(t["X"], t["W"], act=act)
    assert set(alone) == {"H"} and torch.equal(alone["H"], got["H"])
    ref, err = R.gated_bwd(t["dY"], t["Wd"], t["GU"], act)
    got = tg.tg_gated_bwd(t["dY"], t["Wd"], t["GU"], act=act, keep=True)
    check_all(got, ref, err, f"{T}x{f}x{d} {act} {dtype} backward")
    alone = tg.tg_gated_bwd(t["dY"], t["Wd"], t["GU"], act=act)
    assert set(alone) == {"dGU"} and torch.equal(alone["dGU"], got["dGU"])
    GU = t["GU"].clone()
    inplace = tg.tg_gated_bwd(t["dY"], t["Wd"], GU, act=act, outs={"dGU": GU})
    assert torch.equal(inplace["dGU"], got["dGU"])


@pytest.mark.parametrize("dtype", (BF, HF))
@pytest.mark.parametrize("T,f,d", [(5, 64, 64), (130, 264, 72), (260, 33, 40)])
def test_gated_off_16_bytes(T, f, d, dtype):
    t = gated_inputs(T, f, d, dtype, off16)
    outs = {"H": off16(torch.zeros(T, f, dtype=dtype, device="cuda")),
            "GU": off16(torch.zeros(T, 2 * f, dtype=dtype, device="cuda"))}
    check_all(tg.tg_gated_fwd(t["X"], t["W"], keep=True, outs=outs), *R.gated_fwd(t["X"], t["W"], "silu"), f"{T}x{f}x{d}")
    outs = {"H": outs["H"], "dGU": outs["GU"]}
    check_all(tg.tg_gated_bwd(t["dY"], t["Wd"], t["GU"], keep=True, outs=outs),
              *R.gated_bwd(t["dY"], t["Wd"], t["GU"], "silu"), f"{T}x{f}x{d} backward")


def test_gated_writes_nothing_else():
    """Rows behind the last and columns behind the widths' tiles stay as they were."""
    for T, f, d in ((130, 200, 64), (3, 33, 40)):
        t = gated_inputs(T, f, d, BF)
        H, GU = (torch.full((T + 70, n), 7.0, dtype=BF, device="cuda") for n in (f, 2 * f))
        tg.tg_gated_fwd(t["X"], t["W"], keep=True, outs={"H": H[:T], "GU": GU[:T]})
        assert (H[T:] == 7).all() and (GU[T:] == 7).all()
        H.fill_(7), GU.fill_(7)
        tg.tg_gated_bwd(t["dY"], t["Wd"], t["GU"], keep=True, outs={"H": H[:T], "dGU": GU[:T]})
        assert (H[T:] == 7).all() and (GU[T:] == 7).all()


@pytest.mark.parametrize("act", ACTS)
def test_gated_extremes(act):
    """The activations at the ends of the types, through an identity: values, no overflow in between, and what is not a
    number stays in its element."""
    n = 64
    for dtype in (BF, HF):
        top = torch.finfo(dtype).max
        x = torch.tensor([0.0, -0.0, 1e-3, -1e-3, 1.0, -1.0, 5.0, -5.0, 12.0, -12.0, 30.0, -30.0, 100.0, -100.0, 1e4, -1e4,
                          top, -top], device="cuda").to(dtype)
        G = torch.zeros(len(x), n, dtype=dtype, device="cuda")
        G[:, 0] = x
        GU = torch.cat((G, torch.ones_like(G)), 1)
        eye = torch.eye(n, dtype=dtype, device="cuda")
        ref, err = R.gated_bwd(torch.ones_like(G), eye, GU, act)
        check_all(tg.tg_gated_bwd(torch.ones_like(G), eye, GU, act=act, keep=True), ref, err, f"{act} {dtype}")
        W = torch.cat((eye, torch.zeros_like(eye)), 0)
        W[n, 1] = 1  # U = x's second column
        G[:, 1] = 1
        ref, err = R.gated_fwd(G, W, act)
        check_all(tg.tg_gated_fwd(G, W, act=act, keep=True), ref, err, f"{act} {dtype}")
    t = gated_inputs(40, 72, 64, BF)
    t["GU"][3, 5], t["GU"][4, 72 + 6] = math.nan, math.nan
    got = tg.tg_gated_bwd(t["dY"], t["Wd"], t["GU"], act=act, keep=True)
    bad = got["dGU"].isnan()
    assert bad[3, 72 + 5] and bad[4, 6] and int(bad.sum()) <= 3 and got["H"].isnan().sum() == 2


def test_gated_empty():
    e = lambda *s: torch.empty(*s, dtype=BF, device="cuda")  # noqa: E731
    assert tg.tg_gated_fwd(e(0, 64), e(16, 64), keep=True)["GU"].shape == (0, 16)
    assert tg.tg_gated_fwd(e(5, 64), e(0, 64))["H"].shape == (5, 0)
    got = tg.tg_gated_fwd(e(5, 0), e(40, 0), keep=True)  # an empty sum
    assert not got["H"].any() and not got["GU"].any()
    GU = randn((5, 40), 1.0, BF, "GU")
    got = tg.tg_gated_bwd(e(5, 0), e(0, 20), GU, keep=True)
    assert not got["dGU"].any()
    check_all({"H": got["H"]}, *R.gated_bwd(e(5, 0), e(0, 20), GU, "silu"), "empty sum")


# ------------------------------------------------------------- the update
def orth_check(got, G, coeffs, scale, eps, what):
    """In the Frobenius norm: the bound of the parts, and half a step of the result's type."""
    for i in range(G.shape[0]):
        ref, noise = R.orthogonalize(G[i], coeffs, scale, eps, got.dtype)
        size = float(torch.linalg.vector_norm(ref))
        off = float(torch.linalg.vector_norm(got[i].double() - ref))
        half = float(torch.linalg.vector_norm(R.half_step(ref.abs() + noise / math.sqrt(ref.numel()), got.dtype)))
        assert off <= noise + half, (what, i, off / max(size, 1e-300), noise, half)


ORTH_SIZES = [(1, 1, 1), (2, 1, 9), (3, 9, 1), (1, 8, 8), (2, 31, 33), (2, 65, 40), (1, 192, 576), (3, 576, 192),
              (2, 257, 256), (1, 300, 300), (2, 513, 130), (1, 130, 1001), (5, 64, 64), (1, 1003, 517), (1, 700, 1537), (2, 576, 600),
              (1, 640, 1100), (1, 1100, 640), (3, 384, 384)]


def gradient(batch, rows, cols, dtype, rank=8):
    left = randn((batch, rows, rank), 0.1, F32, "left") * 0.7 ** torch.arange(rank, device="cuda")
    return (left @ randn((batch, rank, cols), 1.0, F32, "right") + randn((batch, rows, cols), 0.02, F32, "noise")).to(dtype)


@pytest.mark.parametrize("batch,rows,cols", ORTH_SIZES)
def test_orthogonalize(batch, rows, cols):
    for dtype, out, scale in ((BF, BF, 1.0), (F32, HF, 0.3), (HF, BF, 2.0)):
        G = gradient(batch, rows, cols, dtype)
        got = tg.tg_orthogonalize(G, out_dtype=out, scale=scale)
        orth_check(got, G, [QUINTIC] * 5, scale, 1e-7, f"{batch}x{rows}x{cols} {dtype} {out}")


@pytest.mark.parametrize("rows,cols", [(300, 700), (577, 321)])
def test_orthogonalize_is_sharper_than_its_output(rows, cols):
    """The parts' noise is random, about 5e-5 of a result's size: rounding to fp16 (2^-11 at most, 0.42 of that in the
    mean square) stays the larger error.  For bf16 (2^-8) the last step's, 2e-4 to 4e-4, does the same."""
    G = gradient(1, rows, cols, F32)[0]
    got = tg.tg_orthogonalize(G)
    ref, _ = R.orthogonalize(G, [QUINTIC] * 5, 1.0, 1e-7, BF)
    assert float(torch.linalg.vector_norm(got.double() - ref) / torch.linalg.vector_norm(ref)) < 2.0 ** -9
    got = tg.tg_orthogonalize(G, out_dtype=HF)
    ref, _ = R.orthogonalize(G, [QUINTIC] * 5, 1.0, 1e-7, HF)
    assert float(torch.linalg.vector_norm(got.double() - ref) / torch.linalg.vector_norm(ref)) < 2.0 ** -11


def test_orthogonalize_steps_and_sizes_of_values():
    G = gradient(2, 70, 130, F32)
    cubic = [(2.0, -1.5, 0.5), (1.875, -1.25, 0.375), (1.5, -0.5, 0.0)]
    orth_check(tg.tg_orthogonalize(G, steps=1, scale=-1.5), G, [QUINTIC], -1.5, 1e-7, "one step")
    for by in (1e30, 1e-30, 1e18, 1e-18):
        orth_check(tg.tg_orthogonalize(G * by, eps=0.0), G * by, [QUINTIC] * 5, 1.0, 0.0, f"times {by}")
    orth_check(tg.tg_orthogonalize(G, eps=3.0), G, [QUINTIC] * 5, 1.0, 3.0, "a large eps")
    got = tg.tg_orthogonalize(G[0])
    assert torch.equal(got, tg.tg_orthogonalize(G)[0])
    H = G.to(BF)
    want = tg.tg_orthogonalize(H)
    assert torch.equal(tg.tg_orthogonalize(H, O=H), want)


def test_orthogonalize_zeros_and_what_is_not_finite():
    G = gradient(4, 40, 72, F32)
    want = tg.tg_orthogonalize(G)
    G[1] = 0
    G[2, 3, 4] = math.inf
    G[3, 0, 0] = math.nan
    got = tg.tg_orthogonalize(G)
    assert torch.equal(got[0], want[0]) and not got[1].any() and got[2].isnan().any() and got[3].isnan().all()
    assert tg.tg_orthogonalize(torch.empty(0, 4, 5, device="cuda")).shape == (0, 4, 5)
    assert tg.tg_orthogonalize(torch.empty(4, 0, dtype=HF, device="cuda")).dtype == HF


def test_orthogonalize_off_16_bytes():
    for rows, cols in ((40, 72), (33, 31)):
        G = off16(gradient(2, rows, cols, BF))
        O = off16(torch.zeros_like(G))
        assert torch.equal(tg.tg_orthogonalize(G, O=O), tg.tg_orthogonalize(G.clone()))


# ------------------------------------------------- streams, graphs, repeats
def calls():
    t, n = gated_inputs(200, 136, 96, BF), ln_inputs(200, 96, BF)
    G = gradient(2, 96, 136, F32)
    odd = gated_inputs(50, 33, 41, BF)  # staged copies in the workspace

    def run(**kw):
        f = tg.tg_layer_norm_fwd(n["X"], n["w"], b=n["b"], **kw)
        b = tg.tg_layer_norm_bwd(n["dY"], n["X"], n["w"], f["mean"], f["rstd"], dR=n["dR"], **kw)
        g = tg.tg_gated_fwd(t["X"], t["W"], keep=True, **kw)
        h = tg.tg_gated_bwd(t["dY"], t["Wd"], g["GU"], keep=True, **kw)
        o = tg.tg_gated_fwd(odd["X"], odd["W"], **kw)
        return [*f.values(), *b.values(), *g.values(), *h.values(), *o.values(), tg.tg_orthogonalize(G, **kw)]

    return run


def test_streams_and_graphs_give_the_same_bits():
    run = calls()
    want = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run()
        graphs.append((g, outs))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):  # both at once: their workspaces are their own
        for o in graphs[0][1] + graphs[1][1]:
            o.zero_()
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, outs in graphs:
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert tg.tg_stream_status() == 0


# ------------------------------------------------------- more than 2^31 elements
def test_layer_norm_beyond_32_bits():
    few = ln_inputs(1500, 576, BF)
    t = {k: v.repeat(2500, 1) if v.dim() == 2 else v for k, v in few.items()}
    assert t["X"].numel() > 2 ** 31
    got = tg.tg_layer_norm_fwd(t["X"], t["w"], b=t["b"])
    m, r = got["mean"], got["rstd"]
    check_all({k: v[-1500:] for k, v in got.items()}, *R.layer_norm_fwd(few["X"], few["w"], few["b"], 1e-5), "last rows")
    dX = tg.tg_layer_norm_bwd(t["dY"], t["X"], t["w"], m, r, dR=t["dR"], outs={"dX": got["Y"]})["dX"]
    check_all({"dX": dX[-1500:]}, *R.layer_norm_bwd(few["dY"], few["X"], few["w"], m[-1500:], r[-1500:], few["dR"]), "last rows")


def test_gated_beyond_32_bits():
    few = gated_inputs(380, 5760, 72, BF)
    t = {k: v.repeat(500, 1) if k in ("X", "dY", "GU") else v for k, v in few.items()}
    assert t["GU"].numel() > 2 ** 31
    got = tg.tg_gated_fwd(t["X"], t["W"], keep=True)
    check_all({k: v[-380:] for k, v in got.items()}, *R.gated_fwd(few["X"], few["W"], "silu"), "last rows")
    got = tg.tg_gated_bwd(t["dY"], t["Wd"], t["GU"], keep=True, outs={"dGU": got["GU"], "H": got["H"]})
    check_all({k: v[-380:] for k, v in got.items()}, *R.gated_bwd(few["dY"], few["Wd"], few["GU"], "silu"), "last rows")


def test_orthogonalize_beyond_32_bits():
    few = gradient(10, 576, 1000, BF)
    G = few.repeat(380, 1, 1)
    assert G.numel() > 2 ** 31
    want = tg.tg_orthogonalize(few)
    got = tg.tg_orthogonalize(G, O=G).view(380, 10, 576, 1000)
    for i in (0, 185, 379):
        assert torch.equal(got[i], want)
