"""The expert-block operators against their 64-bit definitions: products grouped by expert, the norms with gate and
residual scale, and the global gradient norm with clipping."""
import math
import threading

import pytest
import torch

import gemms_linear_layers_gb300 as tg
from gemms_linear_layers_gb300 import inputs
import expert_ref as R

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def randn(shape, std, dtype, tag):
    return inputs.normal(shape, std, dtype, inputs.seed_for("expert", *shape, str(dtype), tag)).cuda()


def offsets_of(sizes, lead=0):
    return torch.tensor([lead] + list(sizes), dtype=torch.int32).cumsum(0, dtype=torch.int32)


def grouped_inputs(sizes, lead, spare, d_in, d_out, dtype):
    off = offsets_of(sizes, lead)
    T = int(off[-1]) + spare
    E = len(sizes)
    return (randn((T, d_in), 1.0, dtype, "X"), randn((E, d_out, d_in), 0.05, dtype, "W"),
            randn((T, d_out), 0.1, dtype, "dY"), off)


OPS = ("fwd", "dgrad", "wgrad")


def grouped(op, X, W, dY, off, **kw):
    o = off.cuda()
    if op == "fwd":
        return tg.tg_grouped_fwd(X, W, o, **kw)
    if op == "dgrad":
        return tg.tg_grouped_dgrad(dY, W, o, **kw)
    return tg.tg_grouped_wgrad(dY, X, o, **kw)


def expect(op, X, W, dY, off):
    return R.grouped_fwd(X, W, off) if op == "fwd" else R.grouped_dgrad(dY, W, off) if op == "dgrad" \
        else R.grouped_wgrad(dY, X, off)


def check_grouped(op, got, X, W, dY, off, what):
    ref, S = expect(op, X, W, dY, off)
    R.check(got, ref, R.PRODUCT * S, what)


SIZES = [
    ([1], 0, 0),
    ([3, 0, 1], 0, 0),
    ([0, 0, 5, 0], 2, 3),
    ([15, 16, 17, 31, 33, 64, 65], 0, 1),
    ([130, 0, 257, 256], 7, 40),
    ([300, 1, 513], 0, 300),
]
WIDTHS = [(64, 64), (8, 16), (192, 72), (576, 264), (72, 520), (100, 52), (33, 7), (1, 1), (7, 300)]


@pytest.mark.parametrize("widths", WIDTHS, ids=str)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s[0])))
@pytest.mark.parametrize("op", OPS)
def test_grouped_products(op, sizes, widths):
    """Every op over ragged, empty and single-row groups, rows of no group before and after, widths below and
    beyond a tile and widths TMA cannot address; both 16-bit types, 16-bit and FP32 output."""
    n = len(sizes[0]) + widths[0]
    dtype, other = (BF, HF) if n % 2 else (HF, BF)
    d_in, d_out = widths
    X, W, dY, off = grouped_inputs(*sizes, d_in, d_out, dtype)
    check_grouped(op, grouped(op, X, W, dY, off), X, W, dY, off, f"{op} {dtype}")
    check_grouped(op, grouped(op, X.to(other), W.to(other), dY.to(other), off, out_dtype=F32), X.to(other), W.to(other),
                  dY.to(other), off, f"{op} {other} -> f32")
    torch.cuda.synchronize()
    assert tg.tg_stream_status() == 0


@pytest.mark.parametrize("op", OPS)
def test_grouped_rows_of_others_never_reach_a_result(op):
    """Infinities and NaN in one expert's rows and in rows of no expert leave the other experts' results as
    they were, bit for bit, and rows of no expert come out as zeros."""
    sizes, lead, spare = [13, 70, 0, 37, 100], 5, 9
    X, W, dY, off = grouped_inputs(sizes, lead, spare, 136, 200, BF)
    clean = grouped(op, X, W, dY, off)
    a, b = int(off[1]), int(off[2])
    for t in (X, dY):
        t[a:b:2], t[a + 1:b:2] = float("nan"), float("inf")
        t[:lead], t[int(off[-1]):] = float("nan"), float("-inf")
    got = grouped(op, X, W, dY, off)
    if op == "wgrad":
        for e in (0, 2, 3, 4):
            assert torch.equal(got[e], clean[e])
        assert (clean[2] == 0).all() and not torch.isfinite(got[1]).any()
    else:
        keep = torch.ones(X.shape[0], dtype=torch.bool)
        keep[a:b] = False
        assert torch.equal(got[keep.cuda()], clean[keep.cuda()])
        assert (got[:lead] == 0).all() and (got[int(off[-1]):] == 0).all() and not torch.isfinite(got[a:b]).any()


@pytest.mark.parametrize("op", OPS)
def test_grouped_many_experts(op):
    """More experts than one launch takes, most of them with few rows or none."""
    sizes = [(k * 7) % 5 for k in range(600)]
    X, W, dY, off = grouped_inputs(sizes, 3, 2, 40, 24, BF)
    check_grouped(op, grouped(op, X, W, dY, off), X, W, dY, off, op)


@pytest.mark.parametrize("op", OPS)
def test_grouped_empty_sizes(op):
    X, W, dY, off = grouped_inputs([0, 0], 0, 0, 16, 24, BF)
    got = grouped(op, X, W, dY, off)
    assert (got == 0).all() and got.numel() == (2 * 24 * 16 if op == "wgrad" else 0)
    X, W, dY, off = grouped_inputs([], 0, 6, 16, 24, BF)  # no expert at all
    got = grouped(op, X, W, dY, off)
    assert (got == 0).all() and got.numel() == {"fwd": 6 * 24, "dgrad": 6 * 16, "wgrad": 0}[op]
    if op != "wgrad":  # an empty reduction
        X, W, dY, off = grouped_inputs([4, 2], 0, 0, 0 if op == "fwd" else 16, 0 if op == "dgrad" else 24, BF)
        assert (grouped(op, X, W, dY, off) == 0).all()


@pytest.mark.parametrize("op", OPS)
def test_grouped_output_type_follows_a_given_output(op):
    X, W, dY, off = grouped_inputs([9, 30], 0, 1, 64, 40, BF)
    want = grouped(op, X, W, dY, off, out_dtype=F32)
    got = grouped(op, X, W, dY, off, **{{"fwd": "Y", "dgrad": "dX", "wgrad": "dW"}[op]: torch.empty_like(want)})
    assert got.dtype == F32 and torch.equal(got, want)


@pytest.mark.parametrize("op", OPS)
def test_grouped_unaligned_bases(op):
    """Operands and output that start in the middle of a 16-byte word."""
    X, W, dY, off = grouped_inputs([37, 0, 90], 0, 3, 64, 72, HF)

    def shifted(t):
        u = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return u.copy_(t)

    Xs, Ws, dYs = shifted(X), shifted(W), shifted(dY)
    aligned = grouped(op, X, W, dY, off)
    out = shifted(torch.zeros_like(aligned))
    got = grouped(op, Xs, Ws, dYs, off, **{{"fwd": "Y", "dgrad": "dX", "wgrad": "dW"}[op]: out})
    assert got is out and torch.equal(got, aligned)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("bad", [[-5, 3, 2, 90], [10, 1 << 30, 40, 20], [0, 0, -2147483648, 2147483647]])
def test_grouped_offsets_that_break_the_rules_address_nothing_outside(op, bad):
    """Offsets below zero, above T or decreasing: the neighbouring memory of the output stays as it was."""
    X, W, dY, _ = grouped_inputs([20, 20, 20], 0, 0, 48, 40, BF)
    shape = {"fwd": (60, 40), "dgrad": (60, 48), "wgrad": (3, 40, 48)}[op]
    n = math.prod(shape)
    room = torch.full((n + 8192,), 7.0, dtype=BF, device="cuda")
    out = room[4096:4096 + n].view(shape)
    off = torch.tensor(bad, dtype=torch.int32)
    grouped(op, X, W, dY, off, **{{"fwd": "Y", "dgrad": "dX", "wgrad": "dW"}[op]: out})
    torch.cuda.synchronize()
    assert (room[:4096] == 7).all() and (room[4096 + n:] == 7).all()
    assert tg.tg_stream_status() == 0


@pytest.mark.parametrize("op", OPS)
def test_grouped_layer_sizes(op):
    """2B-class widths at 1,024 tokens over 8 uneven experts."""
    X, W, dY, off = grouped_inputs([400, 250, 130, 100, 64, 40, 39, 1], 0, 0, 2304, 5760, BF)
    got = grouped(op, X, W, dY, off)
    check_grouped(op, got, X, W, dY, off, op)
    for _ in range(3):
        assert torch.equal(grouped(op, X, W, dY, off), got)


@pytest.mark.parametrize("case", [
    ("fwd", [5], 0, 0, 2304, 300), ("fwd", [0, 3, 40], 2, 5, 2312, 37), ("dgrad", [60, 1], 1, 0, 72, 3000),
    ("wgrad", [3000, 17, 0], 3, 4, 64, 72), ("wgrad", [7000, 17, 0], 3, 4, 64, 72), ("wgrad", [4111], 0, 0, 33, 101), ("wgrad", [2600, 2500], 0, 9, 264, 300)],
    ids=str)
def test_grouped_long_reductions_of_few_tiles(case):
    """Reductions that are cut into ranges and added afterwards: rows of no expert, empty experts, odd widths and
    lengths, both output types; the same bits each time."""
    op, sizes, lead, spare, d_in, d_out = case
    X, W, dY, off = grouped_inputs(sizes, lead, spare, d_in, d_out, BF)
    # an even share of 3,024 rows over three experts is too short to be cut
    cut = tg.tg_workspace_size({"fwd": 13, "dgrad": 14, "wgrad": 15}[op], X.shape[0], len(sizes), d_out, d_in, BF, BF) > 0
    assert cut == (sizes != [3000, 17, 0])
    for out in (BF, F32):
        got = grouped(op, X, W, dY, off, out_dtype=out)
        check_grouped(op, got, X, W, dY, off, f"{case} {out}")
        assert torch.equal(grouped(op, X, W, dY, off, out_dtype=out), got)


def test_grouped_workspace_too_small():
    X, W, dY, off = grouped_inputs([5], 0, 0, 2304, 300, BF)
    o, Y = off.cuda(), torch.empty(5, 300, dtype=BF, device="cuda")
    from gemms_linear_layers_gb300 import _binding as B
    need = tg.tg_workspace_size(B.TG_OP_GROUPED_FWD, 5, 1, 300, 2304, BF, BF)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    call = lambda p, n: B.lib().tg_grouped_fwd(X.data_ptr(), W.data_ptr(), o.data_ptr(), Y.data_ptr(), 5, 1, 300, 2304,
                                               B.TG_BF16, B.TG_BF16, p, n, torch.cuda.current_stream().cuda_stream)
    assert call(0, 0) == 4 and call(ws.data_ptr(), need - 1) == 4 and call(ws.data_ptr(), need) == 0
    check_grouped("fwd", Y, X, W, dY, off, "given workspace")


def test_grouped_gradients_match_differences():
    """<G, Y> is linear in X and in W: its change along a direction is <dX, direction>, <dW, direction>."""
    X, W, G, off = grouped_inputs([20, 0, 33, 7], 1, 2, 64, 48, BF)
    dX = tg.tg_grouped_dgrad(G, W, off.cuda(), out_dtype=F32).double()
    dW = tg.tg_grouped_wgrad(G, X, off.cuda(), out_dtype=F32).double()
    sizes = {"X": R.grouped_dgrad(G, W, off)[1], "W": R.grouped_wgrad(G, X, off)[1]}
    for name, t, grad in (("X", X, dX), ("W", W, dW)):
        D = randn(tuple(t.shape), 1.0, F32, "direction").double()
        at = lambda s: (G.double() * R.grouped_fwd(*((X.double() + s * D, W) if name == "X" else (X, W.double() + s * D)), off)[0]).sum()
        diff = (at(0.5) - at(-0.5)).item()
        scale = (sizes[name] * D.abs()).sum().item()
        assert abs((grad * D).sum().item() - diff) <= R.PRODUCT * scale


@pytest.mark.parametrize("op", OPS)
def test_grouped_on_another_stream_and_in_a_graph(op):
    """A call captured once follows new offsets and new values; a call on a side stream gives the same bits."""
    X, W, dY, off = grouped_inputs([50, 3, 0, 77], 0, 30, 96, 160, BF)
    dev = off.cuda()
    call = lambda **kw: (tg.tg_grouped_fwd(X, W, dev, **kw) if op == "fwd" else tg.tg_grouped_dgrad(dY, W, dev, **kw)
                         if op == "dgrad" else tg.tg_grouped_wgrad(dY, X, dev, **kw))
    eager = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(eager)
    call(**{{"fwd": "Y", "dgrad": "dX", "wgrad": "dW"}[op]: other}, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other, eager)
    out = torch.empty_like(eager)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(**{{"fwd": "Y", "dgrad": "dX", "wgrad": "dW"}[op]: out})
    new = offsets_of([0, 80, 70, 10])
    dev.copy_(new)
    g.replay()
    torch.cuda.synchronize()
    check_grouped(op, out, X, W, dY, new, op)
    assert torch.equal(out, call())


def test_grouped_refuses():
    X, W, dY, off = grouped_inputs([4, 4], 0, 0, 16, 24, BF)
    o = off.cuda()
    for bad in (off, o.long(), o[:2], torch.stack([o, o], 1)[:, 0]):
        with pytest.raises(ValueError):
            tg.tg_grouped_fwd(X, W, bad)
    with pytest.raises(ValueError):
        tg.tg_grouped_fwd(X, W.transpose(1, 2), o)
    with pytest.raises(ValueError):
        tg.tg_grouped_fwd(X, W.to(HF), o)
    with pytest.raises(ValueError):
        tg.tg_grouped_dgrad(dY, W, o, dX=torch.empty_like(dY))
    with pytest.raises(ValueError):
        tg.tg_grouped_wgrad(dY[:4], X, o)
    with pytest.raises(tg.TGError) as e:
        tg.tg_grouped_fwd(X.float(), W.float(), o)
    assert e.value.status == 2
    with pytest.raises(tg.TGError) as e:
        tg.tg_grouped_fwd(X, W, o, out_dtype=HF)
    assert e.value.status == 2


# ------------------------------------------------------------------- norms
GATES = ("none", "channel", "token", "full")


def norm_inputs(T, d, gate, dtype, res, tag=""):
    shape = {"none": None, "channel": (d,), "token": (T, 1), "full": (T, d)}[gate]
    g = None if shape is None else randn(shape, 0.7, dtype, "gate" + tag)
    return {"B": randn((T, d), 1.3, dtype, "B" + tag), "H": randn((T, d), 2.0, res, "H" + tag),
            "w_post": (1 + randn((d,), 0.2, F32, "wp" + tag)).to(dtype), "w_pre": (1 + randn((d,), 0.2, F32, "wq" + tag)).to(dtype),
            "gate": g}


def norm_fwd(i, scale, eps=1e-6, **kw):
    return tg.tg_norm_residual_fwd(i["B"], i["H"], i["w_post"], i["w_pre"], gate=i["gate"], res_scale=scale, eps=eps, **kw)


def check_fwd(got, i, scale, eps, what):
    ref = R.norm_fwd(i["B"], i["H"], i["w_post"], i["w_pre"], i["gate"], scale, eps)
    for k, (v, e) in ref.items():
        R.check(got[k], v, e, f"{what} {k}")


def bwd_case(T, d, gate, dtype, res, scale, out=None, **kw):
    i = norm_inputs(T, d, gate, dtype, res)
    dHo, dN = randn((T, d), 0.1, res, "dHo"), randn((T, d), 0.1, dtype, "dN")
    rb = (i["B"].double().square().mean(1) + 1e-6).rsqrt().float()
    rh = (i["H"].double().square().mean(1) + 1e-6).rsqrt().float()
    got = tg.tg_norm_residual_bwd(dHo, dN, i["B"], i["H"], i["w_post"], i["w_pre"], rb, rh, gate=i["gate"],
                                  res_scale=scale, out_dtype=out, **kw)
    ref = R.norm_bwd(dHo, dN, i["B"], i["H"], i["w_post"], i["w_pre"], rb, rh, i["gate"], scale)
    return got, ref


ROWS = [(1, 1), (1, 8), (3, 7), (2, 64), (37, 100), (5, 573), (130, 576), (700, 72), (9, 2304), (4, 4096), (3, 4104),
        (3, 5760), (2, 8191), (2, 8200), (2, 16384)]
TYPES = [(BF, BF), (BF, F32), (HF, HF), (HF, F32), (F32, F32)]


@pytest.mark.parametrize("shape", ROWS, ids=str)
@pytest.mark.parametrize("gate", GATES)
def test_norm_forward(shape, gate):
    T, d = shape
    k = GATES.index(gate) + ROWS.index(shape)
    for dtype, res in (TYPES[k % 5], TYPES[(k + 2) % 5]):
        i = norm_inputs(T, d, gate, dtype, res)
        check_fwd(norm_fwd(i, 0.75), i, 0.75, 1e-6, f"{gate} {dtype} {res}")


@pytest.mark.parametrize("shape", ROWS, ids=str)
@pytest.mark.parametrize("gate", GATES)
def test_norm_backward(shape, gate):
    T, d = shape
    k = GATES.index(gate) + ROWS.index(shape)
    for (dtype, res), out in ((TYPES[k % 5], None), (TYPES[(k + 2) % 5], F32)):
        got, ref = bwd_case(T, d, gate, dtype, res, 0.75, out)
        assert set(got) == set(ref)
        for n, (v, e) in ref.items():
            R.check(got[n], v, e, f"{gate} {dtype} {res} {n}")


@pytest.mark.parametrize("gate", GATES)
def test_norm_gradients_match_differences(gate):
    """The backward's directional derivative against central differences of the 64-bit forward."""
    T, d, scale, eps = 6, 40, 0.8, 1e-6
    i = norm_inputs(T, d, gate, F32, F32)
    f = norm_fwd(i, scale, eps)
    dHo, dN = randn((T, d), 1.0, F32, "dHo"), randn((T, d), 1.0, F32, "dN")
    got = tg.tg_norm_residual_bwd(dHo, dN, i["B"], f["H"], i["w_post"], i["w_pre"], f["rstd_b"], f["rstd_h"],
                                  gate=i["gate"], res_scale=scale)
    x = {k: v.double() for k, v in i.items() if v is not None}

    def value(y):
        r = R.norm_fwd(y["B"], y["H"], y["w_post"], y["w_pre"], y.get("gate"), scale, eps)
        return ((dHo.double() * r["H"][0]).sum() + (dN.double() * r["N"][0]).sum()).item()

    for k in x:
        D = randn(tuple(x[k].shape), 1.0, F32, "dir" + k).double()
        h = 1e-4
        diff = (value({**x, k: x[k] + h * D}) - value({**x, k: x[k] - h * D})) / (2 * h)
        grad = got["dgate" if k == "gate" else k if k[0] == "d" else "d" + k].double()
        scale_of = (grad.abs() * D.abs()).sum().item()
        # FP32 arithmetic (some 100 roundings) and the difference's own h^2 term
        assert abs((grad * D).sum().item() - diff) <= (200 * R.U + 1e-6) * scale_of + 1e-6


def test_norm_rows_of_zeros_and_large_values():
    i = norm_inputs(4, 256, "none", BF, BF)
    i["B"][1] = 0
    i["H"][2], i["B"][2] = 0, 0
    i["B"][3] *= 1e15
    got = norm_fwd(i, 1.0)
    check_fwd(got, i, 1.0, 1e-6, "zeros")
    assert (got["H"][2] == 0).all() and (got["N"][2] == 0).all() and float(got["rstd_h"][2]) == pytest.approx(1000.0, rel=1e-6)
    i["B"][0, 3] = float("nan")  # stays in its row
    again = norm_fwd(i, 1.0)
    assert torch.isnan(again["N"][0]).all() and torch.equal(again["N"][1:], got["N"][1:])


def test_norm_in_place_streams_graphs_and_unaligned():
    i = norm_inputs(65, 576, "full", BF, F32)
    want = norm_fwd(i, 0.5)
    H = i["H"].clone()
    got = norm_fwd({**i, "H": H}, 0.5, outs={"H": H})
    assert got["H"] is H and all(torch.equal(got[k], want[k]) for k in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = norm_fwd(i, 0.5, outs={k: torch.empty_like(v) for k, v in want.items()}, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)

    def shifted(t):
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)

    got = norm_fwd({k: shifted(v) for k, v in i.items()}, 0.5)
    assert all(torch.equal(got[k], want[k]) for k in want)
    # backward: in place over its gradients, captured, twice the same bits
    dHo, dN = randn((65, 576), 0.1, F32, "dHo"), randn((65, 576), 0.1, BF, "dN")
    call = lambda a, b, **kw: tg.tg_norm_residual_bwd(a, b, i["B"], want["H"], i["w_post"], i["w_pre"], want["rstd_b"],
                                                      want["rstd_h"], gate=i["gate"], res_scale=0.5, **kw)
    eager = call(dHo, dN)
    a, b = dHo.clone(), dN.clone()
    g = torch.cuda.CUDAGraph()
    outs = {k: torch.empty_like(v) for k, v in eager.items()}
    with torch.cuda.graph(g):
        call(a, b, outs=outs)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(outs[k], eager[k]) for k in eager)
    got = call(a, b, outs={"dH": a, "dB": b})
    assert got["dH"] is a and all(torch.equal(got[k], eager[k]) for k in eager)


def test_norm_empty_and_refusals():
    i = norm_inputs(0, 64, "channel", BF, BF)
    r = norm_fwd(i, 1.0)
    assert r["N"].shape == (0, 64)
    e = torch.empty(0, device="cuda")
    g = tg.tg_norm_residual_bwd(i["H"], i["B"], i["B"], i["H"], i["w_post"], i["w_pre"], e, e, gate=i["gate"])
    assert (g["dw_post"] == 0).all() and (g["dw_pre"] == 0).all() and (g["dgate"] == 0).all()
    i = norm_inputs(4, 64, "none", BF, BF)
    with pytest.raises(ValueError):
        norm_fwd({**i, "H": i["H"].half()}, 1.0)
    with pytest.raises(ValueError):
        norm_fwd({**i, "w_pre": i["w_pre"].float()}, 1.0)
    with pytest.raises(ValueError):
        norm_fwd({**i, "gate": i["w_pre"][:4]}, 1.0)  # one value a row is [T, 1]
    with pytest.raises(ValueError):
        norm_fwd({**i, "B": i["B"].t()}, 1.0)
    for kw in ({"scale": float("nan")}, {"scale": 1.0, "eps": -1.0}, {"scale": 1.0, "eps": float("inf")}):
        with pytest.raises(tg.TGError) as err:
            norm_fwd(i, **kw)
        assert err.value.status == 1
    wide = norm_inputs(1, 16385, "none", BF, BF)
    with pytest.raises(tg.TGError) as err:
        norm_fwd(wide, 1.0)
    assert err.value.status == 1


# -------------------------------------------------------------------- clipping
# FP32 groups of at most 32 squares (33 roundings, halved by the root), the factor and the product
CLIP = 24 * R.U


def check_clip(grads, max_norm, got_norm, got):
    norm, c, ref = R.clip(grads, max_norm)
    assert abs(float(got_norm) - norm) <= CLIP * norm, (float(got_norm), norm)
    for k, (g, r) in enumerate(zip(got, ref)):
        R.check(g, r, CLIP * r.abs() + 2.0 ** -149, f"tensor {k}")


CLIP_SIZES = [[1], [0, 5, 0], [7, 8, 9, 4096, 8192, 8193, 16384, 16385], [100003, 1, 300000], [3] * 70, [17] * 700]


@pytest.mark.parametrize("sizes", CLIP_SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip(sizes, max_norm):
    types = (BF, F32, HF)
    grads = [randn((n,), 0.5, types[k % 3], f"g{k}") for k, n in enumerate(sizes)]
    src = [g.clone() for g in grads]
    norm = tg.tg_grad_norm(grads)
    outs = [torch.empty_like(g) for g in grads]
    n2 = tg.tg_grad_clip(grads, max_norm, outs=outs)
    assert torch.equal(norm, n2) and all(torch.equal(a, b) for a, b in zip(grads, src))
    check_clip(src, max_norm, norm, outs)
    n3 = tg.tg_grad_clip(grads, max_norm)
    assert torch.equal(n3, norm) and all(torch.equal(a, b) for a, b in zip(grads, outs))


@pytest.mark.parametrize("off", [1, 2, 3, 7])
def test_clip_any_alignment(off):
    """Tensors that start and end anywhere in a 16-byte word; neighbours stay as they were."""
    grads, rooms = [], []
    for k, t in enumerate((BF, HF, F32)):
        room = torch.full((5000,), 3.0, dtype=t, device="cuda")
        g = room[off:off + 4099 + k]
        g.copy_(randn((g.numel(),), 1.0, t, f"a{k}"))
        grads.append(g)
        rooms.append(room)
    src = [g.clone() for g in grads]
    outs = [torch.empty(g.numel() + 5, dtype=g.dtype, device="cuda")[5:] for g in grads]
    norm = tg.tg_grad_clip(grads, 2.0, outs=outs)
    check_clip(src, 2.0, norm, outs)
    tg.tg_grad_clip(grads, 2.0)
    for k, (g, room) in enumerate(zip(grads, rooms)):
        assert torch.equal(g, outs[k]) and (room[:off] == 3).all() and (room[off + g.numel():] == 3).all()


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e25, 3e38])
def test_clip_magnitudes_whose_square_leaves_fp32(size):
    grads = [randn((5000,), 1.0, F32, "m").clamp(-1, 1) * size, torch.zeros(100, device="cuda"),
             (randn((300,), 1.0, F32, "n").clamp(-1, 1) * size).to(BF)]
    outs = [torch.empty_like(g) for g in grads]
    max_norm = 1e-28 if size < 1 else 1.0
    norm, c, ref = R.clip(grads, max_norm)
    got = tg.tg_grad_clip(grads, max_norm, outs=outs)
    if norm < 3.4e38:
        assert abs(float(got) - norm) <= CLIP * norm + 2.0 ** -149
    else:
        assert float(got) == float("inf")  # the FP32 norm; the factor comes from the FP64 one
    for g, r in zip(outs, ref):
        R.check(g, r, CLIP * r.abs() + abs(c < 2.0 ** -126) * size * 2.0 ** -149 + 2.0 ** -149, "scaled")


def test_clip_not_finite():
    g = [randn((100,), 1.0, F32, "a"), randn((50,), 1.0, BF, "b")]
    g[0][3] = float("inf")
    outs = [torch.empty_like(t) for t in g]
    assert float(tg.tg_grad_clip(g, 1.0, outs=outs)) == float("inf")
    assert math.isnan(float(outs[0][3])) and (outs[1] == 0).all() and int((outs[0] == 0).sum()) == 99
    g[1][7] = float("nan")
    assert math.isnan(float(tg.tg_grad_clip(g, 1.0, outs=outs)))
    assert all(torch.isnan(t).all() for t in outs)


def test_clip_edges_graph_and_refusals():
    z = [torch.zeros(1000, device="cuda")]
    assert float(tg.tg_grad_clip(z, 1.0)) == 0.0 and (z[0] == 0).all()
    assert float(tg.tg_grad_norm([])) == 0.0 and float(tg.tg_grad_clip([], 1.0)) == 0.0
    g = [randn((333,), 1.0, BF, "e")]
    tg.tg_grad_clip(g, 0.0)
    assert (g[0] == 0).all()
    src = [randn((40000,), 1.0, t, "g" + str(t)) for t in (BF, F32)]
    work = tg.tg_tensor_list([s.clone() for s in src])
    eager = [s.clone() for s in src]
    n0 = tg.tg_grad_clip(eager, 1.0)
    norm = torch.empty(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tg.tg_grad_clip(work, 1.0, norm=norm)
    for w, s in zip(work, src):
        w.copy_(s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(norm, n0) and all(torch.equal(a, b) for a, b in zip(work, eager))
    inf = [s.clone() for s in src]
    tg.tg_grad_clip(inf, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(inf, src))
    with pytest.raises(ValueError):
        tg.tg_grad_clip([src[0].cpu()], 1.0)
    with pytest.raises(ValueError):
        tg.tg_grad_clip([src[0].long()], 1.0)
    with pytest.raises(ValueError):
        tg.tg_grad_clip([src[0].view(200, 200).t()], 1.0)
    with pytest.raises(ValueError):
        tg.tg_grad_clip(src, 1.0, outs=[src[0], src[1].half()])
    for bad in (-1.0, float("nan")):
        with pytest.raises(tg.TGError) as e:
            tg.tg_grad_clip(src, bad)
        assert e.value.status == 1


def test_workspaces_kept_by_the_binding():
    """Calls of all sizes in a row on one stream share its workspace; calls on two torch streams, and a graph
    captured in between, have others: every result is that of the call alone."""
    cases = [bwd_case(T, d, "channel", BF, BF, 0.75) for T, d in ((40, 576), (700, 4096), (3, 72))]
    for got, ref in cases:
        for n, (v, e) in ref.items():
            R.check(got[n], v, e, n)
    i = norm_inputs(200, 2304, "none", BF, BF)
    rb, rh = (torch.ones(200, device="cuda") for _ in range(2))
    call = lambda outs=None: tg.tg_norm_residual_bwd(i["H"], i["B"], i["B"], i["H"], i["w_post"], i["w_pre"], rb, rh,
                                                     outs=outs)
    want = call()
    outs = {k: torch.empty_like(v) for k, v in want.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(call())
        graph.replay()
    bwd_case(900, 4096, "channel", BF, F32, 1.0)  # a larger workspace on the current stream
    graph.replay()
    torch.cuda.synchronize()
    for g in got + [outs]:
        assert all(torch.equal(g[k], want[k]) for k in want)


def test_threads_on_one_stream():
    """Host threads that call on one stream at once, with workspaces that grow on the way: every result is that of
    the call alone, bit for bit."""
    def clip(k, sizes):
        grads = [randn((n,), 0.5, F32, f"{k}{n}") for n in sizes]
        return lambda: (lambda outs: [tg.tg_grad_clip(grads, 0.1, outs=outs), *outs])([torch.empty_like(g) for g in grads])

    def norm(T, d, tag):
        i = norm_inputs(T, d, "channel", BF, BF, tag)
        rb, rh = torch.ones(T, device="cuda"), torch.full((T,), 0.5, device="cuda")
        return lambda: list(tg.tg_norm_residual_bwd(i["H"], i["B"], i["B"], i["H"], i["w_post"], i["w_pre"], rb, rh,
                                                    gate=i["gate"]).values())

    def product(op, sizes, d_in, d_out):
        X, W, dY, off = grouped_inputs(sizes, 0, 0, d_in, d_out, BF)
        o = off.cuda()
        return lambda: [tg.tg_grouped_wgrad(dY, X, o) if op == "wgrad" else tg.tg_grouped_fwd(X, W, o)]

    jobs = [[norm(40, 72, "a"), clip("a", (5000, 301)), product("wgrad", [4096], 72, 64), norm(300, 576, "b"),
             product("fwd", [9, 30], 33, 101)],
            [norm(41, 80, "c"), clip("b", (70000, 9)), product("wgrad", [5000], 576, 264), norm(700, 4096, "d"),
             product("fwd", [70, 2], 101, 33)]]
    want = [[f() for f in fs] for fs in jobs]
    torch.cuda.synchronize()
    got, failed, gate = [[], []], [], threading.Barrier(2)

    def work(k):
        try:
            gate.wait()
            for _ in range(60):
                got[k].append([f() for f in jobs[k]])
        except Exception as e:  # shown below: an exception in a thread is not the test's
            failed.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for k in range(2):
        for run in got[k]:
            for a, b in zip(run, want[k]):
                assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_memory_of_a_call_on_a_given_stream():
    """A call on a stream of the caller's, which does not wait for the current one, allocates nothing that work
    queued on the current stream still reads."""
    i = norm_inputs(300, 4096, "channel", BF, BF)
    rb, rh = (torch.ones(300, device="cuda") for _ in range(2))
    call = lambda **kw: tg.tg_norm_residual_bwd(i["H"], i["B"], i["B"], i["H"], i["w_post"], i["w_pre"], rb, rh,
                                                gate=i["gate"], **kw)
    want = call()
    need = tg.tg_workspace_size(17, 300, 4096, 0, 0, BF, BF)
    side, big = torch.cuda.Stream(), torch.ones(8192, 8192, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    read = [torch.full((n,), 3, dtype=torch.uint8, device="cuda") for n in (need, want["dB"].numel() * 2, 8192, 1 << 22)]
    torch.cuda.synchronize()
    for _ in range(20):
        big @ big
    kept = [x + 1 for x in read]  # read when the products are done; freed now
    del read
    got = call(stream=side)
    torch.cuda.synchronize()
    assert all((k == 4).all() for k in kept)
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
def test_clip_adds_each_group_of_squares_in_64_bits(dtype):
    """Groups of at most 32 squares in FP32, 64 bits beyond.  The groups here are exact, 4,096^2 and 1 by turns, so
    the norm is the correctly rounded root; were two groups joined in FP32, the ones would vanish beside 2^24 and the
    root would fall below the middle of two FP32 values."""
    words = torch.zeros(4096, 16 // dtype.itemsize, dtype=dtype, device="cuda")  # 64 KB, 16 bytes a row
    words[:512, 0], words[512:1024, 0] = 4096.0, 1.0
    total = 512 * (4096 ** 2 + 1) + 14 ** 2
    want = torch.tensor(math.sqrt(total), dtype=F32)
    assert want > torch.tensor(math.sqrt(total - 512), dtype=F32)
    assert float(tg.tg_grad_norm([words, torch.full((1,), 14.0, device="cuda")])) == float(want)


def test_a_captured_call_on_a_forked_stream_allocates_for_the_graph():
    """A call with stream= inside a capture, on a stream forked from the captured one: outputs and workspace are the
    graph's, and replays give the bits of the eager call."""
    i = norm_inputs(300, 576, "channel", BF, BF)
    rb, rh = (torch.ones(300, device="cuda") for _ in range(2))
    call = lambda **kw: tg.tg_norm_residual_bwd(i["H"], i["B"], i["B"], i["H"], i["w_post"], i["w_pre"], rb, rh,
                                                gate=i["gate"], **kw)
    want = call()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = call(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        for t in got.values():
            t.zero_()
        torch.cuda.empty_cache()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
