"""The norms around a block where a team of threads takes many rows: the ring of rows in flight wraps, columns' sums
build up over rows, a row's scalars are loaded a row ahead.  Rows that start on 16 bytes and rows that do not, one and
several groups of columns a thread, every gate and stream type, all outputs against the 64-bit definitions."""
import pytest
import torch

import expert_ref as R
import gemms_linear_layers_gb300 as tg

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
GATES = ("none", "channel", "token", "full")
# at least three rows for some teams of each: the ring has two stages
SHAPES = [(20011, 100), (20000, 104), (13001, 573), (5001, 2300), (5000, 2304), (2501, 4099), (3000, 5760), (1200, 8191),
          (2000, 10240), (1200, 12291), (1500, 16384)]
SCALE, EPS = 0.75, 1e-6


def types_of(k):
    """16-bit values with a 16-bit and an FP32 stream, and FP32 throughout."""
    a, b = ((BF, HF), (HF, BF))[k % 2]
    return (a, a), (b, F32), (F32, F32)


class Case:
    def __init__(self, T, d, gate, dtype, res, off=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(T * 31 + d)

        def randn(shape, std, t, mean=0.0):
            v = (torch.randn(shape, generator=g, device="cuda") * std + mean).to(t)
            if off:  # the base moved by `off` elements
                room = torch.empty(v.numel() + off, dtype=t, device="cuda")
                v = room[off:].view(shape).copy_(v)
            return v

        shape = {"none": None, "channel": (d,), "token": (T, 1), "full": (T, d)}[gate]
        self.B, self.H = randn((T, d), 1.3, dtype), randn((T, d), 2.0, res)
        self.w_post, self.w_pre = randn((d,), 0.2, dtype, 1.0), randn((d,), 0.2, dtype, 1.0)
        self.gate = None if shape is None else randn(shape, 0.7, dtype)
        self.dHo, self.dN = randn((T, d), 0.1, res), randn((T, d), 0.1, dtype)
        self.rb = (self.B.double().square().mean(1) + EPS).rsqrt().float()
        self.rh = (self.H.double().square().mean(1) + EPS).rsqrt().float()

    def forward(self, H=None, outs=None):
        return tg.tg_norm_residual_fwd(self.B, self.H if H is None else H, self.w_post, self.w_pre, gate=self.gate,
                                       res_scale=SCALE, eps=EPS, outs=outs)

    def backward(self, dHo=None, dN=None, **kw):
        return tg.tg_norm_residual_bwd(self.dHo if dHo is None else dHo, self.dN if dN is None else dN, self.B, self.H,
                                       self.w_post, self.w_pre, self.rb, self.rh, gate=self.gate, res_scale=SCALE, **kw)

    def check_forward(self, what):
        got = self.forward()
        ref = R.norm_fwd(self.B, self.H, self.w_post, self.w_pre, self.gate, SCALE, EPS)
        for k, (v, e) in ref.items():
            R.check(got[k], v, e, f"{what} {k}")
        H = self.H.clone()  # over the stream itself: the same bits
        again = self.forward(H, {"H": H})
        assert again["H"] is H and all(torch.equal(again[k], got[k]) for k in got)

    def check_backward(self, what):
        T, d = self.B.shape
        got = self.backward(out_dtype=F32)
        ref = R.norm_bwd(self.dHo, self.dN, self.B, self.H, self.w_post, self.w_pre, self.rb, self.rh, self.gate, SCALE)
        # the definition's error scale counts T additions for every output: a row's sums have none of them, a column's
        # those of the rows of one multiprocessor, of its teams (15 at most), of a 32nd of the partials and of 32
        rows = 2 * (d / 32 + 10) + 30
        cols = rows + -(-T // (torch.cuda.get_device_properties(0).multi_processor_count - 7)) + 15 + 8 + 5
        assert set(got) == set(ref)
        for k, (v, e) in ref.items():
            col = k in ("dw_post", "dw_pre") or (k == "dgate" and v.dim() == 1)
            R.check(got[k], v, e * ((cols if col else rows) / (rows + T)), f"{what} {k}")
        a, b = self.dHo.clone(), self.dN.clone()  # over its own gradients: the same bits
        again = self.backward(a, b, out_dtype=F32, outs={"dH": a, "dB": b})
        assert again["dH"] is a and all(torch.equal(again[k], got[k]) for k in got)


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norms_of_many_rows(shape, gate):
    for dtype, res in types_of(SHAPES.index(shape) + GATES.index(gate)):
        c = Case(*shape, gate, dtype, res)
        c.check_forward(f"{gate} {dtype} {res}")
        c.check_backward(f"{gate} {dtype} {res}")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("shape", [(65, 576), (20011, 100), (5000, 2304), (1200, 5763), (900, 8200), (700, 16383)], ids=str)
def test_norms_off_16_bytes(shape, gate):
    """Every tensor starts one element past a multiple of 16 bytes: element by element, forward and backward."""
    for dtype, res in types_of(GATES.index(gate)):
        c = Case(*shape, gate, dtype, res, off=1)
        assert c.B.data_ptr() % 16 and c.dHo.data_ptr() % 16
        c.check_forward(f"{gate} {dtype} {res}")
        c.check_backward(f"{gate} {dtype} {res}")


# aligned rows of which two do not fit shared memory: straight into registers, in words of 16 bytes
PAST_THE_RING = [("none", BF, F32, 10240), ("token", HF, F32, 12288), ("none", BF, F32, 9224), ("none", F32, F32, 6920),
                 ("token", F32, F32, 12288), ("channel", F32, F32, 7176), ("channel", F32, F32, 8192), ("full", F32, F32, 5640),
                 ("full", F32, F32, 8192), ("none", BF, BF, 12296), ("full", BF, BF, 8200)]


@pytest.mark.parametrize("gate,dtype,res,d", PAST_THE_RING, ids=str)
@pytest.mark.parametrize("T", [3, 1000])
def test_wide_aligned_rows_are_taken_by_words(T, gate, dtype, res, d):
    c = Case(T, d, gate, dtype, res)
    c.check_backward(f"{gate} {dtype} {res}")
    assert "rows by vector" in tg.tg_last_call()
    c = Case(T, d, gate, dtype, res, off=1)
    c.check_backward(f"{gate} {dtype} {res} off 16 bytes")
    assert "rows by element" in tg.tg_last_call()


def test_how_rows_are_taken():
    for d, want in ((2304, "ring"), (2301, "shifted ring")):
        c = Case(40, d, "full", BF, BF)
        for call in (c.forward, c.backward):
            call()
            assert f"rows by {want} ok" in tg.tg_last_call()
