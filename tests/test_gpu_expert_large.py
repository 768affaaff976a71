"""The expert-block operators on tensors of more than 2^31 elements: values far beyond the 32-bit range of an index,
checked at sampled rows against the 64-bit definitions."""
import os
import subprocess
import sys

import pytest
import torch

import expert_ref as R
import gemms_linear_layers_gb300 as tg

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ROWS = 400_000  # times 5,760 columns: 2.3e9 elements


def randn(shape, std, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=BF) * std


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def sampled(off, T):
    """A few rows of each group, the tensor's first and last."""
    o = [int(x) for x in off]
    return sorted({0, T - 1, *(r for a, b in zip(o, o[1:]) for r in (a, (a + b) // 2, b - 1))})


@pytest.mark.parametrize("op", ["fwd", "dgrad"])
def test_grouped_rows_beyond_32_bits(op):
    off = torch.tensor([0, 150_001, 150_001, 399_000, ROWS - 3], dtype=torch.int32)
    W = randn((4, 5760, 64) if op == "fwd" else (4, 64, 5760), 0.1, 1)
    A = randn((ROWS, 64), 1.0, 2)
    got = tg.tg_grouped_fwd(A, W, off.cuda()) if op == "fwd" else tg.tg_grouped_dgrad(A, W, off.cuda())
    assert got.numel() > 2 ** 31
    for r in sampled(off, ROWS):
        e = int(torch.searchsorted(off[1:], torch.tensor(r, dtype=torch.int32), right=True))
        if e == 4:
            assert (got[r] == 0).all()
            continue
        w = (W[e] if op == "fwd" else W[e].T).double()
        x = A[r].double()
        R.check(got[r], w @ x, R.PRODUCT * (w.abs() @ x.abs()), f"{op} row {r}")


def test_grouped_weight_gradient_beyond_32_bits():
    E, T, d = 34, 70, 8064  # 34 x 8,064 x 8,064 = 2.2e9
    off = (torch.arange(E + 1, dtype=torch.int32) * 2).clamp(max=T)
    dY, X = randn((T, d), 0.1, 3), randn((T, d), 1.0, 4)
    got = tg.tg_grouped_wgrad(dY, X, off.cuda())
    assert got.numel() > 2 ** 31
    for e in (0, 16, 33):
        a, b = int(off[e]), int(off[e + 1])
        for m in (0, 4000, d - 1):
            y, x = dY[a:b, m].double(), X[a:b].double()
            R.check(got[e, m], y @ x, R.PRODUCT * (y.abs() @ x.abs()), f"expert {e} row {m}")


def test_norms_beyond_32_bits():
    d = 5760
    B, H = randn((ROWS, d), 1.0, 5), randn((ROWS, d), 1.0, 6)
    w_post, w_pre = randn((d,), 1.0, 7), randn((d,), 1.0, 8)
    f = tg.tg_norm_residual_fwd(B, H, w_post, w_pre, res_scale=0.5)
    rows = torch.tensor([0, 1, 372_827, 372_828, ROWS - 1], device="cuda")  # 2^31 / 5,760 = 372,827.5
    ref = R.norm_fwd(B[rows], H[rows], w_post, w_pre, None, 0.5, 1e-6)
    for k, (v, e) in ref.items():
        R.check(f[k][rows], v, e, k)
    g = tg.tg_norm_residual_bwd(H, f["N"], B, f["H"], w_post, w_pre, f["rstd_b"], f["rstd_h"], res_scale=0.5)
    ref = R.norm_bwd(H[rows], f["N"][rows], B[rows], f["H"][rows], w_post, w_pre, f["rstd_b"][rows], f["rstd_h"][rows],
                     None, 0.5)
    for k in ("dB", "dH"):
        R.check(g[k][rows], *ref[k], k)


def test_clip_beyond_32_bits():
    n = 2 ** 31 + 12_345
    g = torch.zeros(n, dtype=BF, device="cuda")
    at = torch.tensor([0, 2 ** 31 - 1, 2 ** 31, n - 1], device="cuda")
    g[at] = torch.tensor([3.0, 4.0, 12.0, 84.0], dtype=BF, device="cuda")  # norm 85
    small = torch.full((1,), 132.0, device="cuda")  # with it 157
    norm = tg.tg_grad_clip([g, small], 15.7)
    assert float(norm) == pytest.approx(157.0, rel=1e-6)
    want = torch.tensor([0.3, 0.4, 1.2, 8.4], dtype=torch.float64, device="cuda")
    assert ((g[at].double() - want).abs() <= want * 2.0 ** -8).all() and float(small) == pytest.approx(13.2, rel=1e-6)
    assert int((g != 0).sum()) == 4


LONG = """
import torch
import gemms_linear_layers_gb300 as tg
E, d, T = 78, 8, 1 << 26
off = torch.full((E + 1,), T, dtype=torch.int32)
off[0], off[E - 1] = 0, T + 5  # the first expert: T rows; the last but one, which the same pair takes next: 5
off[E] = T + 5
dY, X = (torch.zeros(T + 5, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
g = torch.Generator(device="cuda")
g.manual_seed(9)
for t in (dY, X):  # whole numbers whose sums FP32 holds
    t[::16] = torch.randint(0, 2, t[::16].shape, generator=g, device="cuda").to(t.dtype)
    t[-5:] = 1
got = tg.tg_grouped_wgrad(dY, X, off.cuda(), out_dtype=torch.float32)
a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
a.record()
tg.tg_grouped_wgrad(dY, X, off.cuda(), dW=got)
b.record()
torch.cuda.synchronize()
assert tg.tg_stream_status() == 0
assert torch.equal(got[0].double(), dY[:T:16].double().T @ X[:T:16].double())
assert (got[E - 2] == 5).all() and (got[1:E - 2] == 0).all() and (got[E - 1] == 0).all()
assert a.elapsed_time(b) > 100, a.elapsed_time(b)  # longer than twice the bound
"""


def test_a_reduction_longer_than_the_bound_on_waits():
    """The bound on a wait is 50 ms here; the waits for one long unit, and for the slice after it, last longer."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", LONG], env={**os.environ, "TG_WAIT_TIMEOUT_MS": "50"}, cwd=root,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
