"""The expert block of expert_step.py, end to end: its results and gradients against 64-bit autograd of the same
routing, and a few clipped steps that lower the loss."""
import pytest
import torch

import gemms_linear_layers_gb300 as tg
from gemms_linear_layers_gb300 import expert_step, inputs

pytestmark = pytest.mark.gpu


def near(got, want, roundings, what):
    """2-norm of the difference; each rounding to fp16 moves a value by at most 2^-11 of itself."""
    off = (got.double() - want).norm() / want.norm()
    assert off <= roundings * 2.0 ** -11, (what, float(off))


@pytest.mark.parametrize("T,hidden,ffn,experts", [(300, 192, 320, 8), (64, 72, 136, 16)])
def test_block_gradients_match_autograd(T, hidden, ffn, experts):
    dtype = torch.float16
    block = expert_step.ExpertBlock(hidden, ffn, experts, dtype=dtype)
    draw = lambda name, std: inputs.normal((T, hidden), std, dtype, inputs.seed_for("step", T, hidden, name)).cuda()
    N, H, dH_out, dN_out = draw("N", 1.0), draw("H", 1.0), draw("dH", 0.1), draw("dN", 0.1)
    Ho, No = block.forward(N, H)
    dH, dN = block.backward(dH_out, dN_out)

    expert, order = block.saved[4], block.saved[3]
    route = torch.empty_like(expert)
    route[order] = expert
    w = {k: v.double().requires_grad_() for k, v in block.weights.items()}
    n, h = N.double().requires_grad_(), H.double().requires_grad_()
    p = torch.softmax(n @ w["router"].T, dim=1)
    gate = p.gather(1, route[:, None])
    a = torch.einsum("th,tfh->tf", n, w["up"][route])
    b = torch.einsum("tf,thf->th", torch.nn.functional.silu(a), w["down"][route])
    norm = lambda x: x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    ho = h + gate * norm(b) * w["w_post"]
    no = norm(ho) * w["w_pre"]
    ((ho * dH_out.double()).sum() + (no * dN_out.double()).sum()).backward()

    # roundings on the way: A, Z, B, gate, H' forward (their effect on a gradient of the same order); dB, dZ, dA,
    # dN twice, the result
    near(Ho, ho, 6, "H'")
    near(No, no, 7, "N'")
    near(dH, h.grad, 8, "dH")
    near(dN, n.grad, 14, "dN")
    for k in block.NAMES:
        near(block.grads[k], w[k].grad, 14, k)
    assert tg.tg_stream_status() == 0


def test_a_few_steps_lower_the_loss():
    losses = expert_step.main(["--steps", "6", "--tokens", "512"])
    assert all(torch.isfinite(torch.tensor(losses))) and losses[-1] < losses[0]
