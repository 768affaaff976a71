"""The dense block of dense_step.py, end to end: its result and gradients against 64-bit autograd, its update against
the polynomial in 64 bits."""
import math

import pytest
import torch

import gemms_linear_layers_gb300 as tg
from gemms_linear_layers_gb300 import dense_step, inputs
import block_ref as R

pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)


def near(got, want, roundings, what):
    """2-norm of the difference; each rounding to fp16 moves a value by at most 2^-11 of itself."""
    off = (got.double() - want).norm() / want.norm()
    assert off <= roundings * 2.0 ** -11, (what, float(off))


@pytest.mark.parametrize("act", ("silu", "gelu"))
@pytest.mark.parametrize("T,hidden,ffn", [(300, 192, 320), (70, 72, 136)])
def test_block_gradients_match_autograd(T, hidden, ffn, act):
    dtype = torch.float16
    block = dense_step.DenseBlock(hidden, ffn, act, dtype=dtype)
    for k, s in (("w", 0.2), ("b", 0.1)):
        block.weights[k].add_(inputs.normal((hidden,), s, dtype, inputs.seed_for("dense", hidden, k)).cuda())
    X, dY = (inputs.normal((T, hidden), s, dtype, inputs.seed_for("dense", T, hidden, n)).cuda()
             for n, s in (("X", 1.0), ("dY", 0.1)))
    Y = block.forward(X)
    dX = block.backward(dY)

    w = {k: v.double().requires_grad_() for k, v in block.weights.items()}
    x = X.double().requires_grad_()
    n = torch.nn.functional.layer_norm(x, (hidden,), w["w"], w["b"], 1e-5)
    g, u = (n @ w["up"].T).split(ffn, 1)
    y = x + (R.act(act, g)[0] * u) @ w["down"].T
    (y * dY.double()).sum().backward()
    # roundings on the way: N, H, H W^T, Y forward; N, G and U backward, dGU, dN, the result (gradients of the
    # weights: N, G and U, H or dGU, the result)
    near(Y, y, 4, "Y")
    near(dX, x.grad, 8, "dX")
    for k in ("up", "down", "w", "b"):
        near(block.grads[k], w[k].grad, 8, k)

    before = {k: v.clone() for k, v in block.weights.items()}
    block.step(0.1, mu=0.5)
    for k in ("up", "down"):
        m = block.grads[k].float()
        for part, got in zip(m.split(ffn) if k == "up" else (m,),
                             block.updates[k].split(ffn) if k == "up" else (block.updates[k],)):
            scale = math.sqrt(max(1.0, part.shape[0] / part.shape[1]))
            ref, noise = R.orthogonalize(part, [QUINTIC] * 5, scale, 1e-7, dtype)
            off = torch.linalg.vector_norm(got.double() - ref)
            assert off <= noise + 2.0 ** -11 * torch.linalg.vector_norm(ref), (k, float(off), noise)
        assert torch.equal(block.weights[k], before[k].add(block.updates[k], alpha=-0.1))
    assert tg.tg_stream_status() == 0


def test_it_runs():
    losses = dense_step.main(["--steps", "3", "--tokens", "333", "--hidden", "200", "--ffn", "328", "--act", "gelu_tanh"])
    assert len(losses) == 3 and all(math.isfinite(x) for x in losses)
