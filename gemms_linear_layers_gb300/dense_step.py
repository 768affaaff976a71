"""A training step of a dense feed-forward block on the library's entry points.

The block, for a residual stream X [T, hidden]:
  norm      N = layer_norm(X; w, b)                            tg_layer_norm_fwd
  gated     [G U] = N W_up^T, H = act(G) U, W_up [2 ffn, hidden]   tg_gated_fwd
  down      Y = X + H W_down^T                                 tg_gemm_fwd
Backward: tg_gated_bwd goes through the down projection and the gate and gives H
again (only G and U are kept), tg_gemm_dgrad and tg_gemm_wgrad do the projections,
tg_layer_norm_bwd adds the residual stream's gradient.  The matrices take
orthogonalised steps from their momentum (tg_orthogonalize; the gate and the up
projection each by itself), the norm's vectors plain ones.

``python -m gemms_linear_layers_gb300.dense_step`` runs a few steps on synthetic
data.
"""
from __future__ import annotations

import argparse
import math

import torch

import gemms_linear_layers_gb300 as tg
from . import inputs
from .expert_step import loss_and_gradient


class DenseBlock:
    """Weights, gradient and momentum buffers (kept for the whole run) and one step's saved tensors."""

    MATRICES = ("up", "down")
    VECTORS = ("w", "b")

    def __init__(self, hidden, ffn, act="silu", dtype=torch.bfloat16, device="cuda", tag="dense_step"):
        def normal(shape, name):
            return inputs.normal(shape, inputs.STD_W, dtype, inputs.seed_for(tag, *shape, str(dtype), name)).to(device)

        self.act = act
        self.weights = {"up": normal((2 * ffn, hidden), "up"), "down": normal((hidden, ffn), "down"),
                        "w": torch.ones(hidden, dtype=dtype, device=device),
                        "b": torch.zeros(hidden, dtype=dtype, device=device)}
        self.grads = {k: torch.zeros_like(v) for k, v in self.weights.items()}
        self.momentum = {k: torch.zeros_like(self.weights[k], dtype=torch.float32) for k in self.MATRICES}
        self.updates = {k: torch.zeros_like(self.weights[k]) for k in self.MATRICES}

    def forward(self, X):
        w = self.weights
        n = tg.tg_layer_norm_fwd(X, w["w"], b=w["b"])
        g = tg.tg_gated_fwd(n["Y"], w["up"], act=self.act, keep=True)
        self.saved = (X, n, g["GU"])
        return X + tg.tg_gemm_fwd(g["H"], w["down"])

    def backward(self, dY):
        """dX for the gradient of Y; fills the weights' gradients."""
        w, g = self.weights, self.grads
        X, n, GU = self.saved
        b = tg.tg_gated_bwd(dY, w["down"], GU, act=self.act, keep=True)
        tg.tg_gemm_wgrad(dY, b["H"], dW=g["down"])
        tg.tg_gemm_wgrad(b["dGU"], n["Y"], dW=g["up"])
        dN = tg.tg_gemm_dgrad(b["dGU"], w["up"])
        r = tg.tg_layer_norm_bwd(dN, X, w["w"], n["mean"], n["rstd"], dR=dY, outs={"dw": g["w"], "db": g["b"]})
        return r["dX"]

    def step(self, lr, mu=0.95, vector_lr=0.01):
        for k in self.MATRICES:
            m = self.momentum[k].mul_(mu).add_(self.grads[k])
            rows, cols = m.shape
            parts = (2, rows // 2, cols) if k == "up" else (1, rows, cols)
            scale = math.sqrt(max(1.0, parts[1] / parts[2]))
            tg.tg_orthogonalize(m.view(parts), O=self.updates[k].view(parts), scale=scale)
            self.weights[k].add_(self.updates[k], alpha=-lr)
        for k in self.VECTORS:
            self.weights[k].add_(self.grads[k], alpha=-vector_lr)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=576)
    ap.add_argument("--ffn", type=int, default=1536)
    ap.add_argument("--act", default="silu", choices=("silu", "gelu", "gelu_tanh", "relu"))
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--lr", type=float, default=0.02)
    a = ap.parse_args(argv)
    block = DenseBlock(a.hidden, a.ffn, a.act)
    X, target = (inputs.normal((a.tokens, a.hidden), 1.0, torch.bfloat16, inputs.seed_for("dense_step", n)).cuda()
                 for n in ("X", "target"))
    losses = []
    for _ in range(a.steps):
        loss, dY = loss_and_gradient(block.forward(X), target)
        block.backward(dY)
        block.step(a.lr)
        losses.append(loss)
    for k, loss in enumerate(losses):
        print(f"step {k}: loss {float(loss):.5f}")
    assert tg.tg_stream_status() == 0
    return [float(loss) for loss in losses]


if __name__ == "__main__":
    main()
