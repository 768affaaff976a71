"""A training step of a mixture-of-experts block on the library's entry points.

The block, for tokens N [T, hidden] (normed) beside a residual stream H:
  router    p = softmax(N R^T), each token to its likeliest expert e with probability g
  experts   B = W_down[e] silu(W_up[e] N)          tg_grouped_fwd, rows sorted by expert
  join      H' = H + g norm(B; w_post), N' = norm(H'; w_pre)    tg_norm_residual_fwd
Backward: tg_norm_residual_bwd (its token gate's gradient is the router's),
tg_grouped_dgrad, tg_grouped_wgrad; then all gradients are clipped by their
global norm (tg_grad_clip) and a plain gradient step is taken.  Nothing waits
for the host: the experts' row counts stay on the device.

``python -m gemms_linear_layers_gb300.expert_step`` runs a few steps on
synthetic data.
"""
from __future__ import annotations

import argparse

import torch

import gemms_linear_layers_gb300 as tg
from . import inputs


class ExpertBlock:
    """Weights, gradient buffers (kept for the whole run) and one step's saved tensors."""

    NAMES = ("router", "up", "down", "w_post", "w_pre")

    def __init__(self, hidden, ffn, experts, dtype=torch.bfloat16, device="cuda", tag="expert_step"):
        def normal(shape, std, name):
            return inputs.normal(shape, std, dtype, inputs.seed_for(tag, *shape, str(dtype), name)).to(device)

        self.experts = experts
        self.weights = {"router": normal((experts, hidden), inputs.STD_W, "router"),
                        "up": normal((experts, ffn, hidden), inputs.STD_W, "up"),
                        "down": normal((experts, hidden, ffn), inputs.STD_W, "down"),
                        "w_post": torch.ones(hidden, dtype=dtype, device=device),
                        "w_pre": torch.ones(hidden, dtype=dtype, device=device)}
        self.grads = {k: torch.zeros_like(w) for k, w in self.weights.items()}
        self.grad_list = tg.tg_tensor_list(self.grads[k] for k in self.NAMES)

    def forward(self, N, H):
        """(H', N') for tokens N and stream H, both [T, hidden]."""
        w = self.weights
        p = torch.softmax(tg.tg_gemm_fwd(N, w["router"], out_dtype=torch.float32), dim=1)
        prob, expert = p.max(dim=1)
        expert, order = torch.sort(expert, stable=True)
        first = torch.arange(self.experts + 1, device=N.device)
        offsets = torch.searchsorted(expert, first).to(torch.int32)
        X = N[order]
        A = tg.tg_grouped_fwd(X, w["up"], offsets)
        Z = torch.nn.functional.silu(A)
        B = torch.empty_like(N)
        B[order] = tg.tg_grouped_fwd(Z, w["down"], offsets)
        gate = prob[:, None].to(N.dtype)
        r = tg.tg_norm_residual_fwd(B, H, w["w_post"], w["w_pre"], gate=gate)
        self.saved = (N, p, prob, order, expert, offsets, X, A, Z, B, gate, r)
        return r["H"], r["N"]

    def backward(self, dH_out, dN_out):
        """(dH, dN) for the gradients of H' and N'; fills the weights' gradients."""
        w, g = self.weights, self.grads
        N, p, prob, order, expert, offsets, X, A, Z, B, gate, r = self.saved
        b = tg.tg_norm_residual_bwd(dH_out, dN_out, B, r["H"], w["w_post"], w["w_pre"], r["rstd_b"], r["rstd_h"],
                                    gate=gate, outs={"dw_post": g["w_post"], "dw_pre": g["w_pre"]})
        dB = b["dB"][order]
        tg.tg_grouped_wgrad(dB, Z, offsets, dW=g["down"])
        dZ = tg.tg_grouped_dgrad(dB, w["down"], offsets)
        s = torch.sigmoid(A.float())
        dA = (dZ.float() * s * (1 + A.float() * (1 - s))).to(A.dtype)
        tg.tg_grouped_wgrad(dA, X, offsets, dW=g["up"])
        dN = torch.empty_like(N)
        dN[order] = tg.tg_grouped_dgrad(dA, w["up"], offsets)
        # the router: d prob / d logits = prob (1[e] - p)
        chosen = torch.zeros_like(p)
        chosen[order, expert] = 1.0
        dlogits = (b["dgate"].float() * prob[:, None] * (chosen - p)).to(N.dtype)
        tg.tg_gemm_wgrad(dlogits, N, dW=g["router"])
        dN += tg.tg_gemm_dgrad(dlogits, w["router"])
        return b["dH"], dN

    def step(self, lr, max_norm):
        """Clips the gradients by their global norm and takes a gradient step; returns the norm (on the device)."""
        norm = tg.tg_grad_clip(self.grad_list, max_norm)
        for k in self.NAMES:
            self.weights[k].add_(self.grads[k], alpha=-lr)
        return norm


def loss_and_gradient(out, target):
    """The squared distance of a token's output from its target, averaged over the tokens, and its gradient for
    `out` in out's type."""
    diff = out.float() - target.float()
    return diff.square().sum(1).mean(), (diff * (2.0 / out.shape[0])).to(out.dtype)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=576)
    ap.add_argument("--ffn", type=int, default=1536)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--lr", type=float, default=0.5)
    ap.add_argument("--max-norm", type=float, default=1.0)
    a = ap.parse_args(argv)
    block = ExpertBlock(a.hidden, a.ffn, a.experts)
    shape = (a.tokens, a.hidden)
    H, target = (inputs.normal(shape, 1.0, torch.bfloat16, inputs.seed_for("expert_step", n)).cuda() for n in ("H", "target"))
    N = (H.float() * torch.rsqrt(H.float().square().mean(1, keepdim=True) + 1e-6)).to(H.dtype)
    zero = torch.zeros_like(H)
    losses = []
    for k in range(a.steps):
        _, out = block.forward(N, H)
        loss, dN = loss_and_gradient(out, target)
        block.backward(zero, dN)
        norm = block.step(a.lr, a.max_norm)
        losses.append((loss, norm))
    for k, (loss, norm) in enumerate(losses):
        print(f"step {k}: loss {float(loss):.5f}, gradient norm {float(norm):.4f}")
    assert tg.tg_stream_status() == 0
    return [float(loss) for loss, _ in losses]


if __name__ == "__main__":
    main()
