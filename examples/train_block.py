"""Training a pre-norm gated FFN block, Y = X + FFN(LN(X)), with the library's
training operators: layer norm, the gated FFN's forward and backward passes,
and Muon's orthogonalised updates for the three weight matrices.

    python examples/train_block.py            # fits a random target, prints the loss
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import transformer_ffn_gb300 as tffn  # noqa: E402


class Block:
    """Weights and momenta of one block, N wide with O hidden columns."""

    def __init__(self, N, O, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[0] ** -0.5).bfloat16()

        self.gamma, self.beta = torch.ones(N, device=device), torch.zeros(N, device=device)
        self.W1, self.W3, self.W2 = normal(N, O), normal(N, O), normal(O, N)
        self.momentum = {k: torch.zeros(getattr(self, k).shape, device=device) for k in ("W1", "W3", "W2")}

    def forward(self, X):
        """The block's output X + FFN(LN(X)) as (branch output, saved tensors)."""
        Z, S, mean, rstd = tffn.layer_norm_forward(X, self.gamma, self.beta)
        Y, G, U = tffn.ffn_glu_forward_train(Z, self.W1, self.W3, self.W2, "silu")
        return Y, (S, mean, rstd, Z, G, U)

    def backward(self, dY, saved):
        """(dX, gradients) from the gradient dY of X + FFN(LN(X)): it reaches X past
        the branch as it is, and through it."""
        S, mean, rstd, Z, G, U = saved
        dZ, dW1, dW3, dW2 = tffn.ffn_glu_backward(dY, Z, self.W1, self.W3, self.W2, G, U, "silu")
        dX, dgamma, dbeta = tffn.layer_norm_backward(dZ, S, self.gamma, mean, rstd, dS=dY)
        return dX, {"W1": dW1, "W3": dW3, "W2": dW2, "gamma": dgamma, "beta": dbeta}

    def update(self, grads, lr=0.02, momentum=0.9):
        for k, m in self.momentum.items():
            m.mul_(momentum).add_(grads[k])
            W = getattr(self, k)
            # each singular direction of the update moves by the same step
            step = lr * max(1.0, W.shape[0] / W.shape[1]) ** 0.5
            W.add_(tffn.muon_orthogonalize(m), alpha=-step)
        self.gamma.add_(grads["gamma"], alpha=-lr)
        self.beta.add_(grads["beta"], alpha=-lr)


def train(steps=30, tokens=512, N=256, O=1024, seed=0):
    """Fits the block to a fixed random target; returns the losses."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    X = torch.randn((tokens, N), generator=g, device="cuda").bfloat16()
    target = torch.randn((tokens, N), generator=g, device="cuda")
    block, losses = Block(N, O, seed), []
    for _ in range(steps):
        Y, saved = block.forward(X)
        err = X.float() + Y.float() - target
        losses.append(err.square().mean())
        _, grads = block.backward((err * (2.0 / err.numel())).bfloat16(), saved)
        block.update(grads)
    tffn.check()
    return [float(x) for x in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps)):
        print(f"step {i:3d}  loss {loss:.4f}")
