"""Trains a small mixture-of-experts layer under a language-model head with the library's products.

One step, all on the device and with no host synchronisation between the calls:

  router        tkg.moe_route, tkg.moe_dispatch (top-1 expert per token; tokens put in expert order, row counts left in
                device memory)
  forward       D_g = A_g B_g^T            tkg.gemm_grouped_dev_bf16     (expert products)
                Y = A + D                  (residual)
                loss, lse                  tkg.linear_ce_loss            (head and cross entropy, logits never kept)
  backward      dY, dW                     tkg.linear_ce_grad
                dA = dY + dD_g B_g         tkg.gemm_grouped_dev_bf16_dgrad
                dB_g += dD_g^T A_g         tkg.gemm_grouped_dev_bf16_wgrad (accumulated in FP32 over micro-batches)
  update        plain SGD on FP32 copies of the embedding, the experts and the head

The task is to name each token's successor under a fixed random permutation, so the loss falls from log(vocab).

    python examples/expert_head_training.py [--steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_block_scaled_gb300 import tkg  # noqa: E402

BF16 = torch.bfloat16


class Model:
    def __init__(self, vocab=4000, hidden=512, experts=8, tokens=2048, micro_batches=2, seed=1):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
        self.vocab, self.hidden, self.experts, self.tokens = vocab, hidden, experts, tokens
        self.micro_batches, self.gen = micro_batches, gen
        # FP32 parameters; the products take BF16 copies
        self.E = r(vocab, hidden)
        self.B = r(experts, hidden, hidden) * hidden ** -0.5
        self.W = r(vocab, hidden) * hidden ** -0.5
        self.R = r(hidden, experts)                     # a fixed router
        self.succ = torch.randperm(vocab, generator=gen, device="cuda")
        self.dloss = torch.full((tokens,), 1.0 / (tokens * micro_batches), device="cuda")
        self.workspace = torch.empty(max(tkg.linear_ce_loss_workspace_bytes(tokens, vocab),
                                         tkg.linear_ce_grad_workspace_bytes(tokens, vocab, hidden)),
                                     dtype=torch.uint8, device="cuda")

    def step(self, lr):
        B, W = self.B.to(BF16), self.W.to(BF16)
        dB, dW, dE = torch.zeros_like(self.B), torch.zeros_like(self.W), torch.zeros_like(self.E)
        total = torch.zeros((), device="cuda")
        for _ in range(self.micro_batches):
            ids = torch.randint(0, self.vocab, (self.tokens,), generator=self.gen, device="cuda")
            x = self.E[ids].to(BF16)
            # tokens in expert order, and how many each expert has
            i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")
            expert, rows, sizes, order = i32(self.tokens, 1), i32(self.tokens, 1), i32(self.experts), i32(self.tokens)
            tkg.moe_route(x.float() @ self.R, expert, torch.empty(self.tokens, 1, device="cuda"), sizes, rows, order)
            A = torch.empty_like(x)
            tkg.moe_dispatch(x, rows, A)
            ids = ids[order.long()]
            labels = self.succ[ids]
            # forward
            D = torch.empty_like(A)
            tkg.gemm_grouped_dev_bf16(sizes, A, B, D)
            Y = A + D
            loss, lse = torch.empty_like(self.dloss), torch.empty_like(self.dloss)
            tkg.linear_ce_loss(Y, W, labels, loss, lse, workspace=self.workspace)
            # backward
            dY, dA = torch.empty_like(Y), torch.empty_like(A)
            tkg.linear_ce_grad(Y, W, labels, lse, self.dloss, dY, dW, accumulate=True, workspace=self.workspace)
            tkg.gemm_grouped_dev_bf16_dgrad(sizes, dY, B, dA)
            tkg.gemm_grouped_dev_bf16_wgrad(sizes, dY, A, dB, accumulate=True)
            dE.index_add_(0, ids, dY.float() + dA.float())
            total += loss.sum()
        for p, g in ((self.E, dE), (self.B, dB), (self.W, dW)):
            p.sub_(g, alpha=lr)
        return total / (self.tokens * self.micro_batches)


def train(steps=60, lr=10.0, log=print, **kw):
    """Mean losses of the steps."""
    model = Model(**kw)
    losses = [model.step(lr) for _ in range(steps)]
    if tkg.device_status() != tkg.OK:
        raise RuntimeError("a kernel reported an error")
    losses = [float(x) for x in losses]
    for i in range(0, steps, max(1, steps // 10)):
        log(f"step {i:4d}  loss {losses[i]:.4f}")
    log(f"step {steps - 1:4d}  loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    train(steps=ap.parse_args().steps)
