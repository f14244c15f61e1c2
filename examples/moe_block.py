"""A mixture-of-experts block, forward and backward, from the library's calls; trained on a small regression.

All on the device, with no host synchronisation between the calls.  T tokens of H columns, E experts of I, k of them per
token; R = T k rows in expert order:

  forward   z = X Wr^T                       tkg.gemm_bf16                     (router's logits)
            ids, weights, sizes, rows, slots tkg.moe_route
            Xs = X in expert order           tkg.moe_dispatch
            GU = Xs W1_e^T                   tkg.gemm_grouped_dev_bf16         (gate and up in one product)
            h = silu(g) u                    tkg.swiglu                        (saves GU in 8 bits)
            O = h W2_e^T                     tkg.gemm_grouped_dev_bf16
            Y = sum weights O                tkg.moe_combine
  kept      X and GU in 8 bits               tkg.checkpoint_mxfp8, tkg.swiglu  (H + 2 I k bytes a token and 1/32 of that)
  backward  dYs = dY in expert order         tkg.moe_dispatch
            dh = dYs W2_e                    tkg.gemm_grouped_dev_bf16_dgrad   (without the router's weights)
            dGU, w h, dweights               tkg.swiglu_grad                   (they come in here: O is not kept)
            dW2_e += dYs^T (w h)             tkg.gemm_grouped_dev_bf16_wgrad
            dW1_e += dGU^T X                 tkg.gemm_grouped_dev_mxfp8_wgrad  (X's saved rows, once per token)
            dX = sum over the choices        tkg.gemm_grouped_dev_bf16_dgrad, tkg.moe_combine
            dz                               tkg.moe_route_grad

    python examples/moe_block.py [--steps 40]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dense_block_scaled_gb300 import tkg  # noqa: E402

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _empty(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Block:
    """Weights in BF16 (copies of FP32 ones, if there are any): Wr (E x H), W1 (E x 2 I x H), W2 (E x H x I)."""

    def __init__(self, Wr, W1, W2, topk, **rule):
        self.Wr, self.W1, self.W2, self.topk, self.rule = Wr, W1, W2, topk, rule

    def forward(self, X, keep=None, bias=None):
        t, hidden = X.shape
        experts, k = self.Wr.shape[0], self.topk
        inner, r = self.W1.shape[1] // 2, t * k
        z = _empty(t, experts)
        tkg.gemm_bf16(X, self.Wr, z)
        ids, weights, sizes = _empty(t, k, dtype=I32), _empty(t, k, dtype=F32), _empty(experts, dtype=I32)
        rows, slots = _empty(t, k, dtype=I32), _empty(r, dtype=I32)
        tkg.moe_route(z, ids, weights, sizes, rows, slots, bias=bias, keep=keep, **self.rule)
        Xs, GU, h, O, Y = _empty(r, hidden), _empty(r, 2 * inner), _empty(r, inner), _empty(r, hidden), _empty(t, hidden)
        tkg.moe_dispatch(X, rows, Xs)
        tkg.gemm_grouped_dev_bf16(sizes, Xs, self.W1, GU)
        saved = _empty(r, 2 * inner, dtype=U8), _empty(r, inner // 16, dtype=U8)
        tkg.swiglu(GU, h, *saved)
        tkg.gemm_grouped_dev_bf16(sizes, h, self.W2, O)
        tkg.moe_combine(O, rows, Y, weights=weights)
        saved_x = _empty(t, hidden, dtype=U8), _empty(t, hidden // 32, dtype=U8)
        tkg.checkpoint_mxfp8(X, *saved_x)
        self.kept = z, ids, weights, sizes, rows, slots, saved, saved_x
        return Y

    def backward(self, dY, dW1, dW2):
        """dX through the experts, and the logits' gradient; adds to dW1 and dW2 (FP32)."""
        z, ids, weights, sizes, rows, slots, saved, saved_x = self.kept
        r, hidden, inner = slots.shape[0], dY.shape[1], self.W1.shape[1] // 2
        dYs, dXs, dh, h, dGU = _empty(r, hidden), _empty(r, hidden), _empty(r, inner), _empty(r, inner), _empty(r, 2 * inner)
        dweights, dz, dX = torch.zeros_like(weights), torch.empty_like(z), torch.empty_like(dY)
        tkg.moe_dispatch(dY, rows, dYs)
        tkg.gemm_grouped_dev_bf16_dgrad(sizes, dYs, self.W2, dh)
        tkg.swiglu_grad(*saved, dh, dGU, h, slots=slots, weights=weights, dweights=dweights)
        tkg.gemm_grouped_dev_bf16_wgrad(sizes, dYs, h, dW2, accumulate=True)
        tkg.gemm_grouped_dev_mxfp8_wgrad(sizes, dGU, *saved_x, dW1, slots=slots, topk=self.topk, accumulate=True)
        tkg.gemm_grouped_dev_bf16_dgrad(sizes, dGU, self.W1, dXs)
        tkg.moe_combine(dXs, rows, dX)
        rule = {n: v for n, v in self.rule.items() if n in ("scores", "renormalise", "scale")}
        tkg.moe_route_grad(z, ids, dweights, dz, **rule)
        return dX, dz


def train(steps=40, tokens=2048, hidden=256, inner=128, experts=16, topk=4, lr=2.0, seed=1, log=print):
    """Mean squared errors of the steps, of a block that learns what a fixed one of the same shape does."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    make = lambda: [r(experts, hidden) * hidden ** -0.5, r(experts, 2 * inner, hidden) * hidden ** -0.5,
                    r(experts, hidden, inner) * inner ** -0.5]
    teacher = Block(*[w.to(BF16) for w in make()], topk)
    params, losses = make(), []
    params[0] = teacher.Wr.float()       # the same routing at the start
    for _ in range(steps):
        X = r(tokens, hidden).to(BF16)
        target = teacher.forward(X)
        block = Block(*[w.to(BF16) for w in params], topk)
        off = block.forward(X).float() - target.float()
        losses.append(off.square().mean())
        dW1, dW2 = torch.zeros_like(params[1]), torch.zeros_like(params[2])
        _, dz = block.backward((off * (2.0 / hidden)).to(BF16), dW1, dW2)     # of the mean over a token's columns
        dWr = dz.float().T @ X.float()
        for p, g in zip(params, (dWr, dW1, dW2)):
            p.sub_(g, alpha=lr / tokens * experts / topk)
    if tkg.device_status() != tkg.OK:
        raise RuntimeError("a kernel reported an error")
    losses = [float(x) for x in losses]
    for i in range(0, steps, max(1, steps // 8)):
        log(f"step {i:4d}  error {losses[i]:.4f}")
    log(f"step {steps - 1:4d}  error {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    train(steps=ap.parse_args().steps)
