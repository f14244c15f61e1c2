"""The training loop of examples/moe_block.py: the error that it reports, the gradient that it starts from, and the step that it
takes along each parameter's gradient, against the formulas in 64 bits.

Tolerances.  A gradient is off by 5 x 2^-8 in norm, as in test_moe_block_gpu; parameters are seen as the blocks get them, in
BF16, so a step between two of them is off by half a BF16 step (2^-8) of each end's norm at most."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_moe_block_gpu import example, reference  # noqa: F401

pytestmark = pytest.mark.gpu
F32, F64 = torch.float32, torch.float64


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [(256, 256, 128, 16, 4), (300, 128, 64, 8, 1), (200, 64, 96, 24, 3)])
def test_a_step_goes_along_the_gradients(example, monkeypatch, tokens, hidden, inner, experts, topk):  # noqa: F811
    made = []

    class Recorded(example.Block):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            made.append(self)

        def forward(self, X, **kw):
            self.X, self.Y = X, super().forward(X, **kw)
            return self.Y

        def backward(self, dY, dW1, dW2):
            assert (dW1 == 0).all() and (dW2 == 0).all()
            self.dY = dY
            return super().backward(dY, dW1, dW2)

    monkeypatch.setattr(example, "Block", Recorded)
    lr = 250.0     # a step about as long as the parameters, so that it is seen through their BF16 copies
    losses = example.train(steps=2, tokens=tokens, hidden=hidden, inner=inner, experts=experts, topk=topk, lr=lr, log=lambda *_: None)
    teacher, first, second = made
    target = Recorded(teacher.Wr, teacher.W1, teacher.W2, topk).forward(first.X)
    off = first.Y.to(F64) - target.to(F64)
    assert abs(losses[0] - float(off.square().mean())) <= 1e-4 * losses[0]
    dY = off * (2.0 / hidden)
    assert ((first.dY.to(F64) - dY).abs() <= (2.0 ** -8 + 2.0 ** -22) * dY.abs()).all()
    _, _, dz, dW1, dW2 = reference(first, first.X, first.dY)
    # the loss's sums over a token's columns, scaled by the rows that an expert has on average
    scale = lr / (tokens * topk / experts)
    for name, grad in (("Wr", dz.T @ first.X.to(F64)), ("W1", dW1), ("W2", dW2)):
        before, after = getattr(first, name).to(F64), getattr(second, name).to(F64)
        step = scale * grad
        if topk == 1 and name == "Wr":      # (the weight of a single choice is 1)
            assert dz.abs().max() < 1e-12 and torch.equal(before, after)    # (in 64 bits w / w has its roundings)
            continue
        assert step.norm() > 0.1 * before.norm(), name
        room = 5 * 2.0 ** -8 * step.norm() + 2.0 ** -8 * (before.norm() + after.norm())
        err = (after - before + step).norm()
        assert err <= room, f"{name}: {float(err):.3g} of {float(room):.3g}"
