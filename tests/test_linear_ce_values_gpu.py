"""Values at which the cross entropy of a head and its gradient can go wrong without showing it: weights and operands
that are not finite, tokens that the model is sure of, sums that are long."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_linear_ce_gpu import BF16, F32, F64, Head, run_grad, run_loss

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK
    tkg.set_option(tkg.OPT_CTA_GROUP, 0)


def weight_gradient(h, lse, kind, dX):
    """(dX or None, dW) with dW in BF16, FP32, or added to FP32 ones."""
    gX = torch.full(h.X.shape, 7.0, device="cuda", dtype=BF16) if dX else None
    dW = torch.ones(h.W.shape, device="cuda", dtype=BF16 if kind == "bf16" else F32)
    tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, gX, dW, alpha=h.alpha, accumulate=kind == "add")
    return gX, dW


# 8 tokens: the rows of X are weighted beside the logits; 200: by a kernel of their own
@pytest.mark.parametrize("tokens", [8, 200])
@pytest.mark.parametrize("kind", ["bf16", "f32", "add"])
@pytest.mark.parametrize("others", ["nan", "zero", "one", "kept"])
def test_a_weight_that_is_not_a_number_reaches_dw(tokens, kind, others):
    h = Head(tokens, 600, 72, ignored=0.0)
    h.y[1] = -100   # an ignored row stays out
    lse = h.forward()[2].float()
    if others != "kept":
        h.dloss[:] = {"nan": float("nan"), "zero": 0.0, "one": 1.0}[others]
    clean = weight_gradient(h, lse, kind, True)[0]
    h.dloss[3] = float("nan")
    for dX in (True, False):
        gX, dW = weight_gradient(h, lse, kind, dX)
        assert torch.isnan(dW).all()
        if dX:
            rest = torch.arange(tokens, device="cuda") != 3
            assert torch.isnan(gX[3]).all() and torch.equal(gX[rest].view(torch.int16), clean[rest].view(torch.int16))
            assert (gX[1] == 0).all()


@pytest.mark.parametrize("tokens", [8, 200])
@pytest.mark.parametrize("kind", ["bf16", "f32", "add"])
def test_an_infinite_weight_gives_infinite_gradients(tokens, kind):
    h = Head(tokens, 600, 72, ignored=0.0)
    z, _, lse, _, _ = h.forward()
    h.dloss[5] = float("inf")
    g = torch.exp(z[5] - lse[5])
    g[h.y[5]] -= 1
    want = float("inf") * g[:, None] * h.X[5].to(F64)[None, :]   # infinities, and NaN where X holds a zero
    gX, dW = weight_gradient(h, lse.float(), kind, True)
    assert torch.equal(torch.nan_to_num(dW.to(F64), nan=0.5), torch.nan_to_num(want, nan=0.5))
    assert torch.isinf(gX[5]).all() and torch.isfinite(gX[torch.arange(tokens, device="cuda") != 5]).all()


def test_zero_weights_give_zero_gradients():
    for tokens in (8, 200):
        h = Head(tokens, 600, 72, ignored=0.0)
        h.dloss[:] = 0
        gX, dW = weight_gradient(h, h.forward()[2].float(), "add", True)
        assert (gX == 0).all() and (dW == 1).all()
