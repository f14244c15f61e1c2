"""The gated activation's gradient where w dh u alone is past FP32's range but the gradient, which is at most 1.1 of it and
far less for low gates, is not.

Tolerances as in test_checkpoints_gpu: 2^-8 of the result and 2^-16 of the sizes of its two terms."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_checkpoints_gpu import normal, save, values

pytestmark = pytest.mark.gpu
BF16, F64 = torch.bfloat16, torch.float64


@pytest.mark.parametrize("up,grad,weight", [(2.0 ** 40, 2.0 ** 90, 1.0), (2.0 ** 100, 2.0 ** 30, 0.5), (2.0 ** 70, 1.0, 2.0 ** 60)])
@pytest.mark.parametrize("inner", [32, 288])
def test_large_factors_of_low_gates(up, grad, weight, inner):
    torch.manual_seed(1)
    rows = 50
    X = normal(rows, 2 * inner).float()
    X[:, :inner] = -40 - 5 * X[:, :inner].abs()
    X[:, inner:] *= up
    Q, sf = save(X.to(BF16))
    dH = (normal(rows, inner, seed=1).float() * grad).to(BF16)
    w = (torch.rand(rows, device="cuda") + 0.5) * weight
    dX = torch.empty(rows, 2 * inner, device="cuda", dtype=BF16)
    tkg.swiglu_grad(Q, sf, dH, dX, weights=w)
    assert tkg.device_status() == tkg.OK
    g, u = values(Q, sf).chunk(2, dim=1)
    s, d = torch.sigmoid(g), dH.to(F64) * w.to(F64)[:, None]
    want = torch.cat([d * u * s * (1 + g * (1 - s)), d * g * s], dim=1)
    size = torch.cat([(d * u * s).abs() * (1 + (g * (1 - s)).abs()), (d * g * s).abs()], dim=1)
    assert ((d * u).abs() > 2.0 ** 128).any() and (want.abs() < 2.0 ** 127).all()
    assert ((dX.to(F64) - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16 * size).all()
