"""Sigmoid scores of low logits: below -88.7 exp(-z) is past FP32's range and sigma among its subnormal numbers or below
them, but the chosen's shares of their sum are ordinary numbers.

Reference: log sigma(z) = min(z, 0) - log(1 + exp(-|z|)) in 64 bits; the shares are its softmax over the chosen.  Tolerances: of a share as
in test_moe_route_gpu (2^-16 of it, and the least normal number); of a sigma alone 2^-16 of it, and 10 steps of the
subnormal numbers (exp's 2, times the scale of 2.5, and the product's rounding)."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_moe_route_gpu import choice, normal, route

pytestmark = pytest.mark.gpu
F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
TINY, STEP = 2.0 ** -126, 2.0 ** -149
BASES = [-20.0, -80.0, -88.0, -95.0, -104.0, -200.0, -600.0, -1000.0, -30000.0]


@pytest.fixture(autouse=True)
def _healthy():
    torch.manual_seed(1)
    yield
    assert tkg.device_status() == tkg.OK


def log_sigmoid(z):
    z = z.to(F64)
    return z.clamp(max=0) - torch.log1p(torch.exp(-z.abs()))


def shares(z, ids):
    """Renormalised weights of the chosen: 0 where all of them are -inf."""
    low = log_sigmoid(z).gather(1, ids)
    top = low.amax(dim=1, keepdim=True)
    e = torch.exp(low - torch.where(top == -torch.inf, 0.0, top))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def check_shares(z, topk, **kw):
    ids, w, *_ = route(z, topk, scores="sigmoid", renormalise=True, scale=2.5, **kw)
    want = 2.5 * shares(z, ids.long())
    assert ((w - want).abs() <= 2.0 ** -16 * want + TINY).all()
    return ids, w


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("base", BASES)
@pytest.mark.parametrize("tokens,experts,topk", [(1, 8, 2), (50, 64, 6), (300, 200, 32), (700, 512, 1)])
def test_all_logits_low(tokens, experts, topk, base, dtype):
    z = (normal(tokens, experts) + base).to(dtype)
    ids, w = check_shares(z, topk)
    assert torch.equal(ids.long(), choice(z, topk)) and ((w.sum(dim=1) - 2.5).abs() < 1e-5).all()


def test_two_low_logits():
    z = torch.full((3, 16), -torch.inf, device="cuda")
    z[:, 3], z[:, 9] = -90.0, -91.0
    ids, w = check_shares(z, 4)
    assert ids[0, :2].tolist() == [3, 9] and (w[0, 2:] == 0).all()
    assert abs(float(w[0, 0]) / 2.5 - 0.7310586) < 1e-5
    z[1] = -torch.inf
    assert (check_shares(z, 4)[1][1] == 0).all()


@pytest.mark.parametrize("base", BASES[1:])
@pytest.mark.parametrize("groups,stay", [(1, 1), (8, 3)])
def test_low_logits_beside_high_ones(base, groups, stay):
    # rows with none, one or all of the chosen low; a bias chooses the low ones
    z = normal(120, 64)
    z[::3] += base
    z[1::3, 1:] += base
    bias = torch.zeros(64, device="cuda")
    bias[40:] = 4.0
    z[2::3, 40:] += base
    check_shares(z, 5, bias=bias, groups=groups, topk_groups=stay)
    check_shares(z, 5, groups=groups, topk_groups=stay)


@pytest.mark.parametrize("base", BASES)
def test_sigmas_themselves(base):
    z = (normal(200, 64, scale=5.0) + base)
    ids, w, *_ = route(z, 8, scores="sigmoid", renormalise=False, scale=2.5)
    want = 2.5 * torch.exp(log_sigmoid(z).gather(1, ids.long()))
    assert ((w - want).abs() <= 2.0 ** -16 * want + 10 * STEP).all()


def weights_of(z, ids, renormalise):
    low = (z.clamp(max=0) - torch.log1p(torch.exp(-z.abs()))).gather(1, ids.clamp(min=0))
    w = torch.softmax(low, dim=1) if renormalise else torch.exp(low)
    return torch.where(ids >= 0, 2.5 * w, 0.0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("base", BASES)
@pytest.mark.parametrize("tokens,experts,topk", [(1, 8, 2), (60, 64, 6), (300, 200, 32)])
def test_gradient_of_low_logits(tokens, experts, topk, base, dtype):
    z = (normal(tokens, experts) + base).to(dtype)
    z[1::3] = normal(tokens, experts, dtype=dtype)[1::3]               # and of ordinary ones
    z[2::3, ::2] = normal(tokens, experts, dtype=dtype)[2::3, ::2]     # and of both in a row
    keep = torch.arange(tokens, device="cuda") % 5 != 3
    ids = torch.rand(tokens, experts, device="cuda").topk(topk, dim=1).indices   # not the largest ones alone
    ids = torch.where(keep[:, None], ids, -1)
    dw = normal(tokens, topk, scale=1.0)
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -23
    for renormalise in (True, False):
        got = torch.empty_like(z)
        tkg.moe_route_grad(z, ids.to(torch.int32), dw, got, scores="sigmoid", renormalise=renormalise, scale=2.5)
        x = z.to(F64).requires_grad_(True)
        w = weights_of(x, ids, renormalise)
        (w * dw.to(F64)).sum().backward()
        w = w.detach()
        of = dw.abs() + (w * dw.abs()).sum(dim=1, keepdim=True) if renormalise else dw.abs()
        size = torch.zeros_like(x).scatter_add_(1, ids.clamp(min=0), w * of)
        assert ((got.to(F64) - x.grad).abs() <= 2.0 ** -16 * size + half * x.grad.abs() + 1e-38).all()
        # and against differences of the weights: along v, which spreads over 8 at most, a share's third derivative is below
        # 1100 (8^3 + 3 x 8 x 4^2 and v's third moment) of it, and a sixth of that counts
        v = torch.randn(tokens, experts, device="cuda", dtype=F64).clamp(-4, 4)
        h = 1e-4
        up, down = (weights_of(z.to(F64) + d * v, ids, renormalise) for d in (h, -h))
        along, diff = (got.to(F64) * v).sum(dim=1), ((up - down) / (2 * h) * dw.to(F64)).sum(dim=1)
        room = h * h * 1100 / 6 * 2.5 * dw.abs().sum(dim=1) + ((2.0 ** -16 * size + half * x.grad.abs()) * v.abs()).sum(dim=1)
        assert ((along - diff).abs() <= room + 1e-9).all()
    assert (got[~keep] == 0).all()
