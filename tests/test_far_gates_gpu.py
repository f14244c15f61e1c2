"""The gated activation and its gradient at gates below -87, whose sigma is among FP32's subnormal numbers or below them: what
the products with u and dH are, is kept.

References in 64 bits.  Tolerances: a far gate's exponential is the fourth power of one that is off by 2 units (2^-20), and
five products are rounded: below 2^-16, as ordinary gates are.  A BF16 result is rounded once, half a step: 2^-8 of it, or
2^-134 among its subnormal numbers.  dweights sums FP32 values of h (off by 2^-150 among the subnormal ones) times dH:
2^-17 of the sum of sizes, as in test_checkpoints_gpu."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_checkpoints_gpu import normal, save, values

pytestmark = pytest.mark.gpu
BF16, F32, F64, U8 = torch.bfloat16, torch.float32, torch.float64, torch.uint8
GATES = [-80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -89.0, -95.0, -104.0, -120.0, -150.0, -180.0, -250.0, -349.0, -500.0, -1e30]
UPS = [1.0, -3.0, 2.0 ** -20, 2.0 ** 40, -2.0 ** 100, 2.0 ** 127]


@pytest.fixture(autouse=True)
def _healthy():
    torch.manual_seed(1)
    yield
    assert tkg.device_status() == tkg.OK


def silu(g):
    return g * torch.sigmoid(g)


def activate(X, save_too):
    H = torch.empty(X.shape[0], X.shape[1] // 2, device="cuda", dtype=BF16)
    if save_too:
        tkg.swiglu(X, H, torch.empty(X.shape, device="cuda", dtype=U8), torch.empty(X.shape[0], X.shape[1] // 32, device="cuda", dtype=U8))
    else:
        tkg.swiglu(X, H)
    return H


@pytest.mark.parametrize("save_too", [False, True])
def test_activation(save_too):
    g, u = torch.cartesian_prod(torch.tensor(GATES), torch.tensor(UPS)).to(BF16).cuda().T
    X = torch.cat([g.repeat(5, 1), u.repeat(5, 1)], dim=1)           # 96 columns
    H = activate(X, save_too).to(F64)
    ref = silu(g.to(F64)) * u.to(F64)
    assert ((H - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 2.0 ** -134).all()
    assert (H[:, ((g == -88) & (u.abs() >= 1)).nonzero()[:, 0]] != 0).all()    # (times 2^-20: below 2^-134)


@pytest.mark.parametrize("save_too", [False, True])
@pytest.mark.parametrize("share", [0.02, 0.5])
def test_activation_of_other_gates_is_as_before(share, save_too):
    X = normal(70, 2 * 320) * 3
    far = torch.rand(70, 320, device="cuda") < share
    want = activate(X, save_too)
    Y = X.clone()
    Y[:, :320] = torch.where(far, torch.tensor(-100.0, dtype=BF16, device="cuda"), X[:, :320])
    got = activate(Y, save_too)
    assert torch.equal(got[~far], want[~far])
    ref = silu(Y[:, :320].to(F64)) * Y[:, 320:].to(F64)
    assert ((got.to(F64) - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 2.0 ** -134).all()


def gradient(Q, sf, dH, w):
    rows, inner = dH.shape
    dX, H, dw = torch.empty(rows, 2 * inner, device="cuda", dtype=BF16), torch.empty_like(dH), torch.empty_like(w)
    tkg.swiglu_grad(Q, sf, dH, dX, H, weights=w, dweights=dw)
    return dX, H, dw


def check_gradient(Q, sf, dH, w):
    got, H, dw = gradient(Q, sf, dH, w)
    g, u = values(Q, sf).chunk(2, dim=1)
    s, d = torch.sigmoid(g), dH.to(F64)
    ww = w.to(F64)[:, None]
    h = g * s * u
    dg, du = ww * d * u * s * (1 + g * (1 - s)), ww * d * g * s
    want = torch.cat([dg, du], dim=1)
    size = torch.cat([(ww * d * u * s).abs() * (1 + (g * (1 - s)).abs()), du.abs()], dim=1)
    fits = want.abs() < 2.0 ** 127                                  # past 2^128 a BF16 is infinite
    off = (got.to(F64) - want).abs()
    # (u sigma' is held in FP32: half a step of its subnormal numbers, times w dh)
    room = 2.0 ** -8 * want.abs() + 2.0 ** -16 * size + 2.0 ** -134 + 2.0 ** -150 * (ww * d).abs().repeat(1, 2)
    assert (off <= room)[fits].all()
    assert (got.to(F64) == torch.where(want > 0, torch.inf, -torch.inf))[want.abs() > 2.0 ** 129].all()
    assert ((H.to(F64) - ww * h).abs() <= (2.0 ** -8 + 2.0 ** -16) * (ww * h).abs() + 2.0 ** -134).all()
    # (where the sum is subnormal itself, each of its additions rounds to steps of 2^-149: half a step for each column)
    room = 2.0 ** -17 * (d * h).abs().sum(dim=1) + 2.0 ** -150 * (d.abs().sum(dim=1) + d.shape[1])
    assert ((dw.to(F64) - (d * h).sum(dim=1)).abs() <= room)[(d * h).abs().sum(dim=1) < 2.0 ** 127].all()
    return got, H


SAVED = [-56.0, -80.0, -88.0, -96.0, -104.0, -112.0, -120.0, -128.0, -144.0, -176.0, -208.0, -240.0, -288.0, -352.0, -448.0, 1.0]


@pytest.mark.parametrize("up", [1.0, 2.0 ** -20, 2.0 ** 40, 2.0 ** 100])
@pytest.mark.parametrize("grad", [1.0, 2.0 ** -20, 2.0 ** 20, 2.0 ** 90])
@pytest.mark.parametrize("inner", [64, 544, 2080])
def test_gradient(inner, up, grad):
    rows = 40
    X = normal(rows, 2 * inner).float()
    X[:, :inner] = torch.tensor(SAVED, device="cuda")[torch.randint(0, len(SAVED), (rows, inner), device="cuda")]
    X[::4, :inner] = 2 * X[::4, :inner].clamp(max=0)
    X[:, inner:] *= up
    Q, sf = save(X.to(BF16))
    got, H = check_gradient(Q, sf, (normal(rows, inner, seed=1).float() * grad).to(BF16), torch.rand(rows, device="cuda") + 0.1)
    g = values(Q, sf)[:, :inner]
    if up == grad == 1.0:
        assert (got[:, :inner][g == -88] != 0).float().mean() > 0.9 and (H[g == -88] != 0).float().mean() > 0.9


def test_gradient_of_other_gates_is_as_before():
    rows, inner = 60, 320
    X = normal(rows, 2 * inner) * 30
    X[:, :inner].clamp_(min=-86)
    X[:, 0] = -85
    Q, sf = save(X)                                 # blocks whose scale leaves room for far gates
    X[:, ::32] = 224
    dH, w = normal(rows, inner, seed=3), torch.rand(rows, device="cuda")
    dX, H, _ = gradient(Q, sf, dH, w)
    far = torch.rand(rows, inner, device="cuda") < 0.3
    codes = Q.clone()
    codes[:, :inner] = torch.where(far, torch.tensor(0xfe, dtype=U8, device="cuda"), Q[:, :inner])   # -448 of the scale
    got, H2 = check_gradient(codes, sf, dH, w)
    assert torch.equal(H2[~far], H[~far]) and torch.equal(got[:, :inner][~far], dX[:, :inner][~far])
    assert torch.equal(got[:, inner:][~far], dX[:, inner:][~far])


def test_infinities_and_nan_among_far_gates():
    X = torch.ones(4, 64, device="cuda", dtype=BF16)
    X[:, :32] = -90
    X[0, 5], X[1, 6], X[2, 7] = float("nan"), -torch.inf, torch.inf
    X[3, 32] = float("nan")
    H = activate(X, True)
    assert H.isnan().sum() == 3 and H[0, 5].isnan() and H[1, 6].isnan() and H[3, 0].isnan() and H[2, 7] == torch.inf
