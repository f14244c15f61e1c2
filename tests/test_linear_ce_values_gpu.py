"""Values at which the cross entropy of a head and its gradient can go wrong without showing it: weights and operands
that are not finite, tokens that the model is sure of, sums that are long."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_linear_ce_gpu import BF16, F32, F64, Head, check_grad, run_grad, run_loss

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


def product_error(h):
    """Largest error of each token's logits: products are exact, and the accumulator of 16-product steps loses less than
    2^-23 of what it holds, at most the sum of magnitudes, at each; two roundings more (the scale, a sum of sums)."""
    mag = abs(h.alpha) * (h.X.to(F64).abs() @ h.W.to(F64).abs().T).max(dim=1).values
    return (h.shape[2] / 16 + 2) * 2.0 ** -23 * mag


# forms of the loss: a few tokens without tensor cores, and on them (cta_group 2); narrow, wide, and sums in parts
LOSS_FORMS = [(1, 3000, 264, 0), (3, 1001, 4104, 0), (4, 777, 256, 2), (20, 20003, 256, 0), (40, 20000, 4104, 0),
              (100, 1500, 520, 0), (300, 700, 4104, 0), (513, 2049, 64, 0), (2, 1, 64, 0), (90, 1, 64, 0)]


@pytest.mark.parametrize("alpha", [1.0, -0.5, 3.0])
@pytest.mark.parametrize("tokens,vocab,hidden,cta_group", LOSS_FORMS)
def test_loss_to_its_last_bits(tokens, vocab, hidden, cta_group, alpha):
    """lse moves by no more than its logits; exponentials 2^-21 each, their sums' additions under 40 roundings: 2^-18 in
    all.  The definition's loss is not negative, and neither is the kernel's."""
    tkg.set_option(tkg.OPT_CTA_GROUP, cta_group)
    h = Head(tokens, vocab, hidden, alpha=alpha, ignored=0.0, seed=21)
    _, _, lse, loss, _ = h.forward()
    got, got_lse = run_loss(h)
    tol = product_error(h) + 2.0 ** -18 + 2.0 ** -23 * lse.abs()
    assert ((got_lse.to(F64) - lse).abs() <= tol).all()
    assert ((got.to(F64) - loss).abs() <= 2 * tol).all()
    assert (got >= 0).all()


@pytest.mark.parametrize("alpha", [1.0, -0.5])
@pytest.mark.parametrize("scale", [0.25, 1.0])
@pytest.mark.parametrize("tokens,vocab,hidden,cta_group", [f for f in LOSS_FORMS if f[1] > f[0]])
def test_loss_of_tokens_the_model_is_sure_of(tokens, vocab, hidden, cta_group, scale, alpha):
    """A label whose row is the token's own: its logit is above the others by more than 30, whose exponentials vanish
    beside it in 32 bits, so that lse is that logit and the loss exactly 0."""
    tkg.set_option(tkg.OPT_CTA_GROUP, cta_group)
    h = Head(tokens, vocab, hidden, alpha=alpha, ignored=0.0, seed=22, spread=1e-3)
    h.y = torch.randperm(vocab, device="cuda")[:tokens]
    # powers of two: the rows stay exact; logits of 64 to 256 whatever hidden is
    h.W[h.y] = (h.X.float() * (scale / alpha * 2.0 ** (8 - round(torch.log2(torch.tensor(float(hidden))).item())))).to(BF16)
    z, _, lse, loss, _ = h.forward()
    own = z.gather(1, h.y[:, None])[:, 0]
    rest = z.scatter(1, h.y[:, None], float("-inf")).max(dim=1).values
    sure = own - rest > 30
    assert sure.any()
    got, got_lse = run_loss(h)
    assert (got[sure] == 0).all() and (got >= 0).all()
    assert ((got_lse.to(F64) - lse).abs() <= product_error(h) + 2.0 ** -18 + 2.0 ** -23 * lse.abs()).all()


@pytest.mark.parametrize("tokens,vocab,hidden,cta_group", LOSS_FORMS)
def test_infinities_in_rows_that_count(tokens, vocab, hidden, cta_group):
    tkg.set_option(tkg.OPT_CTA_GROUP, cta_group)
    clean = Head(tokens, vocab, hidden, ignored=0.0, seed=23)
    want, want_lse = run_loss(clean)
    for where in ("one", "all"):
        h = Head(tokens, vocab, hidden, ignored=0.0, seed=23)
        at = tokens // 2
        h.W[:, 0] = torch.where(h.W[:, 0] == 0, torch.ones_like(h.W[:, 0]), h.W[:, 0])
        if where == "all":   # every logit of the token -inf: nothing to sum
            h.W[:, 0] = -h.W[:, 0].abs()
            h.X[at] = 0
        h.X[at, 0] = float("inf")
        z = h.X[at].to(F64) * h.W.to(F64)
        z = torch.where((h.X[at] == 0)[None, :], torch.zeros_like(z), z).sum(dim=1)
        lse = torch.logsumexp(z, 0)
        loss = lse - z[h.y[at]]
        got, got_lse = run_loss(h)
        assert torch.equal(torch.nan_to_num(got_lse[at].to(F64), nan=0.5, posinf=2.0, neginf=-2.0),
                           torch.nan_to_num(lse, nan=0.5, posinf=2.0, neginf=-2.0))
        assert torch.equal(torch.nan_to_num(got[at].to(F64), nan=0.5, posinf=2.0, neginf=-2.0),
                           torch.nan_to_num(loss, nan=0.5, posinf=2.0, neginf=-2.0))
        if where == "one":
            rest = torch.arange(tokens, device="cuda") != at
            assert torch.equal(got[rest], want[rest]) and torch.equal(got_lse[rest], want_lse[rest])


# forms of the gradient's logits: wide, narrow, and both with sums in parts
GRAD_FORMS = [(40, 700, 264), (300, 1500, 64), (20, 20003, 256), (20, 20003, 1024), (40, 20000, 4096), (40, 20000, 4104),
              (300, 700, 4104), (130, 900, 8200)]


@pytest.mark.parametrize("tokens,vocab,hidden", [(1, 19713, 768), (32, 20003, 768), (40, 21648, 1032), (70, 19800, 2056),
                                                 (128, 24000, 4096)])
def test_gradient_in_the_narrow_form(tokens, vocab, hidden):
    check_grad(Head(tokens, vocab, hidden, seed=26))
    check_grad(Head(tokens, vocab, hidden, seed=27, alpha=-0.5, ignored=0.9), dtype=F32)


@pytest.mark.parametrize("alpha", [1.0, -0.5, 0.37])
@pytest.mark.parametrize("tokens,vocab,hidden", GRAD_FORMS)
def test_gradient_of_tokens_the_model_is_sure_of(tokens, vocab, hidden, alpha):
    """Where lse is the label's own logit, g is exactly 0 there: what a sure token gives to dX and its label's row of dW
    is the other logits' exponentials, here below e^-30.  (10% of them: logits off by 2^-7 in the worst case.)"""
    tkg.set_option(tkg.OPT_CTA_GROUP, 2)   # logits of the same kernel for the loss of few tokens
    h = Head(tokens, vocab, hidden, alpha=alpha, ignored=0.0, seed=24, spread=1e-3)
    h.y = torch.randperm(vocab, device="cuda")[:tokens]
    scale = 2.0 ** round(7.5 - torch.log2(torch.tensor(abs(alpha) * hidden)).item())
    h.W[h.y] = (h.X.float() * (scale if alpha > 0 else -scale)).to(BF16)   # logits of about 128 to 256
    z, _, lse, _, _ = h.forward()
    loss, got_lse = run_loss(h)
    others = torch.exp(z - lse[:, None]).scatter(1, h.y[:, None], 0.0)
    sure = (loss == 0) & (others.sum(dim=1) < 2.0 ** -30)
    assert sure.any()
    dX, dW = run_grad(h, got_lse, dtype=F32)
    w = (h.dloss.to(F64) * abs(alpha))[:, None]
    # an ulp of BF16 for g, another for the weighted rows and the result
    boundX = 1.1 * (w * others) @ h.W.to(F64).abs() + 1e-30
    boundW = 1.1 * (w * others).T @ h.X.to(F64).abs() + 1e-30
    # a token that is not sure has a g of its own in its label's row only
    assert (dX[sure].to(F64).abs() <= boundX[sure]).all()
    assert (dW[h.y[sure]].to(F64).abs() <= boundW[h.y[sure]]).all()


def test_a_very_wide_head():
    # more rows of dX's parts than one grid dimension past the first has blocks
    tokens, vocab, hidden = 3, 9, 16 * 65536 + 8
    h = Head(tokens, vocab, hidden, ignored=0.0, seed=25)
    z, _, lse, loss, _ = h.forward()
    got, got_lse = run_loss(h)
    tol = product_error(h) + 2.0 ** -18 + 2.0 ** -23 * lse.abs()
    assert ((got_lse.to(F64) - lse).abs() <= tol).all() and ((got.to(F64) - loss).abs() <= 2 * tol).all()
    dX, eX, (gX, gW) = *(h.gradient()[i] for i in (0, 2)), run_grad(h, lse.float())
    assert ((gX.to(F64) - dX).abs() <= eX).all()
