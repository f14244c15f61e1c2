"""Softmax cross entropy of a linear head over a large vocabulary and its
gradient (tkg_linear_ce_loss, tkg_linear_ce_grad) against the definition in 64
bits, at the sizes, labels, layouts and values where they can go wrong.

Tolerances, element by element, from the roundings the operators make:
 - a logit: FP32 accumulation of exact products, at most 1e-5 * |alpha| * sum_h |x w|
   (the library's acceptance bound for its products);
 - lse moves by no more than its logits do, plus the FP32 rounding of exponents
   of up to 2^8 in base 2 and of a sum of exponentials (together under 1e-4 at
   these sizes, and 2^-22 of its own size); loss by twice that;
 - exp(z - lse): a relative error of its exponent's absolute error;
 - g is rounded to BF16 (2^-8), and where a token's weight dloss is folded into
   its row of X for dW, that row once more (2^-8);
 - a BF16 result: 2^-8 of itself; FP32 accumulation of g W and g^T X: 1e-5 of the
   sum of magnitudes."""
import numpy as np
import pytest
import torch

from dense_block_scaled_gb300 import tkg

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0 ** -8


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK
    tkg.set_option(tkg.OPT_BF16_TILE_N, 0)
    tkg.set_option(tkg.OPT_CTA_GROUP, 0)


class Head:
    """Seeded operands of a head and everything the definition says about them, in 64 bits."""

    def __init__(self, tokens, vocab, hidden, alpha=1.0, ignored=0.2, seed=0, spread=2.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 7919 + tokens * 31 + vocab * 17 + hidden)
        self.shape, self.alpha = (tokens, vocab, hidden), alpha
        self.X = torch.randn(tokens, hidden, generator=g, device="cuda").to(BF16)
        scale = spread / (hidden ** 0.5 * max(abs(alpha), 0.1))
        self.W = (torch.randn(vocab, hidden, generator=g, device="cuda") * scale).to(BF16)
        y = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        y[torch.rand(tokens, generator=g, device="cuda") < ignored] = -100
        self.y = y
        self.dloss = (torch.rand(tokens, generator=g, device="cuda") + 0.1) / tokens

    def forward(self):
        _, vocab, _ = self.shape
        z = self.alpha * (self.X.to(F64) @ self.W.to(F64).T)
        kept = (self.y >= 0) & (self.y < vocab)
        lse = torch.logsumexp(z, dim=1)
        loss = torch.where(kept, lse - z.gather(1, self.y.clamp(0, vocab - 1)[:, None])[:, 0], torch.zeros_like(lse))
        dz = 1e-5 * abs(self.alpha) * (self.X.to(F64).abs() @ self.W.to(F64).abs().T).max(dim=1).values
        return z, kept, lse, loss, dz + 1e-4 + 2.0 ** -22 * lse.abs()

    def gradient(self):
        """dX, dW and their element-wise bounds (BF16 outputs)."""
        tokens, vocab, _ = self.shape
        z, kept, lse, _, tol = self.forward()
        p = torch.exp(z - lse[:, None])
        w = torch.where(kept, self.dloss.to(F64) * self.alpha, torch.zeros_like(lse))[:, None]
        hot = torch.nn.functional.one_hot(self.y.clamp(0, vocab - 1), vocab).to(F64)
        g = w * (p - hot)
        eg = g.abs() * (U + 1e-5) + w.abs() * p * 2 * tol[:, None]
        Xk = torch.where(kept[:, None], self.X.to(F64), torch.zeros_like(self.X, dtype=F64))
        Wd = self.W.to(F64)
        dX, dW = g @ Wd, g.T @ Xk
        eX = eg @ Wd.abs() + U * dX.abs() + 1e-30
        eW = eg.T @ Xk.abs() + U * (g.abs().T @ Xk.abs()) + 1e-30
        return dX, dW, eX, eW


def run_loss(h, X=None, W=None, **kw):
    loss = torch.full((h.shape[0],), 7.0, device="cuda")
    lse = torch.full((h.shape[0],), 7.0, device="cuda")
    tkg.linear_ce_loss(h.X if X is None else X, h.W if W is None else W, h.y, loss, lse, alpha=h.alpha, **kw)
    return loss, lse


def run_grad(h, lse, dtype=BF16, dX=True, dW=True, **kw):
    t, v, d = h.shape
    dX = torch.full((t, d), 7.0, device="cuda", dtype=BF16) if dX else None
    dW = torch.full((v, d), 7.0, device="cuda", dtype=dtype) if dW else None
    tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, dX, dW, alpha=h.alpha, **kw)
    return dX, dW


def within(got, ref, bound, what):
    err = (got.to(F64) - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float((err / bound).max()):.3g} bounds"


def check_loss(h, **kw):
    _, kept, lse, loss, tol = h.forward()
    got_loss, got_lse = run_loss(h, **kw)
    within(got_lse, lse, tol, f"lse {h.shape}")
    within(got_loss, loss, 2 * tol, f"loss {h.shape}")
    assert (got_loss[~kept] == 0).all()
    return got_lse


def check_grad(h, lse=None, dtype=BF16, **kw):
    if lse is None:
        lse = h.forward()[2].float()
    dX, dW, eX, eW = h.gradient()
    gX, gW = run_grad(h, lse, dtype=dtype, **kw)
    if gX is not None:
        within(gX, dX, eX, f"dX {h.shape}")
    if gW is not None:
        within(gW, dW, eW + (0 if dtype == F32 else U * dW.abs()), f"dW {h.shape}")
    return gX, gW


SHAPES = [
    (1, 1, 8), (1, 2, 64), (2, 255, 72), (16, 256, 64), (17, 257, 264), (31, 1000, 128), (32, 129, 8),
    (100, 4999, 512), (127, 128, 64), (128, 300, 1032), (129, 1025, 264), (200, 777, 136), (255, 2049, 320),
    (256, 512, 512), (257, 511, 1024), (385, 6001, 256), (777, 5001, 512), (1, 40000, 256), (1030, 3333, 192),
]


@pytest.mark.parametrize("tokens,vocab,hidden", SHAPES)
def test_loss_matches_definition(tokens, vocab, hidden):
    check_loss(Head(tokens, vocab, hidden))


@pytest.mark.parametrize("tokens,vocab,hidden", SHAPES)
def test_grad_matches_definition(tokens, vocab, hidden):
    check_grad(Head(tokens, vocab, hidden))


@pytest.mark.parametrize("tokens,vocab,hidden", [(40, 300, 2048), (40, 300, 2056), (128, 1001, 4096), (100, 300, 4104),
                                                 (130, 700, 2056), (300, 20000, 4104), (129, 400, 12296)])
def test_loss_of_long_sums(tokens, vocab, hidden):
    check_loss(Head(tokens, vocab, hidden, seed=8))
    check_loss(Head(tokens, vocab, hidden, seed=9, alpha=-0.5))


@pytest.mark.parametrize("tokens,vocab,hidden", [(5, 19713, 64), (17, 20001, 4096), (40, 20000, 2056), (64, 33333, 264),
                                                 (65, 20000, 264), (128, 20000, 4104), (33, 40000, 2048)])
def test_loss_of_few_tokens_and_many_entries(tokens, vocab, hidden):
    check_loss(Head(tokens, vocab, hidden, seed=11))
    check_loss(Head(tokens, vocab, hidden, seed=12, alpha=-0.5, ignored=0.9))


@pytest.mark.parametrize("tokens,vocab,hidden,piece", [(5, 19713, 64, 0), (40, 20000, 264, 0), (64, 25000, 136, 20000),
                                                       (128, 20000, 72, 0), (1, 19999, 520, 0)])
def test_grad_of_few_tokens_and_many_entries(tokens, vocab, hidden, piece):
    check_grad(Head(tokens, vocab, hidden, seed=13), piece=piece)
    check_grad(Head(tokens, vocab, hidden, seed=14, alpha=-0.5, ignored=0.9), dtype=F32, piece=piece)


@pytest.mark.parametrize("tokens", [7, 200])
def test_long_sums_keep_their_precision(tokens):
    """Products of one sign, 16384 of them: the accumulator loses less than 2^-23 of itself at each of the 128 steps of
    16 products that it takes, and is half of its sum on average, so less than 2^-17 in all; the sums' additions and lse
    come to less than 2^-20."""
    h = Head(tokens, 300, 16384, seed=10, ignored=0.0)
    h.X, h.W = h.X.abs(), h.W.abs() / 64
    z, _, lse, loss, _ = h.forward()
    got_loss, got_lse = run_loss(h)
    zmax = z.max(dim=1).values
    within(got_lse, lse, (2.0 ** -17 + 2.0 ** -20) * zmax.clamp(min=1.0) + 2.0 ** -20 * lse.abs(), "lse")
    within(got_loss, loss, 2 * (2.0 ** -17 + 2.0 ** -20) * zmax.clamp(min=1.0) + 2.0 ** -19 * lse.abs(), "loss")


@pytest.mark.parametrize("cta_group", [0, 2])   # 2: tensor cores for few tokens too
@pytest.mark.parametrize("tokens,vocab,hidden", [(1, 5000, 2056), (2, 31, 8), (3, 777, 136), (4, 1001, 4104), (5, 33, 264),
                                                 (6, 4097, 520), (7, 10000, 1024), (8, 2049, 2048), (8, 300, 2056),
                                                 (1, 9, 16640), (9, 600, 256)])
def test_loss_of_few_tokens(tokens, vocab, hidden, cta_group):
    tkg.set_option(tkg.OPT_CTA_GROUP, cta_group)
    check_loss(Head(tokens, vocab, hidden, seed=5, ignored=0.1))
    check_loss(Head(tokens, vocab, hidden, seed=6, alpha=-0.5))
    check_loss(Head(tokens, vocab, hidden, seed=7, alpha=0.0))


@pytest.mark.parametrize("tile_n", [256, 512])
@pytest.mark.parametrize("tokens,vocab,hidden,piece", [(5, 333, 64, 0), (130, 700, 264, 0), (300, 1300, 128, 512),
                                                       (777, 900, 1032, 0), (1100, 2100, 520, 1000)])
def test_both_tile_widths(tokens, vocab, hidden, piece, tile_n):
    tkg.set_option(tkg.OPT_BF16_TILE_N, tile_n)
    h = Head(tokens, vocab, hidden, seed=1)
    lse = check_loss(h)
    check_grad(h, lse, piece=piece)
    _, g = check_grad(h, lse, dtype=F32, piece=piece)
    acc = torch.ones_like(g)
    tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, None, acc, alpha=h.alpha, accumulate=True, piece=piece)
    assert torch.equal(acc, 1 + g)


def test_no_tile_is_missed_in_many_launches():
    # back to back on every SM: the roles of a cluster agree on every tile they take over (a role that once read a
    # scheduler answer late missed one in about a hundred of these launches, which then ran into the wait limit)
    h = Head(1333, 50001, 512, ignored=0.0)
    lse = h.forward()[2].float()
    dW = torch.empty_like(h.W)
    first = run_grad(h, lse, dX=False)[1]
    try:
        tkg.set_option(tkg.OPT_TIMEOUT_MS, 200)
        for _ in range(1500):
            tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, None, dW, alpha=h.alpha)
        assert tkg.device_status() == tkg.OK
    finally:
        tkg.set_option(tkg.OPT_TIMEOUT_MS, 0)
    assert torch.equal(dW, first)


@pytest.mark.parametrize("alpha", [-0.5, 0.0, 3.0, 1e-3])
def test_scales(alpha):
    h = Head(70, 900, 128, alpha=alpha)
    check_grad(h, check_loss(h))


@pytest.mark.parametrize("spread", [30.0, 1e-3])
def test_wide_and_flat_logits(spread):
    # spread 30: logits to +-100, most probabilities below the least float; 1e-3: nearly uniform
    h = Head(65, 3000, 256, spread=spread)
    check_grad(h, check_loss(h))


def test_equal_logits():
    h = Head(9, 1000, 64, ignored=0.0)
    h.W[:] = h.W[0]
    got = check_loss(h)
    assert torch.allclose(run_loss(h)[0], torch.full((9,), float(np.log(1000.0)), device="cuda"), atol=1e-4)
    check_grad(h, got)


@pytest.mark.parametrize("piece", [1, 64, 256, 300, 1000, 5000])
def test_pieces(piece):
    h = Head(140, 1500, 136, seed=2)
    if piece == 1:   # 1500 pieces of one entry: a smaller vocabulary
        h = Head(140, 20, 136, seed=2)
    check_grad(h, piece=piece)


@pytest.mark.parametrize("tokens", [3, 600])
@pytest.mark.parametrize("want", ["dX", "dW"])
def test_one_gradient_alone(tokens, want):
    h = Head(tokens, 1111, 128)
    gX, gW = check_grad(h, dX=want == "dX", dW=want == "dW")
    assert (gX is None) == (want == "dW") and (gW is None) == (want == "dX")


@pytest.mark.parametrize("piece", [0, 512])
def test_f32_weight_gradient_and_accumulation(piece):
    h = Head(300, 1301, 136, seed=3)
    lse = h.forward()[2].float()
    _, g = check_grad(h, lse, dtype=F32, piece=piece)
    dX = torch.empty(300, 136, device="cuda", dtype=BF16)
    acc = torch.randn(1301, 136, device="cuda")
    before = acc.clone()
    tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, dX, acc, alpha=h.alpha, accumulate=True, piece=piece)
    # one FP32 addition to what was there
    assert torch.equal(acc, before + g)


def test_labels_at_the_edges_and_outside():
    h = Head(12, 1000, 64, ignored=0.0)
    h.y[:] = torch.tensor([0, 999, 1000, -1, 2 ** 40, -2 ** 40, 127, 128, 255, 256, 511, 512], device="cuda")
    check_grad(h, check_loss(h))


def test_all_rows_ignored():
    h = Head(150, 600, 64)
    h.y[:] = -100
    loss, lse = run_loss(h)
    assert (loss == 0).all()
    gX, gW = run_grad(h, lse)
    assert (gX == 0).all() and (gW == 0).all()
    keep = torch.randn(600, 64, device="cuda")
    acc = keep.clone()
    tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, None, acc, accumulate=True)
    assert torch.equal(acc, keep)


@pytest.mark.parametrize("tokens", [7, 20, 333])
def test_ignored_rows_may_hold_anything(tokens):
    clean = Head(tokens, 800, 128, ignored=0.5)
    lse = clean.forward()[2].float()
    want = run_grad(clean, lse) + run_loss(clean)[:1]
    gone = ~(clean.y >= 0)
    assert gone.any() and not gone.all()
    for bad in (float("nan"), float("inf"), torch.finfo(BF16).min):
        h = Head(tokens, 800, 128, ignored=0.5)
        h.X[gone] = bad
        h.dloss[gone] = float("nan")
        l2 = torch.where(gone, torch.full_like(lse, float("nan")), lse)
        gX, gW = run_grad(h, l2)
        assert torch.equal(gX, want[0]) and torch.equal(gW, want[1])
        assert torch.equal(run_loss(h)[0], want[2])


def test_zero_weights():
    h = Head(40, 500, 64, ignored=0.0)
    h.dloss[:] = 0
    gX, gW = run_grad(h, h.forward()[2].float())
    assert (gX == 0).all() and (gW == 0).all()


def test_uneven_and_tiny_weights():
    h = Head(64, 700, 128, ignored=0.1)
    h.dloss *= torch.logspace(-12, 3, 64, device="cuda")
    check_grad(h)


def test_row_pitches():
    h = Head(75, 650, 136)
    lse = h.forward()[2].float()
    want = run_grad(h, lse) + run_loss(h)
    Xp = torch.full((75, 160), float("nan"), device="cuda", dtype=BF16)
    Wp = torch.full((650, 144), float("nan"), device="cuda", dtype=BF16)
    Xp[:, :136], Wp[:, :136] = h.X, h.W
    h.X, h.W = Xp[:, :136], Wp[:, :136]
    got_loss = run_loss(h)
    dXp = torch.full((75, 200), 7.0, device="cuda", dtype=BF16)
    dWp = torch.full((650, 184), 7.0, device="cuda", dtype=BF16)
    tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, dXp[:, :136], dWp[:, :136], alpha=h.alpha)
    for a, b in zip((dXp[:, :136], dWp[:, :136]) + got_loss, want):
        assert torch.equal(a, b)
    assert (dXp[:, 136:] == 7).all() and (dWp[:, 136:] == 7).all()


def test_same_bits_every_time():
    h = Head(500, 9001, 256)
    lse = h.forward()[2].float()
    first = run_grad(h, lse) + run_loss(h)
    for _ in range(3):
        again = run_grad(h, lse) + run_loss(h)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_differences():
    # directional derivatives of sum(dloss * loss) by central differences in 64 bits
    h = Head(50, 600, 64)
    lse = h.forward()[2].float()
    _, _, eX, eW = h.gradient()
    gX, gW = run_grad(h, lse)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    dX, dW = (torch.randn(s, generator=gen, device="cuda", dtype=F64) for s in (h.X.shape, h.W.shape))

    def total(X, W):
        z = h.alpha * (X @ W.T)
        kept = h.y >= 0
        loss = torch.logsumexp(z, 1) - z.gather(1, h.y.clamp(0)[:, None])[:, 0]
        return float((torch.where(kept, loss, torch.zeros_like(loss)) * h.dloss.to(F64)).sum())

    X, W, eps = h.X.to(F64), h.W.to(F64), 1e-5
    for got, bound, step, at in ((gX, eX, dX, lambda s: total(X + s * dX, W)),
                                 (gW, eW + U * gW.to(F64).abs(), dW, lambda s: total(X, W + s * dW))):
        diff = (at(eps) - at(-eps)) / (2 * eps)
        assert abs(float((got.to(F64) * step).sum()) - diff) <= float((bound * step.abs()).sum()) + 1e-7


def test_other_stream_and_own_workspace():
    h = Head(90, 2000, 128)
    lse = h.forward()[2].float()
    want = run_grad(h, lse) + run_loss(h)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [torch.zeros(90, device="cuda"), torch.zeros(90, device="cuda"),
            torch.zeros(90, 128, device="cuda", dtype=BF16), torch.zeros(2000, 128, device="cuda", dtype=BF16)]
    ws = torch.empty(max(tkg.linear_ce_loss_workspace_bytes(90, 2000),
                         tkg.linear_ce_grad_workspace_bytes(90, 2000, 128)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for workspace in (ws, None):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        tkg.linear_ce_loss(h.X, h.W, h.y, outs[0], outs[1], alpha=h.alpha, workspace=workspace, stream=s)
        tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, outs[2], outs[3], alpha=h.alpha, workspace=workspace, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, (want[2], want[3], want[0], want[1])))


def test_workspace_bounds():
    # nothing outside the stated workspace is written, and its contents do not matter
    for tokens, vocab, hidden, piece in [(33, 1000, 64, 0), (300, 900, 136, 256)]:
        h = Head(tokens, vocab, hidden)
        lse = h.forward()[2].float()
        want = run_grad(h, lse, piece=piece) + run_loss(h)
        for fill in (0, 255):
            for call, nbytes in (("loss", tkg.linear_ce_loss_workspace_bytes(tokens, vocab)),
                                 ("grad", tkg.linear_ce_grad_workspace_bytes(tokens, vocab, hidden, piece))):
                room = torch.full((nbytes + 512,), fill, dtype=torch.uint8, device="cuda")
                ws = room[256:256 + nbytes]
                got = run_loss(h, workspace=ws) if call == "loss" else run_grad(h, lse, piece=piece, workspace=ws)
                assert (room[:256] == fill).all() and (room[256 + nbytes:] == fill).all()
                assert all(torch.equal(a, b) for a, b in zip(got, want[2:] if call == "loss" else want[:2]))


def test_graph_capture_and_replay():
    h = Head(64, 1500, 128, ignored=0.0)
    lse = h.forward()[2].float()
    loss, l2 = run_loss(h)
    dX, dW = run_grad(h, lse)
    ws = torch.empty(max(tkg.linear_ce_loss_workspace_bytes(64, 1500),
                         tkg.linear_ce_grad_workspace_bytes(64, 1500, 128)), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tkg.linear_ce_loss(h.X, h.W, h.y, loss, l2, alpha=h.alpha, workspace=ws)
        tkg.linear_ce_grad(h.X, h.W, h.y, l2, h.dloss, dX, dW, alpha=h.alpha, workspace=ws)
    other = Head(64, 1500, 128, ignored=0.0, seed=9)
    h.X.copy_(other.X), h.W.copy_(other.W), h.y.copy_(other.y), h.dloss.copy_(other.dloss)
    graph.replay()
    torch.cuda.synchronize()
    wl, wlse = run_loss(other)
    wX, wW = run_grad(other, wlse)
    assert torch.equal(loss, wl) and torch.equal(l2, wlse) and torch.equal(dX, wX) and torch.equal(dW, wW)


def test_no_tokens():
    h = Head(1, 300, 64)
    empty = torch.empty(0, 64, device="cuda", dtype=BF16)
    y, f = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    tkg.linear_ce_loss(empty, h.W, y, f, f.clone())
    dW = torch.full((300, 64), 7.0, device="cuda")
    tkg.linear_ce_grad(empty, h.W, y, f, f, None, dW, accumulate=True)
    assert (dW == 7).all()
    tkg.linear_ce_grad(empty, h.W, y, f, f, None, dW)
    assert (dW == 0).all()


def test_offsets_past_32_bits():
    # a head of 4.7 GB: its last rows count, and its gradient is written to the end
    tokens, vocab, hidden = 5, 143000, 16384
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    X = torch.randn(tokens, hidden, generator=g, device="cuda").to(BF16)
    W = torch.empty(vocab, hidden, device="cuda", dtype=BF16)
    for v0 in range(0, vocab, 8192):
        n = min(8192, vocab - v0)
        W[v0:v0 + n] = (torch.randn(n, hidden, generator=g, device="cuda") * (2.0 / 128)).to(BF16)
    y = torch.tensor([vocab - 1, 0, vocab - 2, 131072, -1], device="cuda")
    loss, lse = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
    tkg.linear_ce_loss(X, W, y, loss, lse)
    z = torch.cat([X.to(F64) @ W[v0:v0 + 8192].to(F64).T for v0 in range(0, vocab, 8192)], dim=1)
    want = torch.logsumexp(z, 1)
    tol = 1e-5 * 16384 * 2 / 128 + 1e-4   # sum |x w| is about hidden * (2 / 128) * 2 / pi
    assert ((lse.to(F64) - want).abs() <= tol).all()
    picked = want - z.gather(1, y.clamp(0)[:, None])[:, 0]
    picked[4] = 0
    assert ((loss.to(F64) - picked).abs() <= 2 * tol).all()
    dloss = torch.full((tokens,), 0.25, device="cuda")
    dX = torch.empty_like(X)
    dW = torch.full((vocab, hidden), 7.0, device="cuda", dtype=BF16)
    tkg.linear_ce_grad(X, W, y, want.float(), dloss, dX, dW)
    gr = torch.exp(z - want[:, None])
    gr[torch.arange(4, device="cuda"), y[:4]] -= 1
    gr *= 0.25
    gr[4] = 0
    for rows in (slice(0, 300), slice(131000, 131300), slice(vocab - 300, vocab)):
        ref = gr[:, rows].T @ X.to(F64)
        bound = (2 * U + 4 * tol) * (gr[:, rows].abs().T @ X.to(F64).abs()) + U * ref.abs() + 1e-12
        within(dW[rows], ref, bound, f"dW rows {rows}")
    ref = sum(gr[:, v0:v0 + 8192] @ W[v0:v0 + 8192].to(F64) for v0 in range(0, vocab, 8192))
    mag = sum(gr[:, v0:v0 + 8192].abs() @ W[v0:v0 + 8192].to(F64).abs() for v0 in range(0, vocab, 8192))
    within(dX, ref, (U + 4 * tol) * mag + U * ref.abs() + 1e-12, "dX")


def test_refusals():
    h = Head(8, 100, 64)
    loss, lse = run_loss(h)
    dX, dW = torch.empty_like(h.X), torch.empty_like(h.W)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(tkg.TkgError) as e:
        tkg.linear_ce_loss(h.X, h.W, h.y, loss, lse, workspace=small)
    assert e.value.status == tkg.ERR_INVALID_ARG
    with pytest.raises(tkg.TkgError) as e:
        tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, dX, dW, workspace=small)
    assert e.value.status == tkg.ERR_INVALID_ARG
    with pytest.raises(tkg.TkgError) as e:   # 60 elements a row
        tkg.linear_ce_loss(h.X[:, :60], h.W[:, :60], h.y, loss, lse)
    assert e.value.status == tkg.ERR_ALIGNMENT
    with pytest.raises(tkg.TkgError) as e:   # a first element 2 bytes off
        tkg.linear_ce_loss(h.X[:, 1:57], h.W[:, :56], h.y, loss, lse)
    assert e.value.status == tkg.ERR_ALIGNMENT
    for bad in (dict(X=h.X.float()), dict(W=h.W[:, :56]), dict(labels=h.y.int()), dict(loss=loss[:4]),
                dict(X=torch.empty(64, 8, device="cuda", dtype=BF16).T)):
        args = dict(X=h.X, W=h.W, labels=h.y, loss=loss, lse=lse)
        args.update(bad)
        with pytest.raises(ValueError):
            tkg.linear_ce_loss(**args)
    with pytest.raises(ValueError):   # accumulation is FP32's
        tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss, dX, dW, accumulate=True)
    with pytest.raises(ValueError):
        tkg.linear_ce_grad(h.X, h.W, h.y, lse, h.dloss.double(), dX, dW)


def test_stall_times_out_and_recovers():
    h = Head(200, 700, 128)
    lse = h.forward()[2].float()
    try:
        tkg.set_option(tkg.OPT_TIMEOUT_MS, 100)
        tkg.set_option(tkg.OPT_INJECT_STALL, 1)
        run_loss(h)
        assert tkg.device_status() == tkg.ERR_TIMEOUT
        run_grad(h, lse)
        assert tkg.device_status() == tkg.ERR_TIMEOUT
    finally:
        tkg.set_option(tkg.OPT_INJECT_STALL, 0)
        tkg.set_option(tkg.OPT_TIMEOUT_MS, 0)
    check_grad(h, check_loss(h))
