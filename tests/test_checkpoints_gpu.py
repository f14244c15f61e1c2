"""8-bit checkpoints (tkg_checkpoint_mxfp8), the gated activation with one and its gradient from it (tkg_swiglu,
tkg_swiglu_grad), and weight gradients from checkpoints (tkg_gemm_grouped_dev_mxfp8_wgrad).

Tolerances.  Codes and scales are a rule's: equal.  sigma is two approximations of 1 ulp and three roundings, one of them
of an exponent up to 20 here (2^-20 of sigma in all), and a product of up to five such factors keeps 2^-18; BF16 results are
rounded once (half a step: 2^-8).  dweights sums up to 2048 columns in FP32, at most 88 additions deep (one lane's 64 or
8 x 8 and the joins): 2^-17 of the sum of sizes.  The product's bound is the library's own."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg

pytestmark = pytest.mark.gpu
BF16, F32, F64, I32, U8 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.uint8
GUARD = 7.0


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


def normal(*shape, seed=0, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 101 + sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def rule(X):
    """Codes and scales by the definition, in 64 bits."""
    b = X.to(F64).unflatten(1, (-1, 32))
    amax = b.abs().amax(dim=2)
    e = torch.where(amax > 0, torch.ceil(torch.log2(amax / 448)), -127.0)
    e = torch.where(448 * torch.exp2(e - 1) >= amax, e - 1, e)      # (log2's rounding)
    e = torch.where(448 * torch.exp2(e) < amax, e + 1, e).clamp(-127, 127)
    q = (b * torch.exp2(-e)[..., None]).to(F32).to(torch.float8_e4m3fn)
    return q.flatten(1).view(U8), (e + 127).to(U8)


def values(Q, sf, dtype=F64):
    return (Q.view(torch.float8_e4m3fn).to(dtype).unflatten(1, (-1, 32)) * torch.exp2(sf.to(dtype) - 127)[..., None]).flatten(1)


def save(X):
    Q, sf = torch.empty(X.shape, dtype=U8, device="cuda"), torch.empty(X.shape[0], X.shape[1] // 32, dtype=U8, device="cuda")
    tkg.checkpoint_mxfp8(X, Q, sf)
    return Q, sf


@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (1, 4096), (100, 256), (257, 288), (64, 2048), (1000, 1312)])
@pytest.mark.parametrize("pad", [0, 8])
def test_saved_rows(rows, k, pad):
    X = normal(rows, k + pad)[:, :k]
    X *= torch.exp2(torch.randint(-30, 30, (rows, 1), device="cuda").to(F32)).to(BF16)
    X[:, :32] = 0                                                    # a block of zeros
    Q, sf = save(X)
    q, s = rule(X)
    assert torch.equal(Q, q) and torch.equal(sf, s)
    assert ((values(Q, sf) - X.to(F64)).abs() <= 2.0 ** -4 * X.to(F64).abs() + 2.0 ** -10 * torch.exp2(sf.to(F64) - 127).repeat_interleave(32, 1)).all()


def test_same_rule_as_the_quantiser():
    X = normal(130, 256, seed=4)
    Q, sf = save(X)
    q = torch.empty_like(Q)
    tiled, want = (torch.empty(tkg.scale_bytes(130, 256, 32), dtype=U8, device="cuda") for _ in range(2))
    tkg.quantize_mxfp8(X.float(), q, want)
    tkg.scales_to_tiled(sf, tiled)
    assert torch.equal(Q, q) and torch.equal(tiled, want)


def test_saved_extremes():
    X = torch.zeros(6, 32, device="cuda", dtype=BF16)
    X[0, 3] = float("nan")
    X[0, 4] = 1.0
    X[1, 0] = float("inf")
    X[2] = 2.0 ** -133                                               # the smallest BF16
    X[3, 1], X[3, 2] = 448.0, -2.0 ** -4
    X[4, 1] = 450.0
    Q, sf = save(X)
    got = values(Q, sf, F32)
    assert got[0, 3].isnan() and got[0, 4] == 1.0
    assert got[1, 0] == float("inf") and (got[1, 1:] == 0).all()
    assert (got[2] == 2.0 ** -133).all() and sf[2] == 0               # code 2^-6, scale 2^-127
    assert got[3, 1] == 448.0 and got[3, 2] == -2.0 ** -4 and sf[3] == 127
    assert sf[4] == 128 and got[4, 1] == 448.0


def h_of(x):
    g, u = x.chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


@pytest.mark.parametrize("rows,inner", [(1, 32), (1, 2048), (5, 8), (33, 264), (100, 1408), (3, 7168), (1000, 256)])
@pytest.mark.parametrize("pad", [0, 8])
def test_activation(rows, inner, pad):
    X = normal(rows, 2 * inner + pad)[:, :2 * inner] * 2
    H = torch.full((rows + 1, inner + pad), GUARD, device="cuda", dtype=BF16)
    tkg.swiglu(X, H[:rows, :inner])
    ref = h_of(X.to(F64))
    assert ((H[:rows, :inner].to(F64) - ref).abs() <= (2.0 ** -8 + 2.0 ** -18) * ref.abs()).all()
    assert (H[rows:] == GUARD).all() and (H[:, inner:] == GUARD).all()
    if inner % 32 == 0:
        H2 = torch.empty(rows, inner, device="cuda", dtype=BF16)
        Q, sf = torch.empty(rows, 2 * inner, device="cuda", dtype=U8), torch.empty(rows, inner // 16, device="cuda", dtype=U8)
        tkg.swiglu(X, H2, Q, sf)
        assert torch.equal(H2, H[:rows, :inner])
        q, s = rule(X)
        assert torch.equal(Q, q) and torch.equal(sf, s)


def test_activation_of_extremes():
    g = torch.tensor([0.0, -0.0, 60.0, -60.0, -87.0, -88.5, -100.0, 3e38, -3e38, float("inf"), float("nan")], device="cuda")
    X = torch.ones(2 * len(g), 16, device="cuda", dtype=BF16)
    X[:len(g), :8] = g[:, None].to(BF16)
    H = torch.empty(2 * len(g), 8, device="cuda", dtype=BF16)
    tkg.swiglu(X, H)
    ref = h_of(X.to(F64))
    got = H.to(F64)
    assert torch.equal(got.isnan(), ref.isnan())
    # below 2^-126 a sigma is subnormal: the approximations may flush or round it, at most 2^-126 times g
    ok = (got - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs() + 2.0 ** -126 * X[:, :8].to(F64).abs()
    assert (ok | ref.isnan() | (got == ref)).all()


class Grad:
    def __init__(self, rows, inner, choices=None, weighted=True, gone=0.0, pad=0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + rows * 3 + inner)
        self.rows, self.inner = rows, inner
        self.Q, self.sf = save(normal(rows, 2 * inner, seed=seed + 1))
        self.dH = normal(rows, inner + pad, seed=seed + 2)[:, :inner]
        n = rows + 3 if choices is None else choices
        self.slots = torch.randperm(max(n, rows), generator=g, device="cuda")[:rows].to(I32)   # some past the weights
        self.slots[torch.rand(rows, generator=g, device="cuda") < gone] = -1
        self.w = torch.rand(n, generator=g, device="cuda") * 2 - 0.5 if weighted else None
        self.there = (self.slots >= 0) & (self.slots < n) if weighted else self.slots >= 0
        self.pad = pad

    def run(self, with_h=True):
        r, i, p = self.rows, self.inner, self.pad
        dX = torch.full((r + 1, 2 * i + p), GUARD, device="cuda", dtype=BF16)
        H = torch.full((r + 1, i + p), GUARD, device="cuda", dtype=BF16) if with_h else None
        dw = torch.full_like(self.w, GUARD) if self.w is not None else None
        tkg.swiglu_grad(self.Q, self.sf, self.dH, dX[:r, :2 * i], H[:r, :i] if with_h else None, slots=self.slots,
                        weights=self.w, dweights=dw)
        for t in (dX,) + ((H,) if with_h else ()):
            assert (t[r:] == GUARD).all() and (t[:r][~self.there] == GUARD).all()
            if p:
                assert (t[:, -p:] == GUARD).all()
        return dX[:r, :2 * i], H[:r, :i] if with_h else None, dw

    def reference(self):
        x = values(self.Q, self.sf).requires_grad_(True)
        w = torch.ones(self.rows, dtype=F64, device="cuda")
        if self.w is not None:
            w = self.w.to(F64)[self.slots.long().clamp(0, len(self.w) - 1)]
        w.requires_grad_(True)
        h = w[:, None] * h_of(x)
        (h * self.dH.to(F64)).sum().backward()
        return x.detach(), w.detach(), x.grad, h.detach(), w.grad


@pytest.mark.parametrize("rows,inner", [(1, 32), (2, 2048), (7, 288), (64, 1408), (5000, 64), (20, 7168)])
@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("gone,pad", [(0.0, 0), (0.4, 8)])
def test_gradient_from_the_checkpoint(rows, inner, weighted, gone, pad):
    c = Grad(rows, inner, weighted=weighted, gone=gone, pad=pad)
    dX, H, dw = c.run()
    x, w, gx, h, gw = c.reference()
    t = c.there
    g, u = x.chunk(2, dim=1)
    s = 1 / (1 + torch.exp(-g))
    d = (w[:, None] * c.dH.to(F64)).abs()
    # dg's factor 1 + g (1 - sigma) can cancel: its two terms' sizes
    size = torch.cat([d * u.abs() * s * (1 + (g * (1 - s)).abs()), d * (g * s).abs()], dim=1)
    assert ((dX.to(F64) - gx).abs()[t] <= (2.0 ** -8 * gx.abs() + 2.0 ** -18 * size)[t]).all()
    assert ((H.to(F64) - h).abs()[t] <= ((2.0 ** -8 + 2.0 ** -18) * h.abs())[t]).all()
    if weighted:
        at = c.slots[t].long()
        room = 2.0 ** -17 * (c.dH.to(F64) * h_of(x)).abs().sum(dim=1)
        assert ((dw[at].to(F64) - gw[t]).abs() <= room[t]).all()
        rest = torch.ones_like(dw, dtype=torch.bool)
        rest[at] = False
        assert (dw[rest] == GUARD).all()
    again = c.run(with_h=False)
    assert torch.equal(again[0], dX) and (dw is None or torch.equal(again[2], dw))


def test_gradient_against_differences():
    # of sum dh w silu(g) u along random directions, in 64 bits around the saved values: differences of step 1e-4 are off
    # by its square times third derivatives (below 2 |u| + 6 a column), the kernel by half a BF16 step of each term
    c = Grad(16, 64, seed=9)
    dX, _, dw = c.run()
    x, w, gx, h, gw = c.reference()
    v, y = normal(16, 128, seed=11).to(F64), normal(16, seed=12).to(F64)
    f = lambda e: ((w + e * y)[:, None] * h_of(x + e * v) * c.dH.to(F64)).sum(dim=1)
    diff = (f(1e-4) - f(-1e-4)) / 2e-4
    along = (dX.to(F64) * v).sum(dim=1) + dw[c.slots.long().clamp(max=len(dw) - 1)].to(F64) * y
    room = (gx.abs() * v.abs()).sum(dim=1) * 2.0 ** -8 + 1e-8 * 64 * 1000
    assert ((along - diff).abs() <= room)[c.there].all()


def test_no_rows_and_no_slots():
    c = Grad(50, 64)
    c.slots = torch.arange(50, dtype=I32, device="cuda")
    c.there = torch.ones(50, dtype=torch.bool, device="cuda")
    dX, H, dw = c.run()
    a, b, e = torch.empty_like(dX), torch.empty_like(H), torch.empty_like(dw)
    tkg.swiglu_grad(c.Q, c.sf, c.dH, a, b, weights=c.w, dweights=e)
    assert torch.equal(a, dX) and torch.equal(b, H) and torch.equal(e[:50], dw[:50])
    for rows, inner in ((0, 64), (5, 0)):
        X, Hn = torch.empty(rows, 2 * inner, device="cuda", dtype=BF16), torch.empty(rows, inner, device="cuda", dtype=BF16)
        Q, sf = torch.empty(X.shape, device="cuda", dtype=U8), torch.empty(rows, inner // 16, device="cuda", dtype=U8)
        tkg.checkpoint_mxfp8(X, Q, sf)
        tkg.swiglu(X, Hn, Q, sf)
        wts = torch.ones(rows, device="cuda")
        tkg.swiglu_grad(Q, sf, Hn, X, Hn, weights=wts, dweights=wts)
        assert (wts == (0 if rows else 1)).all()                     # without columns dw is 0


# ---------------------------------------------------------------- weight gradients

class Product:
    def __init__(self, sizes, tokens, topk, n, k, spare=0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + n + k + tokens)
        self.sizes, self.topk = sizes, topk
        self.rows = sum(sizes)
        self.dev = torch.tensor(sizes, dtype=I32, device="cuda")
        self.dD = normal(self.rows + spare, n, seed=seed)
        self.dD[self.rows:] = float("nan")
        self.Q, self.sf = save(normal(tokens, k, seed=seed + 1))
        self.slots = torch.randint(0, tokens * topk, (self.rows + spare,), generator=g, device="cuda").to(I32)
        self.slots[self.rows:] = -1

    def A(self):
        v = values(self.Q, self.sf)
        t = torch.div(self.slots.long(), self.topk, rounding_mode="floor")
        inside = (t >= 0) & (t < v.shape[0])
        return torch.where(inside[:, None], v[t.clamp(0, v.shape[0] - 1)], 0.0)

    def check(self, dtype=BF16, alpha=0.5):
        n, k = self.dD.shape[1], self.Q.shape[1]
        dB = torch.full((len(self.sizes), n, k), GUARD, device="cuda", dtype=dtype)
        tkg.gemm_grouped_dev_mxfp8_wgrad(self.dev, self.dD, self.Q, self.sf, dB, slots=self.slots, topk=self.topk, alpha=alpha)
        A, o = self.A(), 0
        for i, m in enumerate(self.sizes):
            d, a = self.dD[o:o + m].to(F64), A[o:o + m]
            ref, mag = alpha * (d.T @ a), abs(alpha) * (d.abs().T @ a.abs())
            room = 1e-5 * mag + (2.0 ** -7 if dtype == BF16 else 2.0 ** -23) * ref.abs()
            assert ((dB[i].to(F64) - ref).abs() <= room).all(), i
            o += m
        return dB


SIZES = [[5], [1, 0, 300, 129, 7], [64, 64], [0, 0, 3], [15, 17, 33, 63, 64, 65], [255, 257, 0, 31, 700]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("n,k", [(264, 544), (64, 32), (8, 64), (1000, 256), (136, 2080)])
def test_weight_gradients(sizes, n, k):
    p = Product(sizes, tokens=40, topk=3, n=n, k=k, spare=70)
    p.check()
    p.check(F32)


def test_weight_gradients_equal_those_of_the_values():
    # the values are exact in BF16: the same bits as the BF16 product of the decoded rows, stored and added
    p = Product([100, 0, 33, 260], tokens=90, topk=4, n=264, k=320, spare=5)
    for accumulate, dtype in ((False, BF16), (False, F32), (True, F32)):
        a, b = (torch.ones(4, 264, 320, device="cuda", dtype=dtype) for _ in range(2))
        tkg.gemm_grouped_dev_mxfp8_wgrad(p.dev, p.dD, p.Q, p.sf, a, slots=p.slots, topk=4, accumulate=accumulate)
        tkg.gemm_grouped_dev_bf16_wgrad(p.dev, p.dD, p.A().to(BF16), b, accumulate=accumulate)
        assert torch.equal(a, b)


def test_rows_without_a_token_and_rows_in_place():
    p = Product([30, 12], tokens=20, topk=2, n=64, k=96, spare=4)
    p.slots[3], p.slots[7], p.slots[35] = -5, 40, 2 ** 31 - 1       # outside: they add nothing
    p.check()
    q = Product([30, 12], tokens=42, topk=1, n=64, k=96)
    q.slots = torch.arange(42, dtype=I32, device="cuda")
    want = q.check()
    got = torch.empty_like(want)
    tkg.gemm_grouped_dev_mxfp8_wgrad(q.dev, q.dD, q.Q, q.sf, got, alpha=0.5)
    assert torch.equal(got, want)


def test_weight_gradients_of_nothing():
    e = lambda *s, dtype=BF16: torch.empty(*s, dtype=dtype, device="cuda")
    sizes = torch.zeros(2, dtype=I32, device="cuda")
    dB = torch.ones(2, 64, 32, device="cuda")
    tkg.gemm_grouped_dev_mxfp8_wgrad(sizes, e(0, 64), e(0, 32, dtype=U8), e(0, 1, dtype=U8), dB, accumulate=True)
    assert (dB == 1).all()
    tkg.gemm_grouped_dev_mxfp8_wgrad(sizes, e(9, 64), e(0, 32, dtype=U8), e(0, 1, dtype=U8), dB)
    assert (dB == 0).all()
