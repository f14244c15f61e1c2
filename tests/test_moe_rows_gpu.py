"""Rows into expert order and back (tkg_moe_dispatch, tkg_moe_combine): copies are exact; sums of k products in FP32 are
off by at most k roundings of 2^-24 of the products' sizes, and rounded once to BF16 (half a step: 2^-8)."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg

pytestmark = pytest.mark.gpu
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
GUARD = 7.0


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


class Case:
    def __init__(self, tokens, topk, hidden, spare=0, dropped=0.0, pad=0, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + tokens * 31 + topk * 7 + hidden)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.cap = tokens * topk + spare
        rows = torch.randperm(self.cap, generator=g, device="cuda")[:tokens * topk].reshape(tokens, topk)
        gone = torch.rand(tokens, topk, generator=g, device="cuda") < dropped
        self.rows = torch.where(gone, torch.tensor([-1, -7, self.cap, 2 ** 31 - 1], device="cuda")[rows % 4], rows).to(I32)
        self.there = ~gone
        self.X = r(tokens, hidden + pad).to(BF16)[:, :hidden]
        self.O = r(self.cap, hidden + pad).to(BF16)[:, :hidden]
        self.w = torch.rand(tokens, topk, generator=g, device="cuda")
        used = torch.zeros(self.cap, dtype=torch.bool, device="cuda")
        used[self.rows[self.there].long()] = True
        self.used = used

    def dispatch(self, pad=0):
        t, h = self.X.shape
        buf = torch.full((self.cap + 1, h + pad), GUARD, device="cuda", dtype=BF16)
        out = buf[:self.cap, :h]
        tkg.moe_dispatch(self.X, self.rows, out)
        assert (buf[self.cap:] == GUARD).all() and (buf[:, h:] == GUARD).all()
        return out

    def combine(self, weights=None, pad=0):
        t, h = self.X.shape
        buf = torch.full((t + 1, h + pad), GUARD, device="cuda", dtype=BF16)
        tkg.moe_combine(self.O, self.rows, buf[:t, :h], weights=weights)
        assert (buf[t:] == GUARD).all() and (buf[:, h:] == GUARD).all()
        return buf[:t, :h]


SHAPES = [(1, 1, 8), (1, 8, 4096), (4, 32, 72), (33, 6, 1024), (100, 9, 2056), (257, 2, 1032), (1000, 8, 256), (3, 17, 7168)]


@pytest.mark.parametrize("tokens,topk,hidden", SHAPES)
@pytest.mark.parametrize("dropped,pad", [(0.0, 0), (0.4, 8), (1.0, 24)])
def test_both_ways(tokens, topk, hidden, dropped, pad):
    c = Case(tokens, topk, hidden, spare=5, dropped=dropped, pad=pad)
    out = c.dispatch(pad)
    want = torch.full_like(out, GUARD)
    for j in range(topk):
        k = c.there[:, j]
        want[c.rows[k, j].long()] = c.X[k]
    assert torch.equal(out, want)
    c.O[~c.used] = float("nan")                     # rows that no place names
    for weights in (None, c.w):
        got = c.combine(weights, pad).to(F64)
        ref, size = torch.zeros_like(got), torch.zeros_like(got)
        for j in range(topk):
            k = c.there[:, j]
            o = c.O[c.rows[k, j].long()].to(F64) * (1.0 if weights is None else weights[k, j:j + 1].to(F64))
            ref[k] += o
            size[k] += o.abs()
        assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + topk * 2.0 ** -24 * size).all()


def test_each_is_the_others_gradient():
    # the inner products agree up to combine's rounding (of each Y, half a BF16 step)
    c = Case(120, 6, 264, dropped=0.2)
    out = c.dispatch().to(F64)
    Y = c.combine().to(F64)
    a = (out * c.O.to(F64))[c.used].sum()
    b = (c.X.to(F64) * Y).sum()
    room = (c.X.to(F64).abs() * Y.abs() * 2.0 ** -8).sum() + 1e-6 * c.O.to(F64).abs().sum()
    assert (a - b).abs() <= room


def test_weights_and_rows_that_are_not_numbers():
    c = Case(50, 4, 64)
    c.w[3, 1] = float("nan")
    c.O[c.rows[9, 2].long(), 5] = float("inf")
    Y = c.combine(c.w)
    assert Y[3].isnan().all() and not Y[4].isnan().any()
    assert Y[9, 5] == float("inf")


@pytest.mark.parametrize("tokens,hidden,cap", [(0, 64, 10), (10, 0, 10), (10, 64, 0)])
def test_nothing_to_do(tokens, hidden, cap):
    rows = torch.full((tokens, 3), 0, device="cuda", dtype=I32)
    X, out = torch.ones(tokens, hidden, device="cuda", dtype=BF16), torch.full((cap, hidden), GUARD, device="cuda", dtype=BF16)
    tkg.moe_dispatch(X, rows, out)
    assert tokens and cap or (out == GUARD).all()
    Y = torch.full((tokens, hidden), GUARD, device="cuda", dtype=BF16)
    tkg.moe_combine(out, rows, Y)
    if cap == 0:
        assert (Y == 0).all()                       # no place is inside: empty sums


def test_offsets_past_32_bits():
    # 2.4 billion elements of O: a row far behind the 2^31st element
    hidden, cap = 8192, 290_000
    O = torch.empty(cap, hidden, device="cuda", dtype=BF16)
    rows = torch.tensor([[cap - 1], [0], [cap - 2]], dtype=I32, device="cuda")
    X = torch.randn(3, hidden, device="cuda").to(BF16)
    tkg.moe_dispatch(X, rows, O)
    assert torch.equal(O[rows[:, 0].long()], X)
    Y = torch.empty_like(X)
    tkg.moe_combine(O, rows, Y)
    assert torch.equal(Y, X)
