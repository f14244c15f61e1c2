"""Seeded random cases of the mixture-of-experts operators: sizes, rules, types, pitches, padding, capacities and streams
mixed, each against its definition.  Tolerances as in the operators' own tests."""
import random

import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_checkpoints_gpu import Grad, Product, h_of, rule, save
from test_moe_rows_gpu import Case
from test_moe_route_gpu import check, normal, scores_of, weights_of

pytestmark = pytest.mark.gpu
BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


def on_some_stream(rng, f):
    if rng.random() < 0.5:
        return f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = f()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("seed", range(40))
def test_route(seed):
    rng = random.Random(seed)
    groups = rng.choice([1, 1, 2, 3, 8, 16, 32])
    per = rng.randint(1, 512 // groups if rng.random() < 0.3 else max(1, 128 // groups))
    experts, stay = groups * per, rng.randint(1, groups)
    topk = rng.randint(1, min(32, stay * per, rng.choice([8, 8, 32])))
    tokens = rng.choice([1, 3, 17, 64, 65, 200, 1111, 5000])
    dtype, pad = rng.choice([BF16, F32]), rng.choice([0, 0, 1, 8])
    z = normal(tokens, experts + pad, seed=seed, scale=rng.choice([0.1, 1.5, 6.0]))[:, :experts].to(dtype)
    if pad:
        z = torch.nn.functional.pad(z, (pad, 0))[:, pad:]
    if rng.random() < 0.3:
        z = (z.float() * 2).round().to(dtype) / 2          # many ties
    keep = normal(tokens, seed=seed) > -0.5 if rng.random() < 0.4 else None
    bias = normal(experts, seed=seed, scale=0.05) if rng.random() < 0.5 else None
    kw = dict(scores=rng.choice(["softmax", "sigmoid"]), renormalise=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]))
    ids, _ = on_some_stream(rng, lambda: check(z, topk, keep=keep, bias=bias, groups=groups, topk_groups=stay, **kw))
    # and the gradient of what was chosen
    dw = normal(tokens, topk, seed=seed, scale=1.0)
    got = torch.empty_like(z)
    tkg.moe_route_grad(z, ids, dw, got, **kw)
    x = z.to(F64).requires_grad_(True)
    w = weights_of(x, ids.long(), **kw)
    (w * dw.to(F64)).sum().backward()
    size = scores_of(z.to(F64), kw["scores"]) * kw["scale"] * 2 * dw.abs().amax(dim=1, keepdim=True)
    if kw["renormalise"]:
        v = w.detach()
        size = torch.zeros_like(size).scatter_(1, ids.long().clamp(min=0), v * (dw.abs() + (v * dw.abs()).sum(dim=1, keepdim=True)))
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -23
    assert ((got.to(F64) - x.grad).abs() <= 2.0 ** -16 * size + half * x.grad.abs() + 1e-38).all()


@pytest.mark.parametrize("seed", range(12))
def test_rows(seed):
    rng = random.Random(100 + seed)
    c = Case(rng.randint(1, 400), rng.randint(1, 12), 8 * rng.randint(1, 400), spare=rng.randint(0, 9),
             dropped=rng.choice([0.0, 0.3]), pad=rng.choice([0, 8, 40]), seed=seed)
    out = on_some_stream(rng, lambda: c.dispatch(rng.choice([0, 8])))
    for j in range(c.rows.shape[1]):
        k = c.there[:, j]
        assert torch.equal(out[c.rows[k, j].long()], c.X[k])
    Y = on_some_stream(rng, lambda: c.combine(c.w)).to(F64)
    ref, size = torch.zeros_like(Y), torch.zeros_like(Y)
    for j in range(c.rows.shape[1]):
        k = c.there[:, j]
        o = c.O[c.rows[k, j].long()].to(F64) * c.w[k, j:j + 1].to(F64)
        ref[k] += o
        size[k] += o.abs()
    assert ((Y - ref).abs() <= 2.0 ** -8 * ref.abs() + 12 * 2.0 ** -24 * size).all()


@pytest.mark.parametrize("seed", range(12))
def test_activation(seed):
    rng = random.Random(200 + seed)
    rows, inner = rng.randint(1, 300), 32 * rng.randint(1, 80)
    X = normal(rows, 2 * inner, seed=seed, scale=rng.choice([0.01, 1.0, 20.0])).to(BF16)
    H = torch.empty(rows, inner, device="cuda", dtype=BF16)
    Q, sf = torch.empty(rows, 2 * inner, device="cuda", dtype=torch.uint8), torch.empty(rows, inner // 16, device="cuda", dtype=torch.uint8)
    on_some_stream(rng, lambda: tkg.swiglu(X, H, Q, sf))
    ref = h_of(X.to(F64))
    # sigma's exponent -x log2(e) is off by 2 x 2^-24 |x|: 2^-16.4 of sigma at |x| = 100; a sigma below 2^-126 is 0, and
    # h = g sigma u then off by at most 2^-126 |g u|
    lost = 2.0 ** -126 * (X[:, :inner].to(F64) * X[:, inner:].to(F64)).abs()
    assert ((H.to(F64) - ref).abs() <= (2.0 ** -8 + 2.0 ** -16) * ref.abs() + lost).all()
    q, s = rule(X)
    assert torch.equal(Q, q) and torch.equal(sf, s) and all(torch.equal(a, b) for a, b in zip(save(X), (q, s)))
    c = Grad(rows, inner, weighted=rng.random() < 0.6, gone=rng.choice([0.0, 0.5]), pad=rng.choice([0, 8]), seed=seed)
    dX, Hw, dw = on_some_stream(rng, c.run)
    x, w, gx, h, gw = c.reference()
    t = c.there
    assert ((Hw.to(F64) - h).abs()[t] <= ((2.0 ** -8 + 2.0 ** -18) * h.abs())[t]).all()
    assert float((dX.to(F64) - gx)[t].norm()) <= 2.0 ** -8 * float(gx[t].norm()) + 1e-30


@pytest.mark.parametrize("seed", range(10))
def test_weight_gradient(seed):
    rng = random.Random(300 + seed)
    sizes = [rng.choice([0, 1, 2, rng.randint(1, 200), rng.randint(1, 200)]) for _ in range(rng.randint(1, 20))]
    if not sum(sizes):
        sizes[0] = 3
    p = Product(sizes, tokens=rng.randint(1, 300), topk=rng.randint(1, 6), n=8 * rng.randint(1, 60), k=32 * rng.randint(1, 30),
                spare=rng.choice([0, 1, 70]), seed=seed)
    on_some_stream(rng, lambda: p.check(rng.choice([BF16, F32]), alpha=rng.choice([1.0, -0.25])))
