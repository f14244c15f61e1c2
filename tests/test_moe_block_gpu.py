"""A whole mixture-of-experts block (examples/moe_block.py) against its formulas in 64 bits: forward, every gradient, on
another stream, captured and replayed, and its training loop.

Tolerance: between an input and a result stand at most five BF16 roundings of half a step each (2^-8 of an element), so a
result is off by at most 5 x 2^-8 = 0.02 in norm where the terms add up as they come; the reference takes the saved rows
as they were saved."""
import importlib.util
import os

import pytest
import torch

from dense_block_scaled_gb300 import tkg

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def values(saved):
    Q, sf = saved
    return (Q.view(torch.float8_e4m3fn).to(F64).unflatten(1, (-1, 32)) * torch.exp2(sf.to(F64) - 127)[..., None]).flatten(1)


def make(example, tokens, hidden, inner, experts, topk, seed=0, **rule):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    Wr, W1, W2 = r(experts, hidden), r(experts, 2 * inner, hidden), r(experts, hidden, inner)
    W1, W2 = (W1.float() * hidden ** -0.5).to(BF16), (W2.float() * inner ** -0.5).to(BF16)
    Wr = (Wr.float() * hidden ** -0.5).to(BF16)
    return example.Block(Wr, W1, W2, topk, **rule), r(tokens, hidden), r(tokens, hidden)


def reference(block, X, dY, keep=None):
    """Y; and, from the rows as they were saved, dX through the experts, dz, dW1, dW2."""
    z, ids, weights, sizes, rows, slots, saved, saved_x = block.kept
    t, hidden = X.shape
    k, inner = block.topk, block.W1.shape[1] // 2
    scale = block.rule.get("scale", 1.0)
    zz = z.to(F64).requires_grad_(True)
    s = torch.softmax(zz, dim=1) if block.rule.get("scores", "softmax") == "softmax" else torch.sigmoid(zz)
    w = s.gather(1, ids.long().clamp(min=0))
    if block.rule.get("renormalise", True):
        w = w / w.sum(dim=1, keepdim=True)
    w = w * scale
    if keep is not None:
        w = w * keep[:, None]
    Y = torch.zeros(t, hidden, dtype=F64, device="cuda")
    dX, dw = torch.zeros_like(Y), torch.zeros_like(w)
    dW1, dW2 = torch.zeros_like(block.W1, dtype=F64), torch.zeros_like(block.W2, dtype=F64)
    gu_saved, x_saved = values(saved), values(saved_x)
    act = lambda gu: torch.nn.functional.silu(gu[:, :inner]) * gu[:, inner:]
    for e in range(block.W1.shape[0]):
        tok, j = (ids == e).nonzero(as_tuple=True)
        if not len(tok):
            continue
        W1, W2 = block.W1[e].to(F64), block.W2[e].to(F64)
        row = rows[tok, j].long()
        Y.index_add_(0, tok, w[tok, j].detach()[:, None] * (act(X[tok].to(F64) @ W1.T) @ W2.T))
        gu = gu_saved[row].requires_grad_(True)
        h = act(gu)
        d = dY[tok].to(F64)
        dh = d @ W2
        dw[tok, j] = (dh * h).sum(dim=1).detach()
        (dgu,) = torch.autograd.grad((w[tok, j].detach()[:, None] * h * dh).sum(), gu)
        dW2[e] = d.T @ (w[tok, j].detach()[:, None] * h).detach()
        dW1[e] = dgu.T @ x_saved[tok]
        dX.index_add_(0, tok, dgu @ W1)
    (w * dw).sum().backward()
    return Y, dX, zz.grad, dW1, dW2


def close(got, want, what):
    err = float((got.to(F64) - want).norm() / want.norm())
    assert err <= 5 * 2.0 ** -8, f"{what}: {err:.3g}"


CASES = [
    dict(tokens=300, hidden=256, inner=128, experts=8, topk=2),
    dict(tokens=129, hidden=512, inner=64, experts=40, topk=5, scores="sigmoid", scale=2.5),
    dict(tokens=1000, hidden=96, inner=160, experts=24, topk=6, scores="sigmoid", groups=4, topk_groups=2),
    dict(tokens=64, hidden=256, inner=96, experts=128, topk=8, renormalise=False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
@pytest.mark.parametrize("padded", [False, True])
def test_block(example, case, padded):
    block, X, dY = make(example, **case)
    keep = torch.rand(case["tokens"], device="cuda") < 0.7 if padded else None
    if padded:
        X[~keep] = float("nan")          # whatever stands in the padding
        dY[~keep] = float("nan")
    Y = block.forward(X, keep=keep)
    dW1, dW2 = torch.ones_like(block.W1, dtype=F32), torch.ones_like(block.W2, dtype=F32)
    dX, dz = block.backward(dY, dW1, dW2)
    if padded:
        X, dY = torch.where(keep[:, None], X, 0.0), torch.where(keep[:, None], dY, 0.0)
        for t in (Y, dX, dz):
            assert (t[~keep] == 0).all()
        z = block.kept[0]
        z[~keep] = 0
    want = reference(block, X, dY, keep)
    for got, ref, what in zip((Y, dX, dz, dW1 - 1, dW2 - 1), want, ("Y", "dX", "dz", "dW1", "dW2")):
        close(got, ref, what)


def test_block_on_another_stream_and_captured(example):
    block, X, dY = make(example, **CASES[0])
    run = lambda g1, g2: (block.forward(X), *block.backward(dY, g1, g2))
    grads = lambda: [torch.zeros_like(w, dtype=F32) for w in (block.W1, block.W2)]
    g = grads()
    want = [x.clone() for x in (*run(*g), *g)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = grads()
        got = [*run(*g), *g]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # two at once, on streams of their own
    block2, X2, dY2 = make(example, **CASES[2])
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):
        g2 = [torch.zeros_like(w, dtype=F32) for w in (block2.W1, block2.W2)]
    other.wait_stream(torch.cuda.current_stream())
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(other):
            block2.forward(X2)
            block2.backward(dY2, *g2)
        with torch.cuda.stream(side):
            g = grads()
            got = [*run(*g), *g]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # captured: the gradients start from zero in the graph
    g = grads()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x in g:
            x.zero_()
        got = [*run(*g), *g]
    for _ in range(2):
        for x in got:
            x.fill_(5)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and with other tokens in the same buffers
    X.copy_(X.flip(0))
    dY.copy_(dY.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0].flip(0))


def test_example_trains(example):
    lines = []
    losses = example.train(steps=4, tokens=256, log=lines.append)
    assert len(losses) == 4 and all(x == x and x < float("inf") for x in losses) and lines
