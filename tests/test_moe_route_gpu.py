"""Routing (tkg_moe_route, tkg_moe_route_grad) against its definition in 64 bits: every choice, row and slot equal, the
weights and the logits' gradient within what FP32 loses.

Tolerances.  A weight is exp(z - top) over a sum, or sigma(z): the difference's rounding (2^-24 of at most 64 here) stands
in the exponent, 2^-18; exp, the quotient and the sum are a few 2^-24 each; renormalised twice that: 2^-16 of the weight,
and the least normal number where one underflows.  A gradient is a sum of two products of such weights with dw: the same
share of those products' sizes, and half a step of its type."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg

pytestmark = pytest.mark.gpu
F32, F64, BF16, I32 = torch.float32, torch.float64, torch.bfloat16, torch.int32
TINY = 2.0 ** -126


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


def scores_of(z, scores):
    if scores == "sigmoid":
        return 1 / (1 + torch.exp(-z))
    top = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - torch.where(top == -torch.inf, 0.0, top))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def order(c):
    """Descending, NaN last, ties to the lowest index."""
    return torch.sort(torch.where(c.isnan(), -torch.inf, c), dim=1, descending=True, stable=True).indices


def choice(logits, topk, scores="softmax", bias=None, groups=1, topk_groups=1, keep=None, **_):
    z = logits.to(F64)
    s = scores_of(z, scores)
    # (the logits themselves where they decide: scores in 64 bits can underflow, or round to 1)
    c = s + bias.to(F64) if bias is not None else (s if topk_groups < groups else z)
    if topk_groups < groups:
        by = c.unflatten(1, (groups, -1))
        best = by.sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
        stay = torch.zeros_like(best, dtype=torch.bool).scatter_(1, order(best)[:, :topk_groups], True)
        # of the groups that stay alone: one of their experts may have -inf itself
        ids = order(c)
        inside = stay.repeat_interleave(by.shape[2], dim=1).gather(1, ids)
        ids = ids.gather(1, torch.sort(inside.to(torch.int8), dim=1, descending=True, stable=True).indices)[:, :topk]
    else:
        ids = order(c)[:, :topk]
    return ids if keep is None else torch.where(keep[:, None].bool(), ids, -1)


def weights_of(z, ids, scores="softmax", renormalise=True, scale=1.0, **_):
    at = ids.clamp(min=0)
    if renormalise and scores == "softmax":
        w = scores_of(z.gather(1, at), scores)
    else:
        w = scores_of(z, scores).gather(1, at)
        if renormalise:
            total = w.sum(dim=1, keepdim=True)
            w = w / torch.where(total == 0, 1.0, total)
    return torch.where(ids >= 0, scale * w, torch.zeros_like(w))


def places(ids, experts):
    flat = ids.flatten()
    where = [(flat == e).nonzero()[:, 0] for e in range(experts)]
    inside = torch.cat(where)
    rows, slots = torch.full_like(flat, -1), torch.full_like(flat, -1)
    rows[inside] = torch.arange(len(inside), device=flat.device)
    slots[:len(inside)] = inside
    return torch.tensor([len(w) for w in where]), rows.reshape(ids.shape), slots


def route(logits, topk, keep=None, bias=None, **kw):
    t, e = logits.shape
    out = [torch.full(s, 7, device="cuda", dtype=d) for s, d in (((t, topk), I32), ((t, topk), F32), ((e,), I32),
                                                                   ((t, topk), I32), ((t * topk,), I32))]
    tkg.moe_route(logits, *out, keep=keep, bias=bias, **kw)
    return out


def check(logits, topk, keep=None, bias=None, **kw):
    ids, w, sizes, rows, slots = route(logits, topk, keep, bias, **kw)
    ref = choice(logits, topk, keep=keep, bias=bias, **kw)
    assert torch.equal(ids.long(), ref), f"{int((ids.long() != ref).any(dim=1).sum())} tokens chosen otherwise"
    want = weights_of(logits.to(F64), ref, **kw)
    bad = ~((w - want).abs() <= 2.0 ** -16 * want.abs() + TINY) & ~(w.isnan() & want.isnan())
    assert not bad.any(), int(bad.sum())
    for got, one in zip((sizes, rows, slots), places(ref, logits.shape[1])):
        assert torch.equal(got.cpu().long(), one.cpu().long())
    return ids, w


def normal(*shape, seed=0, dtype=F32, scale=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + sum(shape))
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 2, 16, 17, 31, 32, 33, 65, 128, 129, 256, 257, 511, 512, 513, 1000])
@pytest.mark.parametrize("experts,topk", [(1, 1), (2, 2), (7, 3), (32, 8), (33, 1), (60, 4), (64, 6), (100, 32), (128, 8),
                                          (200, 5), (256, 8), (511, 9), (512, 2)])
def test_sizes(tokens, experts, topk, dtype):
    check(normal(tokens, experts, dtype=dtype), topk)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("experts,topk,groups,stay", [(128, 8, 1, 1), (256, 8, 8, 4), (60, 4, 6, 2), (24, 3, 24, 3),
                                                      (96, 6, 32, 3), (512, 7, 2, 1), (40, 20, 4, 2), (64, 4, 4, 4)])
def test_rules(scores, renormalise, biased, experts, topk, groups, stay):
    bias = normal(experts, scale=0.1) if biased else None
    for dtype in (BF16, F32):
        check(normal(777, experts, dtype=dtype, seed=3), topk, bias=bias, scores=scores, groups=groups, topk_groups=stay,
              renormalise=renormalise, scale=2.5)


@pytest.mark.parametrize("tokens", [19456, 19457, 40001])
def test_many_tokens(tokens):
    keep = normal(tokens) > -1.0
    check(normal(tokens, 64, dtype=BF16), 6, keep=keep)


@pytest.mark.parametrize("tokens", [5, 300])
@pytest.mark.parametrize("share", [0.0, 0.5])
@pytest.mark.parametrize("kind", [torch.bool, torch.uint8])
def test_padding(tokens, share, kind):
    keep = (torch.rand(tokens, device="cuda") < share).to(kind)
    z = normal(tokens, 60)
    z[~keep.bool()] = float("nan")    # whatever stands in the padding
    check(z, 4, keep=keep)


def test_rows_that_are_pitched_or_start_anywhere():
    for dtype in (BF16, F32):
        big = normal(200, 400, dtype=dtype)
        for view in (big[:, :128], big[:, 8:136], big[:, 1:129], big[:, 3:63], big[5:, 399:], big[::2, 2:66], big[:1, 7:39]):
            check(view, min(4, view.shape[1]))


@pytest.mark.parametrize("groups,stay", [(1, 1), (8, 3)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_index(groups, stay, scores):
    kw = dict(scores=scores, groups=groups, topk_groups=stay)
    check(torch.zeros(100, 64, device="cuda"), 8, **kw)
    check(normal(500, 64).round(), 8, **kw)                                 # a handful of values
    check(normal(500, 64).round(), 8, bias=normal(64).round() / 4, **kw)
    z = torch.zeros(40, 64, device="cuda")
    z[::2] = -0.0
    z[:, 1::2] *= -1                                                        # -0 is 0
    check(z, 5, **kw)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,stay", [(1, 1), (4, 2)])
def test_choices_that_fp32_does_not_decide(scores, groups, stay):
    # biases that all but cancel the scores: what is left is far below FP32's rounding of a score
    z = normal(1, 128, seed=5)
    s = scores_of(z.to(F64), scores)
    bias = (0.25 - s[0]).to(F32)
    rows = z.expand(70, -1).contiguous()
    ids, _ = check(rows, 8, bias=bias, scores=scores, groups=groups, topk_groups=stay)
    wrong = (scores_of(z, scores) + bias)       # what FP32 alone would order by
    assert not torch.equal(order(wrong)[0, :8], ids[0].long()) or groups > 1


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,groups,stay,topk", [(256, 8, 4, 8), (128, 8, 3, 4), (64, 32, 5, 4), (60, 6, 2, 4), (24, 24, 3, 3)])
def test_groups_that_fp32_does_not_decide(scores, experts, groups, stay, topk):
    # biases that make the groups' sums of two all but equal, a few members' or all; rows alike but for tiny differences
    per = experts // groups
    z = normal(1, experts, seed=6, scale=0.5)
    s = scores_of(z.to(F64), scores)[0].unflatten(0, (groups, per))
    two = s.sort(dim=1, descending=True).values[:, :2].sum(dim=1)
    bias = ((2.0 - two) / min(2, per))[:, None].expand(-1, per).flatten().to(F32)
    rows = z.repeat(200, 1)
    rows[100:] += normal(100, experts, seed=7, scale=1e-6)
    check(rows, topk, bias=bias, scores=scores, groups=groups, topk_groups=stay)
    spread = bias + normal(experts, seed=8, scale=0.3) * (torch.arange(experts, device="cuda") // per % 2)
    check(rows, topk, bias=spread, scores=scores, groups=groups, topk_groups=stay)
    level = (1.0 - s.flatten()).to(F32)          # every expert all but equal
    check(rows, topk, bias=level, scores=scores, groups=groups, topk_groups=stay)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_many_rows_with_a_bias(scores, seed):
    # of 30000 rows a few hundred have two scores that FP32 does not tell apart
    check(normal(30000, 256, seed=seed), 8, bias=normal(256, scale=0.05, seed=seed), scores=scores)
    check(normal(30000, 256, seed=seed), 8, bias=normal(256, scale=0.05, seed=seed), scores=scores, groups=8, topk_groups=4)
    check(normal(30000, 128, seed=seed), 6, scores=scores, groups=8, topk_groups=4, renormalise=False)


def test_logits_closer_than_scores_tell():
    # distinct logits whose FP32 (and 64-bit) scores are equal: the logits decide
    z = torch.full((3, 64), -200.0, device="cuda")
    z[:, 0] = 0.0
    z[:, 10] = -199.0
    z[:, 63] = -198.5
    ids, w = check(z, 3)
    assert ids[0].tolist() == [0, 63, 10]
    z = torch.arange(64, device="cuda", dtype=F32).expand(3, -1) + 40
    assert check(z.contiguous(), 4, scores="sigmoid", renormalise=False)[0][0].tolist() == [63, 62, 61, 60]


def test_masked_experts_and_rows():
    z = normal(200, 64)
    z[:, 5:40] = -torch.inf
    z[7] = -torch.inf                                                       # nothing left: weights 0
    z[8, 1:] = -torch.inf
    for renormalise in (True, False):
        for scores in ("softmax", "sigmoid"):
            _, w = check(z, 8, renormalise=renormalise, scores=scores)
            assert (w[7] == 0).all()
    lowest = torch.where(z == -torch.inf, torch.finfo(F32).min, z)
    check(lowest, 8)
    check(lowest.to(BF16), 8)
    check(z, 4, bias=normal(64, scale=0.1))


def test_nan_comes_last():
    z = normal(100, 64)
    z[:, 3] = float("nan")
    z[4] = float("nan")
    ids, w, *_ = route(z, 8)
    assert not (ids[torch.arange(100) != 4] == 3).any() and ids[4].tolist() == list(range(8))
    assert w[4].isnan().all() and torch.equal(ids.long(), choice(z, 8))
    ids, w, *_ = route(z, 8, renormalise=False)
    assert w.isnan().all()


@pytest.mark.parametrize("groups,stay", [(1, 1), (8, 3), (4, 4)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_infinite_and_far_biases(scores, groups, stay):
    kw = dict(scores=scores, groups=groups, topk_groups=stay)
    z = normal(100, 64)
    out = torch.zeros(64, device="cuda")
    out[::3] = -torch.inf                       # experts out of service, more than are left to choose in some groups
    check(z, 6, bias=out, **kw)
    check(z, 20, bias=out, **kw)
    out[5] = torch.inf
    check(z, 6, bias=out, **kw)
    check(z, 6, bias=torch.where(out == -torch.inf, -1e30, normal(64, scale=1e3)), **kw)
    out[7] = float("nan")
    ids, *_ = route(z, 6, bias=out, **kw)
    if groups == 1:
        assert torch.equal(ids.long(), choice(z, 6, bias=out, **kw))
    z[3, 9] = torch.inf
    z[4] = torch.inf
    z[5, :60] = float("nan")
    out = torch.zeros(64, device="cuda")
    ids, w, sizes, rows, slots = route(z, 6, bias=out, **kw)
    assert ((ids >= 0) & (ids < 64)).all() and int(sizes.sum()) == 600 and (ids.sort(dim=1).values.diff(dim=1) > 0).all()
    if scores == "sigmoid" and groups == 1:
        assert torch.equal(ids.long(), choice(z, 6, bias=out, **kw))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("tokens,experts,topk", [(1, 128, 8), (77, 60, 4), (300, 33, 32), (1000, 256, 8), (9, 512, 1), (5, 1, 1)])
def test_gradient(tokens, experts, topk, scores, renormalise, dtype):
    z = normal(tokens, experts + 8, dtype=dtype, seed=2)[:, :experts]
    keep = torch.arange(tokens, device="cuda") % 5 != 3
    ids = choice(z, topk, keep=keep)
    dw = normal(tokens, topk, scale=1.0)
    kw = dict(scores=scores, renormalise=renormalise, scale=2.5)
    got = torch.full((tokens, experts + 8), 7.0, device="cuda", dtype=dtype)
    tkg.moe_route_grad(z, ids.to(I32), dw, got[:, :experts], **kw)
    assert (got[:, experts:] == 7.0).all()
    got = got[:, :experts]
    x = z.to(F64).requires_grad_(True)
    w = weights_of(x, ids, **kw)
    (w * dw.to(F64)).sum().backward()
    s = scores_of(z.to(F64), scores)
    if renormalise:
        size = torch.zeros_like(s).scatter_(1, ids.clamp(min=0), w.detach() * (dw.abs() + (w.detach() * dw.abs()).sum(dim=1, keepdim=True)))
    else:
        size = s * 2.5 * (dw.abs().amax(dim=1, keepdim=True) * 2)
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -23
    assert ((got.to(F64) - x.grad).abs() <= 2.0 ** -16 * size + half * x.grad.abs() + 1e-38).all()
    assert (got[~keep] == 0).all()
    # and against differences of the weights
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    v = torch.randn(tokens, experts, generator=g, device="cuda", dtype=F64)
    h = 1e-4
    up, down = (weights_of(z.to(F64) + d * v, ids, **kw) for d in (h, -h))
    diff = ((up - down) / (2 * h) * dw.to(F64)).sum(dim=1)
    along = (got.to(F64) * v).sum(dim=1)
    # third derivatives of the scores are below 1, times v^3 (below 5^3 a term) and dw: h^2 of their sum
    room = h * h * 125 * 2.5 * dw.abs().sum(dim=1) * (size > 0).sum(dim=1) + ((2.0 ** -16 * size + half * x.grad.abs()) * v.abs()).sum(dim=1)
    assert ((along - diff).abs() <= room + 1e-9).all()


def test_gradient_where_nothing_was_chosen_or_all_is_masked():
    z = torch.full((4, 64), -torch.inf, device="cuda")
    z[1] = normal(64)
    ids = torch.tensor([[0, 1], [-1, 900], [2, -5], [63, 0]], dtype=I32, device="cuda")
    for scores in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            out = torch.full_like(z, 7.0)
            tkg.moe_route_grad(z, ids, torch.ones(4, 2, device="cuda"), out, scores=scores, renormalise=renormalise)
            assert (out == 0).all()


def test_a_scale_that_is_not_a_float():
    z = normal(5, 64)
    scale = torch.tensor(2.0)
    _, a, *_ = route(z, 4, scale=scale)
    scale.mul_(2)
    _, b, *_ = route(z, 4, scale=scale)
    _, c, *_ = route(z, 4, scale=4)
    assert torch.equal(b, 2 * a) and torch.equal(b, c)


def test_no_tokens_and_a_captured_call():
    z = normal(0, 64)
    _, _, sizes, _, _ = route(z, 4)
    assert (sizes == 0).all()
    for tokens in (20, 3000):
        z = normal(tokens, 128, seed=8)
        out = route(z, 8)
        want = [x.clone() for x in out]
        ws = torch.empty(tkg.moe_route_workspace_bytes(tokens, 128), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tkg.moe_route(z, *out, workspace=ws)
        for x in out:
            x.fill_(9)
        graph.replay()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
