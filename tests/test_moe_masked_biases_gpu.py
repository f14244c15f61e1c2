"""Routing with a bias that masks experts by the lowest FP32 value, by far values and by -infinity, the topk reaching one or
more past the experts that are left: ids stay inside, and what stands behind the last expert (in the pitch of the
logits, behind the bias) is not chosen, although it would rank first.

Reference and tolerances are those of test_moe_route_gpu."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_moe_route_gpu import check, normal, route

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
LOWEST = torch.finfo(F32).min


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


def masked(experts, left, value, seed=0):
    """A bias with `left` experts near 0 and the rest at `value`, in front of 40 that would win."""
    g = torch.Generator()
    g.manual_seed(seed * 71 + experts)
    b = torch.full((experts + 40,), 1e30)
    b[:experts] = value
    b[torch.randperm(experts, generator=g)[:left]] = torch.randn(left, generator=g) * 0.1
    return b.cuda()[:experts]


def logits(tokens, experts, dtype, seed=0):
    """Logits with 40 columns of large ones behind each row."""
    z = torch.full((tokens, experts + 40), 100.0, device="cuda", dtype=dtype)
    z[:, :experts] = normal(tokens, experts, dtype=dtype, seed=seed)
    return z[:, :experts]


@pytest.mark.parametrize("value", [LOWEST, -torch.inf, -1e30, -1e9, -1e4], ids=str)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_one_past_the_unmasked(tokens, scores, value):
    for experts in range(1, 34):
        for left in {0, experts // 8, experts // 4, experts // 2, experts - 1}:
            topk = min(left + 1, 32)
            z = logits(tokens, experts, F32 if experts % 2 else BF16, seed=left)
            check(z, topk, bias=masked(experts, left, value), scores=scores)


@pytest.mark.parametrize("value", [LOWEST, -torch.inf, -1e30, -1e4], ids=str)
@pytest.mark.parametrize("experts,groups,stay,topk", [(32, 8, 2, 8), (32, 8, 3, 12), (16, 4, 2, 8), (24, 6, 2, 7), (30, 5, 2, 12),
                                                      (32, 32, 6, 6), (64, 8, 2, 16), (512, 8, 2, 16)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_masked_experts_of_groups_that_stay(scores, experts, groups, stay, topk, value):
    # one expert of each group is masked, so that as many of the chosen are as there are groups that stay
    per = experts // groups
    for seed in range(3):
        b = masked(experts, experts, 0.0, seed)
        b[torch.arange(groups, device="cuda") * per + (seed + 1) % per] = value
        check(logits(100, experts, F32, seed), topk, bias=b, scores=scores, groups=groups, topk_groups=stay)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_all_but_a_few_masked_of_many(scores):
    for experts in (60, 128, 256, 512):
        for value in (LOWEST, -1e9, -torch.inf):
            for left, topk in ((3, 4), (7, 8), (8, 8), (experts // 2, 8), (20, 24)):
                check(logits(200, experts, F32, left), topk, bias=masked(experts, left, value), scores=scores)


@pytest.mark.parametrize("experts,groups,stay,topk", [(64, 8, 3, 6), (60, 6, 2, 4), (24, 24, 5, 4), (512, 8, 4, 8)])
def test_a_group_with_a_nan_comes_last(experts, groups, stay, topk):
    per = experts // groups
    z = normal(100, experts)
    b = normal(experts, scale=0.1)
    b[per // 2] = float("nan")                                             # the first group, for all tokens
    at = torch.arange(100, device="cuda") % (groups - stay - 1) + 1
    z[torch.arange(100, device="cuda"), at * per + per - 1] = float("nan")     # and one more for each token
    ids, *_ = route(z, topk, bias=b, scores="sigmoid", groups=groups, topk_groups=stay)
    group = ids.long() // per
    assert (group != 0).all() and (group != at[:, None]).all()
    # the rest as without those groups
    out = torch.zeros(100, groups, dtype=torch.bool, device="cuda")
    out[:, 0] = True
    out[torch.arange(100, device="cuda"), at] = True
    out = out.repeat_interleave(per, dim=1)
    c = torch.where(out, -100.0, torch.sigmoid(z.double()) + b.double()).unflatten(1, (groups, per))
    best = c.sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
    stays = torch.zeros_like(best, dtype=torch.bool).scatter_(1, best.topk(stay, dim=1).indices, True)
    want = torch.where(stays[:, :, None], c, -1000.0).flatten(1).sort(dim=1, descending=True, stable=True).indices[:, :topk]
    assert torch.equal(ids.long(), want)
