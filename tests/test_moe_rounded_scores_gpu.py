"""Routing where a far bias rounds the scores in 64 bits: those that fall on the same number tie (the lowest index wins), and
which do is decided by the rounding of the exact score, not of one whose sum is approximate.

With scores around 1 / experts and a bias of -1e9, c lies on multiples of 2^-23; the scores are spread over one or two of
those.  The reference's own sum in 64 bits may be off by 2^-50, which moves one in 10^8 of them over a boundary."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg
from test_moe_route_gpu import check, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _healthy():
    yield
    assert tkg.device_status() == tkg.OK


@pytest.mark.parametrize("bias,spread", [(-1e9, 2e-6), (-1e9, 1e-5), (-1e6, 1e-6), (1e9, 4e-6), (-1e8, 3e-6)])
@pytest.mark.parametrize("experts,groups,stay", [(32, 1, 1), (16, 1, 1), (8, 1, 1), (32, 4, 2), (16, 8, 3)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_scores_on_the_grid_of_a_far_bias(scores, experts, groups, stay, bias, spread):
    z = normal(4000, experts, seed=5, scale=spread)
    b = torch.full((experts,), bias, device="cuda")
    for topk in (1, 4, min(8, experts // groups * stay)):
        check(z, topk, bias=b, scores=scores, groups=groups, topk_groups=stay)
