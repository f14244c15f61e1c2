"""A routing rule is kept for the next call by its values: arguments that their owner changes later are read anew."""
import pytest
import torch

from dense_block_scaled_gb300 import tkg


def values(*args):
    r = tkg._rule(*args)._obj
    return r.scores, r.groups, r.topk_groups, r.renormalise, r.scale


def test_arguments_that_change():
    groups, stay, renormalise, scale = torch.tensor(8), torch.tensor(4), torch.tensor(True), torch.tensor(2.0)
    assert values("sigmoid", groups, stay, renormalise, scale) == (1, 8, 4, 1, 2.0)
    groups.fill_(6), stay.fill_(2), renormalise.fill_(False), scale.fill_(0.5)
    assert values("sigmoid", groups, stay, renormalise, scale) == (1, 6, 2, 0, 0.5)


def test_equal_values_share_a_rule():
    one = tkg._rule("softmax", 4, 2, True, 1.5)
    assert tkg._rule("softmax", torch.tensor(4), torch.tensor(2), 1, torch.tensor(1.5)) is one
    assert values("softmax", True, True, 0, 1) == (0, 1, 1, 0, 1.0)


@pytest.mark.parametrize("groups,stay", [(1.0, 1), (8, 2.5), ("8", 1), (None, 1), (torch.tensor([2, 2]), 1)])
def test_what_is_no_whole_number_is_refused(groups, stay):
    tkg._rule("softmax", 1, 1, True, 1.0)      # (1.0 equals a kept 1)
    with pytest.raises(TypeError):
        tkg._rule("softmax", groups, stay, True, 1.0)


@pytest.mark.parametrize("groups,stay", [(2 ** 32 + 1, 1), (8, 2 ** 31), (-2 ** 31 - 1, 1)])
def test_numbers_past_32_bits_are_refused(groups, stay):
    with pytest.raises(ValueError, match="below 2\\^31"):
        tkg._rule("softmax", groups, stay, True, 1.0)


@pytest.mark.parametrize("topk", [2 ** 31, 2 ** 32 + 2])
def test_choices_per_token_past_32_bits_are_refused(topk):
    m = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype)
    u8 = torch.uint8
    with pytest.raises(ValueError, match="topk: below 2\\^31"):
        tkg.gemm_grouped_dev_mxfp8_wgrad(m(4, dtype=torch.int32), m(10, 64), m(5, 32, dtype=u8), m(5, 1, dtype=u8),
                                         m(4, 64, 32), topk=topk)
