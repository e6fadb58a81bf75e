"""Logits of both zeros are equal: picks and groups go to the lower of them."""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fme():
    import fp4_moe_expert_gb300 as m
    return m


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [6, 40, 64, 256, 384, 896, 1024])
def test_zeros_of_both_signs_are_equal(fme, score, dtype, E):
    k = 5
    logits = torch.zeros(4, E, device=DEV)
    logits[0, ::2] = -0.0
    logits[1, 1::2] = -0.0
    logits[2] = -0.0
    logits[2, E - 1] = 0.0
    logits[3] = torch.where(torch.arange(E, device=DEV) % 3 == 0, -0.0, -1.0)
    logits[3, E - 2] = 0.0
    logits = logits.to(dtype)
    assert torch.signbit(logits[0, 0])
    expect = [list(range(k))] * 3 + [sorted(range(E), key=lambda e: (-logits[3, e].item(), e))[:k]]
    for bias in (None, torch.zeros(E, device=DEV), torch.full((E,), -0.0, device=DEV)):
        assert fme.moe_route_groups(logits, bias, k, score)[0].tolist() == expect
        if bias is not None:
            assert fme.moe_route(logits, bias, k)[0].tolist() == expect


@pytest.mark.parametrize("E,groups", [(40, 5), (64, 8), (64, 32), (256, 8), (384, 3), (896, 7), (1024, 32)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_of_zeros_of_both_signs_are_equal(fme, E, groups, group_top):
    size = E // groups
    logits = torch.full((2, E), -0.0, device=DEV)
    logits[1, size:2 * size] = 0.0  # the second group's zeros are no better
    for score in ("sigmoid", "softmax"):
        for bias in (None, torch.full((E,), -0.0, device=DEV)):
            ids = fme.moe_route_groups(logits, bias, 2, score, groups=groups, top_groups=2, group_top=group_top)[0]
            assert ids.tolist() == [[0, 1], [0, 1]]
            ids = fme.moe_route_groups(logits, bias, 2, score, groups=groups, top_groups=1, group_top=group_top)[0]
            assert ids.tolist() == [[0, 1], [0, 1]]
