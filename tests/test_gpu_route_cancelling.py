"""Groups whose two best biased scores cancel: their sum is far smaller than
either, and so is the difference between groups."""
import pytest
import torch

from test_gpu_route import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2, 4, 20])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("level", [1.0, 30.0, 1000.0])
def test_groups_whose_biases_cancel(mx, size, score, level):
    print("cancel", size, score, level, flush=True)
    groups, T = 8, 4000
    g = torch.Generator("cuda").manual_seed(size)
    x = torch.randn((T, groups * size), generator=g, device="cuda") * 0.02
    bias = torch.full((groups, size), -3 * level, device="cuda")
    bias[:, 0], bias[:, -1] = level, -level
    _check(mx, x, 3, score=score, bias=bias.view(-1), groups=groups, groups_kept=3, group_top=2)


def test_groups_with_infinite_biases(mx):
    inf = float("inf")
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn((300, 32), generator=g, device="cuda")
    for low in (1, 2, 3):                                     # groups left with 3, 2 and 1 experts
        bias = torch.zeros((8, 4), device="cuda")
        bias[2, :low] = -inf
        bias[5] = -inf
        for score in ("sigmoid", "softmax"):
            _check(mx, x, 4, score=score, bias=bias.view(-1), groups=8, groups_kept=4, group_top=1)
            if low < 3:
                _check(mx, x, 4, score=score, bias=bias.view(-1), groups=8, groups_kept=4, group_top=2)
