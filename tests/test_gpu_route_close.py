"""The router's choice where scores are closer than fp32 can tell apart: inside
the chosen experts, at their end, between groups, and in runs longer than the
list that the kernel sorts again."""
import numpy as np
import pytest
import torch

from test_gpu_route import _check

pytestmark = pytest.mark.gpu


def _nudge(value, steps):
    """value plus whole steps of fp32."""
    v = torch.full(steps.shape, value, dtype=torch.float32)
    return (v.view(torch.int32) + steps.int()).view(torch.float32)


def _rows(T, E, run, seed):
    """Well-spaced logits; in every row `run` neighbours of the order, from a
    random rank among the first 20 on, lie within 12 steps of fp32."""
    rng = np.random.default_rng(seed)
    x = np.empty((T, E), np.float32)
    for t in range(T):
        level = np.linspace(2.5, -4.01, E).astype(np.float32)      # none is 0, which has no such neighbours
        at = int(rng.integers(0, min(20, E - run)))
        level[at:at + run] = _nudge(float(level[at]), torch.from_numpy(rng.integers(-12, 1, run))).numpy()
        x[t] = level[rng.permutation(E)]
    return torch.from_numpy(x).cuda()


@pytest.mark.parametrize("E,k", [(64, 8), (256, 8), (256, 15), (500, 10), (300, 31), (512, 32), (40, 16), (8, 8)])
@pytest.mark.parametrize("run", [2, 3, 7])
def test_close_scores(mx, E, k, run):
    print("close", E, k, run, flush=True)
    x = _rows(70, E, run, E + k + run)
    far = torch.where(torch.arange(E, device="cuda") % 3 == 0, 10.0, 0.0).float()
    for kw in ({}, dict(score="sigmoid"), dict(bias=torch.zeros(E, device="cuda")),
               dict(score="sigmoid", bias=torch.zeros(E, device="cuda")), dict(score="sigmoid", bias=far),
               dict(bias=-far)):
        _check(mx, x, k, **kw)


@pytest.mark.parametrize("run", [20, 60])
def test_runs_longer_than_the_list(mx, run):
    print("long run", run, flush=True)
    x = _rows(40, 128, run, run)
    zero = torch.zeros(128, device="cuda")
    for kw in ({}, dict(bias=zero), dict(score="sigmoid", bias=zero),
               dict(score="sigmoid", bias=zero, groups=4, groups_kept=2, group_top=2)):
        _check(mx, x, 6, **kw)


@pytest.mark.parametrize("E,groups", [(256, 8), (96, 8), (128, 64), (510, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_close_groups(mx, E, groups, score, group_top):
    """Every group's two best are 0.7 and 0.2 plus a few steps, the others below -1."""
    print("groups", E, groups, score, group_top, flush=True)
    rng = np.random.default_rng(E + groups)
    T, size = 50, E // groups
    x = np.linspace(-1.0, -5.0, E, dtype=np.float32)[np.argsort(rng.random((T, E)), 1)].reshape(T, groups, size)
    steps = torch.from_numpy(rng.integers(0, 6, (2, T, groups)))
    at = rng.integers(0, size, (T, groups))
    other = (at + 1 + rng.integers(0, size - 1, (T, groups))) % size
    np.put_along_axis(x, at[:, :, None], _nudge(0.7, steps[0]).numpy()[:, :, None], 2)
    np.put_along_axis(x, other[:, :, None], _nudge(0.2, steps[1]).numpy()[:, :, None], 2)
    x = torch.from_numpy(x.reshape(T, E)).cuda()
    for kept in {1, max(1, groups // 3), groups - 1}:
        k = min(8, kept * size)
        kw = dict(score=score, groups=groups, groups_kept=kept, group_top=group_top)
        _check(mx, x, k, **kw)
        _check(mx, x, k, bias=torch.full((E,), 0.03, device="cuda"), **kw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_zeros_of_both_signs_are_equal(mx, dtype):
    print("zeros", dtype, flush=True)
    rng = np.random.default_rng(8)
    x = np.where(rng.random((40, 96)) < 0.5, -0.0, 0.0).astype(np.float32)
    x[:20, ::5] = -1.0
    x = torch.from_numpy(x).cuda().to(dtype)
    zero = torch.zeros(96, device="cuda")
    for kw in ({}, dict(score="sigmoid"), dict(groups=8, groups_kept=2), dict(groups=8, groups_kept=2, group_top=2),
               dict(bias=zero), dict(score="sigmoid", bias=-zero)):
        _check(mx, x, 7, **kw)
