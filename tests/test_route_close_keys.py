"""Routing where keys are closer than FP32 can tell: rows of ties, the last slot's border. Ids are exact, weights to
the bound of tests/test_moe.py (an exponential, a sum, quotients and the scale, the exponential's argument)."""
import numpy as np
import pytest

from tests.test_moe import check_route, fmpq_mod  # noqa: F401  (the fixture)


def above(x):
    return float(np.nextafter(np.float32(x), np.float32(np.inf)))


@pytest.mark.gpu
@pytest.mark.parametrize("E", [33, 64, 100, 128, 256, 500, 512])
@pytest.mark.parametrize("k", [1, 6, 32])
def test_one_key_above_a_row_of_ties(fmpq_mod, E, k):  # noqa: F811
    """All logits equal but one, larger by one step of FP32, at the end, in the middle and at the start."""
    import torch
    x = torch.ones(6, E)
    x[0, E - 1] = x[1, E // 2] = x[2, 0] = above(1.0)
    x[3, E - 2:] = above(1.0)
    x[4, ::2] = above(1.0)
    x[5] = -1.0
    x[5, E - 1] = above(-1.0)
    zero = torch.zeros(E).cuda()
    for score in ("softmax", "sigmoid"):
        check_route(fmpq_mod, x.cuda(), k, score=score)
        check_route(fmpq_mod, x.cuda(), k, score=score, bias=zero)
        check_route(fmpq_mod, x.cuda(), k, score=score, bias=zero + 0.3)


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (512, 2), (96, 3)])
def test_ties_in_groups(fmpq_mod, E, groups):  # noqa: F811
    import torch
    x = torch.ones(3, E)
    x[0, E - 1] = x[1, E // 2] = above(1.0)
    x[2, ::3] = above(1.0)
    bias = torch.full((E,), 0.25).cuda()
    for top_groups in (groups, max(2, groups // 2)):
        for k in (4, 32):
            for score in ("softmax", "sigmoid"):
                check_route(fmpq_mod, x.cuda(), k, score=score, groups=groups, top_groups=top_groups)
                check_route(fmpq_mod, x.cuda(), k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_top=2)


@pytest.mark.gpu
@pytest.mark.parametrize("E", [34, 64, 128, 256, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_border_of_the_last_of_32_slots(fmpq_mod, E, score):  # noqa: F811
    """31 clear winners, then two logits a step apart in either order: the larger one takes the last slot."""
    import torch
    x = torch.linspace(-3, -2, E).repeat(8, 1)
    g = torch.Generator().manual_seed(E)
    for t in range(8):
        place = torch.randperm(E, generator=g)
        x[t, place[:31]] = 2 + torch.rand(31, generator=g)
        lo, hi = sorted(place[31:33].tolist())
        x[t, lo], x[t, hi] = (1.0, above(1.0)) if t % 2 == 0 else (above(1.0), 1.0)
    check_route(fmpq_mod, x.cuda(), 32, score=score)
    check_route(fmpq_mod, x.cuda(), 32, score=score, bias=torch.zeros(E).cuda())
