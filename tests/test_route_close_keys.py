"""Routing where keys are closer than FP32 can tell: rows of ties, the last slot's border, sums of large keys
that cancel; and weights of scores below FP32's range. Ids are exact, weights to the bound of tests/test_moe.py (an
exponential, a sum, quotients and the scale, the exponential's argument)."""
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


@pytest.mark.gpu
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 32), (256, 4), (60, 5), (96, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size,spread", [(1000.0, 1.0), (3e7, 1.0), (1000.0, 1e-4), (1e5, 1e-2), (1e5, 1.0)])
def test_groups_whose_best_keys_cancel(fmpq_mod, E, groups, score, size, spread):  # noqa: F811
    """A bias of +size beside one of -size: a group's sum is the two scores', about or far below a step of FP32 at
    `size` apart from the next group's."""
    import torch
    per = E // groups
    g = torch.Generator().manual_seed(E)
    x = torch.full((12, E), float("-inf"))
    x[:, 0::per] = torch.randn(12, groups, generator=g) * spread
    x[:, 1::per] = torch.randn(12, groups, generator=g) * spread
    bias = torch.zeros(E)
    bias[0::per], bias[1::per] = size, -size
    check_route(fmpq_mod, x.cuda(), 3, score=score, bias=bias.cuda(), groups=groups, top_groups=2, group_top=2)


@pytest.mark.gpu
def test_group_sums_past_the_range_of_fp32(fmpq_mod):  # noqa: F811
    import torch
    x = torch.zeros(2, 64)
    bias = torch.full((64,), -1.0)
    bias[0:8], bias[16:24], bias[40:48] = 2e38, 3e38, 2.5e38
    for score in ("softmax", "sigmoid"):
        check_route(fmpq_mod, x.cuda(), 6, score=score, bias=bias.cuda(), groups=8, top_groups=1, group_top=2)
        check_route(fmpq_mod, x[:, :60].cuda(), 6, score=score, bias=bias[:60].cuda(), groups=5, top_groups=1, group_top=2)


@pytest.mark.gpu
@pytest.mark.parametrize("E", [8, 60, 256])
def test_renormalized_weights_of_tiny_scores(fmpq_mod, E):  # noqa: F811
    """Scores below FP32's range still have a sum in 64 bits, so their weights are their ratios."""
    import torch
    g = torch.Generator().manual_seed(E)
    lowest = torch.full((2, E), torch.finfo(torch.float32).min)     # masked by the lowest value: a score of 0
    lowest[0, 0] = 1.0
    bias = torch.linspace(0, 1, E)
    x = torch.randn(3, E, generator=g) - 100.0      # sigmoid: about 1e-44
    x[1] -= 300.0
    x[2] = -87.5 + torch.rand(E, generator=g)       # the subnormal border
    for logits in (x, lowest):
        check_route(fmpq_mod, logits.cuda(), 4, score="sigmoid", renormalize=True)
        check_route(fmpq_mod, logits.cuda(), 4, score="sigmoid", renormalize=True, bias=bias.cuda(), scale=2.5)
    # softmax: the biases keep the expert out that holds nearly all of the scores
    bias[0] = -5.0
    y = torch.randn(2, E, generator=g)
    y[0, 0], y[1, 0] = 150.0, 500.0
    infinite = torch.randn(1, E, generator=g)
    infinite[0, 0] = float("inf")
    for logits in (y, lowest, infinite):
        check_route(fmpq_mod, logits.cuda(), 4, renormalize=True, bias=bias.cuda())
