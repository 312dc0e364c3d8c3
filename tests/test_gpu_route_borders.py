"""route_scored at the ends of its arithmetic, ids against the float64 oracle:
group sums of choices that cancel or overflow."""
import pytest
import torch

from tests.test_gpu_block import check_route, rand

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 8), (256, 8), (48, 8), (60, 5)])
@pytest.mark.parametrize("m", [30.0, 100.0, 1000.0])
def test_group_sums_that_cancel(score, E, groups, m):
    """The two largest choices of a group lie near +m and -m, so their sum is near 1 and its error that of m;
    the groups' sums differ by less."""
    T, per = 192, E // groups
    logits = rand((T, per), torch.float32, E, 1.5).repeat(1, groups)
    noise = rand((T, E), torch.float32, E + 1)
    for i, std in enumerate((1e-6, 1e-5, 1e-4)):
        logits[i::3] += noise[i::3] * std
    bias = torch.full((groups, per), -m, device="cuda")
    bias[:, per // 2] = m
    for top in (1, groups // 2, groups - 1):
        check_route(logits, bias.view(-1), 4 if per * top >= 4 else 1, score=score, groups=groups, top_groups=top,
                    group_rank=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("per", [4, 6])
def test_group_sums_that_overflow(score, per):
    """Sums of two choices beyond FP32, of either sign, beside groups without eligible experts and infinite biases."""
    groups = 8
    logits = rand((16, groups * per), torch.float32, 5)
    logits[1, 2 * per:] = -INF
    logits[2, :6 * per] = -INF
    rows = [(-3.3e38, -3e38, -2e38, -3.4e38, -2.5e38, -2.2e38, -3.1e38, -INF),
            (-INF, -3e38, -3.3e38, -3.2e38, -3.4e38, -INF, -3.25e38, -3.1e38),
            (3e38, 3.2e38, 2e38, 3.3e38, 1e38, -3e38, 3.1e38, 0.0),
            (3e38, INF, 2e38, 0.5, INF, 0.0, -INF, 3.4e38)]
    for row in rows:
        bias = torch.tensor(row, device="cuda").repeat_interleave(per)
        for top in (1, 2, 3, 5, 7):
            for rank in (1, 2):
                check_route(logits, bias, 3, score=score, groups=groups, top_groups=top, group_rank=rank)
        alone = bias.clone().view(groups, per)
        alone[::2, 1:] = -INF   # one choice, or two
        check_route(logits, alone.view(-1), 1, score=score, groups=groups, top_groups=2, group_rank=2)
