"""route_scored at the ends of its arithmetic, ids against the float64 oracle:
group sums of choices that cancel or overflow, scores that are equal though
their logits differ."""
import pytest
import torch

from tests.test_gpu_block import N32, check_route, rand
from w4a16_compact_expert_gb300 import block as B

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


# Logits whose 64-bit scores are equal although the logits differ: sigmoids that
# round to 1, softmax terms below the smallest number, values far below 1.
SATURATED = {"sigmoid": (60.0, 50.0, 45.0, 40.0, 38.0, 20.0, 2.0, -3.0, INF),
             "softmax": (0.0, -750.0, -800.0, -900.0, -2000.0, -3e38, -1.0, 1e-20, -1e-25)}


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(4, 2, 1), (32, 6, 4), (60, 5, 6), (64, 8, 8), (64, 8, 1), (256, 8, 8),
                                        (300, 10, 1)])
def test_saturated_scores_tie(score, E, k, groups):
    """Equal 64-bit scores go to the lower index, with and without a bias."""
    T = 256
    g = torch.Generator().manual_seed(E + k)
    vals = torch.tensor(SATURATED[score])
    logits = vals[torch.randint(0, len(vals), (T, E), generator=g)]
    logits[::4] = torch.where(torch.rand(T // 4, E, generator=g) < 0.8, torch.randn(T // 4, E, generator=g), logits[::4])
    if score == "softmax":
        logits[1::16, 0] = 0.0      # so that the rest underflows
        logits[1::16, 1:] = logits[1::16, 1:].clamp_max(-750)
        logits[2::16, E // 2] = INF
    logits = logits.cuda()
    for top in (1,) if groups == 1 else (1, groups // 2):
        for rank in (1, 2):
            if k > top * (E // groups):
                continue
            kw = dict(score=score, groups=groups, top_groups=top, group_rank=rank)
            ids, _ = check_route(logits, None, k, **kw)
            assert torch.equal(ids, check_route(logits, torch.zeros(E, device="cuda"), k, **kw)[0])


def test_saturated_scores_by_hand():
    logits = torch.tensor([[40.0, 50.0, 1.0, 2.0], [50.0, 2.0, 40.0, 45.0]], device="cuda")
    assert check_route(logits, None, 2, score="sigmoid")[0].tolist() == [[0, 1], [0, 2]]
    assert check_route(logits, None, 1, score="sigmoid", groups=2, top_groups=1)[0].tolist() == [[0], [0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups", [(64, 8), (84, 2), (20, 5), (32, 16), (60, 20), (512, 32)])
def test_infinite_biases_in_groups(score, E, groups):
    """A group with one infinite choice is as good as one with two, or with more."""
    logits = rand((24, E), torch.float32, E)
    g = torch.Generator().manual_seed(E)
    for p in (0.05, 0.3, 0.8):
        bias = torch.randn(E, generator=g)
        bias[torch.rand(E, generator=g) < p] = INF
        bias[torch.rand(E, generator=g) < 0.2] = -INF
        bias[torch.rand(E, generator=g) < 0.1] = 3.4e38
        for top in (1, groups // 2, groups - 1):
            for rank in (1, 2):
                check_route(logits, bias.cuda(), min(6, top * (E // groups)), score=score, groups=groups,
                            top_groups=max(top, 1), group_rank=rank)


@pytest.mark.parametrize("E,groups,top", [(16, 1, 1), (64, 8, 2), (60, 5, 2), (300, 1, 1)])
@pytest.mark.parametrize("m", [INF, 900.0, 60.0])
def test_renormalised_softmax_weights_do_not_underflow(E, groups, top, m):
    """A bias selects experts whose softmax is 0 in 64 bits beside the largest logit; the weights are relative to the
    largest chosen, whichever way the token's order was decided."""
    logits = rand((64, E), torch.float32, E)
    logits[:, E - 1] = m
    bias = torch.zeros(E, device="cuda")
    bias[E - 1] = -2000.0
    ids, w = B.route_scored(logits, 3, bias=bias, groups=groups, top_groups=top, renormalize=True, scale=2.0)
    assert m == 60.0 or (ids == torch.arange(3, device="cuda")).all()
    ref = 2.0 * torch.softmax(logits.double().gather(1, ids.long()), -1)
    assert ((w.double() - ref).abs() <= N32 * ref).all()
