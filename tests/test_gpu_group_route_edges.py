"""Routing by groups on the GPU where scores are far below 1 or below what fp32 holds, and where logits are fp32's lowest."""
import numpy as np
import pytest
import torch

from oracle import group_route_oracle as O

pytestmark = pytest.mark.gpu

EPS = 2.0**-24          # half a step of fp32, relative


def ok(moe):
    torch.cuda.synchronize()
    assert moe.moe_check_device_error() == moe.MOE_OK, moe.moe_last_error_string()


def near_groups(T, E, groups, best, level, seed):
    """Logits [T, E] whose first group is far above the others (near 0), and whose second and third have scores, exp(level) about, that
    are next to each other: the last of the third's `best` is the fp32 number that makes both sums the same."""
    g = np.random.default_rng(seed)
    per = E // groups
    L = (level - 6.0 - 3.0 * g.random((T, E))).astype(np.float32)
    L[:, 0] = g.normal(size=T)
    one, two = L[:, per:2 * per], L[:, 2 * per:3 * per]
    for group in (one, two):
        group[:, per - 1] = level + 0.5 * g.random(T)
    if best == 1:
        two[:, per - 1] = one[:, per - 1]
    else:
        one[:, 0] = level + g.random(T)
        two[:, per - 1] = np.minimum(two[:, per - 1], one[:, 0])
        want = np.logaddexp(one[:, 0].astype(np.float64), one[:, per - 1].astype(np.float64))
        last = two[:, per - 1].astype(np.float64)
        two[:, 0] = want + np.log1p(-np.exp(last - want))
    steps = g.integers(-2, 3, size=T)
    for _ in range(2):          # up to two units in the last place beside it
        x = two[:, 0 if best == 2 else per - 1]
        x[:] = np.where(steps > 0, np.nextafter(x, np.float32(np.inf)), np.where(steps < 0, np.nextafter(x, np.float32(-np.inf)), x))
        steps -= np.sign(steps)
    return L


@pytest.mark.parametrize("level", [-3.0, -20.0, -30.0, -50.0, -70.0, -86.5, -88.0, -120.0])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,T", [(6, 3, 4000), (256, 8, 1000), (900, 9, 300)])
def test_groups_of_small_scores_are_chosen_exactly(gpu_lib, E, groups, T, score, level):
    """Without a bias: what fp32 loses of a small score grows with its logit's distance, and below 2^-126 all of it."""
    for best in (1, 2):
        L = near_groups(T, E, groups, best, level, E + best)
        r = gpu_lib.moe_group_route(torch.from_numpy(L).cuda(), None, 3, groups, 2, score=score, best=best)
        ok(gpu_lib)
        want = O.route(L.astype(np.float64), None, 3, groups, 2, score, best, True, 1.0)
        np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])


def test_a_group_that_leads_in_32_bits_alone(gpu_lib):
    for L in ([-51.9682731628418, -52.71291732788086, -51.97492599487305, -52.69904708862305],
              [-32.525688, -28.630362, -32.475475, -28.631409]):
        L = np.array([L], np.float32)
        r = gpu_lib.moe_group_route(torch.from_numpy(L).cuda(), None, 2, 2, 1)
        ok(gpu_lib)
        want = O.route(L.astype(np.float64), None, 2, 2, 1, "sigmoid", 2, True, 1.0)
        assert (want["ids"] >= 2).all()
        np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])
