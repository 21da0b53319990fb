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


def far_logits(T, E, chosen, distance, score, seed):
    """Logits whose `chosen` experts have scores near exp(-distance): under softmax that far below the others, under sigmoid with all of them
    (another expert's score would be the sum's)."""
    L = torch.randn(T, E, generator=torch.Generator().manual_seed(seed)).numpy()
    if score == "sigmoid":
        return L - np.float32(distance)
    L[:, chosen] -= np.float32(distance)
    return L


@pytest.mark.parametrize("distance", [0.0, 60.0, 69.5, 80.0, 84.0, 87.0, 88.0, 95.0, 104.0, 200.0, 690.0])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups", [(3, 8, 1), (70, 64, 8), (40, 320, 4)])
def test_renormalised_gates_and_their_gradient_at_any_distance(gpu_lib, T, E, groups, score, distance):
    """A bias chooses experts whose scores, or their sum, are below fp32's normal range: the gates are their shares all the same."""
    k, chosen = 4, [1, 3, 4, 6]
    L = far_logits(T, E, chosen, distance, score, E)
    b = np.zeros(E, np.float32)
    b[chosen] = 2.0
    r = gpu_lib.moe_group_route(torch.from_numpy(L).cuda(), torch.from_numpy(b).cuda(), k, groups, 1, score=score, scale=2.5)
    ok(gpu_lib)
    L64 = L.astype(np.float64)
    want = O.route(L64, b, k, groups, 1, score, 2, True, 2.5)
    assert (np.sort(want["ids"], 1) == chosen).all()
    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])
    # exponentials (4 half steps each, and 2 for each unit of their argument, up to 2^-100: 70), the sums of k and the quotient
    rel = (32 + 2 * min(distance + 8, 80)) * EPS
    np.testing.assert_allclose(r["gates"].double().cpu().numpy(), want["gates"], rtol=rel, atol=1e-37)
    dg = torch.randn(T, k, generator=torch.Generator().manual_seed(7))
    f = r["f"].double().cpu().numpy()
    for d_aux in (0.0, 0.7):
        d = gpu_lib.moe_group_route_backward(torch.from_numpy(L).cuda(), r["topk_ids"], dg.cuda(), r["f"], score=score, scale=2.5, alpha=0.5, d_aux=d_aux)
        ok(gpu_lib)
        dwant = O.backward(L64, want["ids"], dg.double().numpy(), f, score, True, 2.5, 0.5, d_aux)
        # the gates' part: share times a difference of gates' gradients; the balance loss's: share of all scores times coefficients
        s = O.scores(L64, score)
        share = np.zeros_like(s)
        np.put_along_axis(share, want["ids"], want["gates"], 1)
        big = share * 2 * np.abs(dg.numpy()).max() + d_aux * 0.5 * E / T * s / s.sum(1, keepdims=True) * 2
        # (under softmax <dp, p> holds all of the chosen experts' terms, which cancel: in the ordinary case to roundings of their largest)
        big += s * big.max(1, keepdims=True)
        assert (np.abs(d.double().cpu().numpy() - dwant) <= (2 * rel + (96 + E) * EPS) * big + 1e-37).all()


def test_renormalised_gates_where_nothing_is_chosen_alive(gpu_lib):
    """Masked experts, and scores that 64 bits do not hold either: gates 0, and no gradient from them."""
    for low in (-float("inf"), -3.4e38, -1000.0):
        for score in ("sigmoid", "softmax"):
            L = torch.zeros(20, 64)
            L[:, :32] = low
            b = torch.zeros(64)
            b[:32] = 5.0
            r = gpu_lib.moe_group_route(L.cuda(), b.cuda(), 4, 2, 1, score=score, best=1) if low != -float("inf") else \
                gpu_lib.moe_group_route(torch.full_like(L, low).cuda(), b.cuda(), 4, 2, 1, score=score, best=1)
            ok(gpu_lib)
            assert (r["topk_ids"].cpu() == torch.arange(4)).all() and (r["gates"] == 0).all(), (low, score)
            d = gpu_lib.moe_group_route_backward(L.cuda(), r["topk_ids"], torch.randn(20, 4).cuda(), r["f"], score=score, d_aux=0.0)
            assert (d == 0).all(), (low, score)


@pytest.mark.parametrize("distance", [0.0, 60.0, 75.0, 86.0, 88.0, 104.0, 300.0, 690.0])
@pytest.mark.parametrize("T,E", [(5, 8), (60, 96), (30, 320), (2, 1024)])
@pytest.mark.parametrize("renorm", [True, False])
def test_shares_of_sigmoid_scores_that_are_all_small(gpu_lib, T, E, distance, renorm):
    """P, the balance loss and its gradient are of s_e / sum s, whatever the sum."""
    g = torch.Generator().manual_seed(E)
    L = torch.randn(T, E, generator=g) - distance
    L[:, torch.rand(E, generator=g) < 0.2] = -float("inf")
    L[:, :2] = torch.randn(T, 2, generator=g) - distance
    L64 = L.double().numpy()
    r = gpu_lib.moe_group_route(L.cuda(), None, 2, 1, 1, renorm=renorm)
    ok(gpu_lib)
    want = O.route(L64, None, 2, 1, 1, "sigmoid", 2, renorm, 1.0)
    # a score's exponential (2 half steps a unit of its argument up to where 64 bits take over, 70) and quotient, sums of E / 32 + 5 terms and of T
    rel = (32 + 2 * min(distance + 8, 80) + E / 32 + T) * EPS
    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])
    np.testing.assert_allclose(r["P"].double().cpu().numpy(), want["P"], rtol=rel, atol=1e-37)
    np.testing.assert_allclose(r["aux"].item(), want["aux"], rtol=rel + E * EPS)
    d = gpu_lib.moe_group_route_backward(L.cuda(), r["topk_ids"], torch.zeros(T, 2).cuda(), r["f"], renorm=renorm, alpha=0.5, d_aux=0.7)
    ok(gpu_lib)
    f = r["f"].double().cpu().numpy()
    dwant = O.backward(L64, want["ids"], np.zeros((T, 2)), f, "sigmoid", renorm, 1.0, 0.5, 0.7)
    s = O.scores(L64, "sigmoid")
    big = 0.35 * E / T * s / s.sum(1, keepdims=True) * 2
    assert (np.abs(d.double().cpu().numpy() - dwant) <= 2 * rel * big + 1e-37).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_the_lowest_finite_logits_come_before_masked_ones(gpu_lib, score):
    """Without a bias: a masked expert's -1e30 is below every score, not below every logit."""
    low, out = np.finfo(np.float32).min, -np.inf
    r = gpu_lib.moe_group_route(torch.tensor([[out, -3e38, -1e31, out, np.nan if score == "sigmoid" else out, low]]).cuda(), None, 6, 1, 1, score=score)
    ok(gpu_lib)
    assert r["topk_ids"].tolist() == [[2, 1, 5, 0, 3, 4]]
    # among many: a few that only their last bits tell apart, and more than a warp has lanes
    g = np.random.default_rng(4)
    for E, groups, top_groups, live in ((64, 1, 1, 5), (64, 4, 2, 9), (256, 1, 1, 100), (256, 8, 3, 200), (900, 9, 4, 400), (1024, 1, 1, 3)):
        L = np.full((30, E), out, np.float32)
        for row in L:
            row[g.permutation(E)[:live]] = low
        steps = g.integers(0, 40, size=L.shape)
        L = np.where(np.isneginf(L), L, (low * (1.0 - steps * 2.0**-24)).astype(np.float32))
        r = gpu_lib.moe_group_route(torch.from_numpy(L).cuda(), None, 8, groups, top_groups, score=score)
        ok(gpu_lib)
        want = O.route(L.astype(np.float64), None, 8, groups, top_groups, score, 2, True, 1.0)
        np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])


@pytest.mark.parametrize("E", [128, 256, 384, 512, 768, 1024])
def test_logits_on_no_boundary_are_routed_as_those_on_one(gpu_lib, E):
    """Rows on 16 bytes are read in pieces of four logits, others one by one."""
    g = torch.Generator().manual_seed(E)
    flat = torch.zeros(37 * E + 1, device="cuda")
    L = torch.randn(37, E, generator=g).cuda()
    flat[1:].copy_(L.view(-1))
    b = (torch.randn(E, generator=g) * 0.05).cuda()
    for bias in (None, b):
        for score in ("sigmoid", "softmax"):
            on, off = (gpu_lib.moe_group_route(x, bias, 8, 8, 3, score=score) for x in (L, flat[1:].view(37, E)))
            ok(gpu_lib)
            assert all(torch.equal(on[name], off[name]) for name in on)


@pytest.mark.parametrize("level", [-22.0, -45.0, -62.0, -66.0, -68.0])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_shares_of_scores_that_are_nothing_beside_larger_ones(gpu_lib, score, level):
    """Chosen scores of exp(level) and others down to below 2^-126, where the larger ones' sum is an ordinary number: the small shares
    are there to 2^-86 (fp32's smallest number in a sum of 2^-40)."""
    L = torch.full((5, 16), level - 3.0)
    L[:, [1, 4, 6, 7]] = torch.tensor([level, level - 0.7, -88.5, -95.0]) + torch.randn(5, 4, generator=torch.Generator().manual_seed(3)) * 0.2
    if score == "softmax":
        L[:, 12] = 0.0
    b = torch.zeros(16)
    b[[1, 4, 6, 7]] = 2.0
    r = gpu_lib.moe_group_route(L.cuda(), b.cuda(), 4, 2, 1, score=score)
    ok(gpu_lib)
    L64 = L.double().numpy()
    want = O.route(L64, b.numpy(), 4, 2, 1, score, 2, True, 1.0)
    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])
    rel = (32 + 2 * 100) * EPS
    np.testing.assert_allclose(r["gates"].double().cpu().numpy(), want["gates"], rtol=rel, atol=2.0**-85)
    np.testing.assert_allclose(r["P"].double().cpu().numpy(), want["P"], rtol=rel, atol=2.0**-85)
    dg = torch.randn(5, 4, generator=torch.Generator().manual_seed(7))
    d = gpu_lib.moe_group_route_backward(L.cuda(), r["topk_ids"], dg.cuda(), r["f"], score=score, d_aux=0.0)
    ok(gpu_lib)
    dwant = O.backward(L64, want["ids"], dg.double().numpy(), r["f"].double().cpu().numpy(), score, True, 1.0, 0.01, 0.0)
    share = np.zeros((5, 16))
    np.put_along_axis(share, want["ids"], want["gates"], 1)
    # a share times a difference of gates' gradients; under softmax, in the ordinary way, <dp, p> cancels to roundings of the largest term
    s = O.scores(L64, score)
    big = 2 * float(dg.abs().max()) * (share + s * share.max(1, keepdims=True))
    assert (np.abs(d.double().cpu().numpy() - dwant) <= 2 * rel * big + 2.0**-83).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_tokens_of_small_sums_among_others(gpu_lib, score):
    """More tokens than all warps take in 32 steps each: every row as in a call of its own, and with the logits' gradient in their place."""
    T, E = 400_000, 32
    g = torch.Generator("cuda").manual_seed(1)
    L = torch.randn(T, E, device="cuda", generator=g)
    far = torch.rand(T, device="cuda", generator=g) < 0.4
    if score == "sigmoid":
        L[far] -= 90.0
    else:
        L[far, :8] -= 90.0
    L[::97] = -float("inf")
    b = torch.zeros(E, device="cuda")
    b[:8] = 2.0
    dg = torch.randn(T, 4, device="cuda", generator=g)
    r = gpu_lib.moe_group_route(L, b, 4, 4, 1, score=score)
    d = gpu_lib.moe_group_route_backward(L, r["topk_ids"], dg, r["f"], score=score, d_aux=0.0)
    ok(gpu_lib)
    assert torch.isfinite(r["gates"]).all() and torch.isfinite(d).all()
    live = torch.isfinite(L).any(1)
    assert (r["gates"].sum(1) - live.float()).abs().max().item() <= 32 * EPS
    # P adds the shares of some 400 of a block's tokens in turn, then the blocks'
    assert abs(r["P"].sum().item() - live.double().mean().item()) <= (64 + T / 800) * EPS
    for lo in (0, 155_600, 311_200, T - 50):
        part = slice(lo, lo + 50)
        one = gpu_lib.moe_group_route(L[part].contiguous(), b, 4, 4, 1, score=score)
        d_one = gpu_lib.moe_group_route_backward(L[part].contiguous(), one["topk_ids"], dg[part].contiguous(), one["f"], score=score, d_aux=0.0)
        ok(gpu_lib)
        assert torch.equal(one["gates"], r["gates"][part]) and torch.equal(one["topk_ids"], r["topk_ids"][part]) and torch.equal(d_one, d[part])
    gpu_lib.moe_group_route_backward(L, r["topk_ids"], dg, r["f"], score=score, d_aux=0.0, d_logits=L)
    ok(gpu_lib)
    assert torch.equal(L, d)
