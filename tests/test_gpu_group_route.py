"""Routing by groups on the GPU against the float64 oracle: the choice exactly, the floats within bounds that count roundings."""
import numpy as np
import pytest
import torch

from oracle import group_route_oracle as O

pytestmark = pytest.mark.gpu

EPS = 2.0**-24          # half a step of fp32, relative


def ok(moe):
    torch.cuda.synchronize()
    assert moe.moe_check_device_error() == moe.MOE_OK, moe.moe_last_error_string()


def logits_of(T, E, seed, masked=0.0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    L = torch.randn(T, E, generator=g) * spread
    if masked:
        L[torch.rand(T, E, generator=g) < masked] = -float("inf")
    return L


def bias_of(E, seed):
    return torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 0.05


def compare(r, want, T, L):
    # a score is off by its exponential (2 units), the logit's difference (|L - max| half steps) and three roundings; a gate adds the sum of
    # up to 16 and two more: 32 half steps and one for each unit of the logits' range; P averages scores, each block's T / 8 of
    # them added in turn
    span = float(np.max(np.abs(np.where(np.isfinite(L), L, 0.0)), initial=0.0)) * 2
    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])
    np.testing.assert_array_equal(r["counts"].cpu().numpy(), want["counts"])
    np.testing.assert_allclose(r["gates"].double().cpu().numpy(), want["gates"], rtol=(32 + span) * EPS, atol=1e-37)
    np.testing.assert_allclose(r["f"].double().cpu().numpy(), want["f"], rtol=2 * EPS)
    np.testing.assert_allclose(r["P"].double().cpu().numpy(), want["P"], rtol=(64 + span + T / 8) * EPS, atol=1e-37)
    np.testing.assert_allclose(r["aux"].item(), want["aux"], rtol=(96 + span + T / 8 + L.shape[1]) * EPS)


SHAPES = [  # T, E, k, groups, top_groups, best
    (1, 1, 1, 1, 1, 1), (3, 4, 2, 2, 1, 2), (5, 16, 4, 4, 2, 2), (7, 32, 8, 8, 4, 2), (9, 33, 3, 3, 2, 2), (4, 64, 16, 8, 2, 1),
    (33, 72, 6, 8, 3, 2), (17, 96, 5, 32, 3, 2), (65, 160, 6, 8, 3, 1), (29, 96, 8, 8, 4, 2), (31, 160, 8, 8, 3, 2), (33, 192, 8, 8, 2, 2), (23, 384, 8, 8, 4, 2), (14, 224, 7, 7, 3, 2), (130, 256, 8, 8, 4, 2), (40, 256, 8, 1, 1, 1), (12, 300, 7, 6, 2, 2),
    (21, 512, 8, 16, 4, 2), (6, 976, 16, 16, 5, 2), (11, 1024, 16, 32, 8, 2), (3, 1024, 4, 1, 1, 2), (2500, 256, 8, 8, 4, 2)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased,renorm,scale,masked", [(True, True, 2.5, 0.0), (False, False, 16.0, 0.0), (True, False, 1.0, 0.1),
                                                        (False, True, 1.0, 0.3)])
@pytest.mark.parametrize("T,E,k,groups,top_groups,best", SHAPES)
def test_route_and_its_gradient(gpu_lib, score, biased, renorm, scale, masked, T, E, k, groups, top_groups, best):
    L, b = logits_of(T, E, T * 31 + E, masked), bias_of(E, E) if biased else None
    r = gpu_lib.moe_group_route(L.cuda(), b.cuda() if biased else None, k, groups, top_groups, score=score, best=best, renorm=renorm, scale=scale)
    ok(gpu_lib)
    L64 = L.double().numpy()
    want = O.route(L64, b.numpy() if biased else None, k, groups, top_groups, score, best, renorm, scale)
    compare(r, want, T, L64)
    dg = torch.randn(T, k, generator=torch.Generator().manual_seed(7))
    d = gpu_lib.moe_group_route_backward(L.cuda(), r["topk_ids"], dg.cuda(), r["f"], score=score, renorm=renorm, scale=scale, alpha=0.5, d_aux=0.7)
    ok(gpu_lib)
    dwant = O.backward(L64, want["ids"], dg.double().numpy(), r["f"].double().cpu().numpy(), score, renorm, scale, 0.5, 0.7)
    # each term is bounded by scale * |d_g| / S (S >= a chosen score) times s; the sums of E products add E half steps of the largest
    s = O.scores(L64, score)
    S = np.take_along_axis(s, want["ids"], 1).sum(1, keepdims=True)
    big = scale * np.abs(dg.numpy()).max() * (1.0 / np.where(S == 0, 1.0, S) if renorm else 1.0) + 0.35 * E / T / np.where(s.sum(1, keepdims=True) == 0, 1.0, s.sum(1, keepdims=True)) + 0.35 * E / T
    err = np.abs(d.double().cpu().numpy() - dwant)
    assert (err <= (96 + E) * EPS * big * s + 1e-37).all(), float((err / (big * s + 1e-37)).max() / EPS)


def test_ties_go_to_the_lower_index(gpu_lib):
    # all equal, in pairs, and equal sums of different members
    for L in (torch.zeros(9, 256), torch.arange(128).repeat_interleave(2).float().repeat(4, 1) * 0.01, torch.full((5, 256), 30.0),
              torch.full((5, 256), -float("inf"))):
        for score in ("sigmoid", "softmax"):
            for b in (None, torch.zeros(256), torch.full((256,), 0.25)):
                r = gpu_lib.moe_group_route(L.cuda(), None if b is None else b.cuda(), 8, 8, 4, score=score)
                ok(gpu_lib)
                want = O.route(L.double().numpy(), None if b is None else b.numpy(), 8, 8, 4, score, 2, True, 1.0)
                np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])
                assert torch.isfinite(r["gates"]).all() and torch.isfinite(r["P"]).all()
                d = gpu_lib.moe_group_route_backward(L.cuda(), r["topk_ids"], torch.ones(L.shape[0], 8).cuda(), r["f"], score=score)
                assert torch.isfinite(d).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_scores_next_to_each_other_are_ordered_exactly(gpu_lib, score):
    # biases that bring the scores of a token's experts within 2^-26 of one another: 32 bits see ties or the wrong order
    g = torch.Generator().manual_seed(1)
    L = torch.randn(64, generator=g) * 0.5
    s = O.scores(L.double().numpy()[None], score)[0]
    b = torch.from_numpy((0.6 - s).astype(np.float32))      # s + b = 0.6 up to b's rounding
    r = gpu_lib.moe_group_route(L.repeat(40, 1).cuda(), b.cuda(), 8, 4, 2, score=score)
    ok(gpu_lib)
    want = O.route(L.double().numpy()[None], b.numpy(), 8, 4, 2, score, 2, True, 1.0)
    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), np.repeat(want["ids"], 40, 0))
    np.testing.assert_allclose(r["gates"][0].double().cpu().numpy(), want["gates"][0], rtol=64 * EPS)


def test_a_bias_decides_the_choice_and_not_the_gate(gpu_lib):
    L = torch.zeros(3, 16)
    b = torch.zeros(16)
    b[[2, 3, 13]] = 5.0
    r = gpu_lib.moe_group_route(L.cuda(), b.cuda(), 3, 4, 2, renorm=False)
    ok(gpu_lib)
    assert r["topk_ids"].tolist() == [[2, 3, 13]] * 3 and r["gates"].tolist() == [[0.5, 0.5, 0.5]] * 3


def test_no_tokens_nan_and_foreign_ids(gpu_lib):
    r = gpu_lib.moe_group_route(torch.empty(0, 64).cuda(), None, 4, 4, 2)
    assert r["counts"].sum().item() == 0 and r["aux"].item() == 0.0 and r["P"].abs().sum().item() == 0.0
    assert gpu_lib.moe_group_route_backward(torch.empty(0, 64).cuda(), r["topk_ids"], r["gates"], r["f"]).shape == (0, 64)
    L = logits_of(4, 64, 5)
    L[1, 7] = float("nan")
    for score in ("sigmoid", "softmax"):
        r = gpu_lib.moe_group_route(L.cuda(), None, 4, 4, 2, score=score)
        ids = r["topk_ids"].cpu()
        assert ((ids >= 0) & (ids < 64)).all() and not (ids[1] == 7).any() and len(set(ids[1].tolist())) == 4
        assert torch.isfinite(r["gates"][[0, 2, 3]]).all() and (score == "sigmoid" or r["gates"][1].isnan().all())
    bad = r["topk_ids"].clone()
    bad[0, 0] = 64
    gpu_lib.moe_group_route_backward(logits_of(4, 64, 5).cuda(), bad, torch.ones(4, 4).cuda(), r["f"])
    torch.cuda.synchronize()
    assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("T,h,E,groups,dtype", [(5, 64, 16, 4, "bf16"), (300, 256, 32, 8, "bf16"), (33, 128, 256, 8, "bf16"), (700, 256, 64, 8, "bf16"),
                                               (9, 64, 8, 4, "fp32"), (40, 72, 96, 8, "fp32"), (64, 128, 66, 6, "bf16"), (0, 64, 64, 4, "bf16")])
def test_router_is_the_route_of_its_logits(gpu_lib, T, h, E, groups, dtype):
    dt = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    g = torch.Generator().manual_seed(T + E)
    x, w = (torch.randn(T, h, generator=g)).to(dt).cuda(), (torch.randn(h, E, generator=g) / h**0.5).to(dt).cuda()
    b = bias_of(E, 2).cuda()
    packed = gpu_lib.moe_pack_router_weight(w)
    r = gpu_lib.moe_group_router(x, packed, E, b, min(4, E // groups * 2), groups, 2, scale=2.5)
    again = gpu_lib.moe_group_route(r["logits"], b, min(4, E // groups * 2), groups, 2, scale=2.5)
    ok(gpu_lib)
    for name in again:
        assert torch.equal(r[name], again[name]), name
    none = gpu_lib.moe_group_router(x, packed, E, b, min(4, E // groups * 2), groups, 2, scale=2.5, want_logits=False)
    assert none["logits"] is None and torch.equal(none["gates"], r["gates"]) and torch.equal(none["topk_ids"], r["topk_ids"])
    if T:
        # fp32 sums of h products: h half steps of the sum of magnitudes
        want, mag = x.double() @ w.double(), x.double().abs() @ w.double().abs()
        assert ((r["logits"].double() - want).abs() <= (h + 4) * EPS * mag).all()


def test_captured_and_on_another_stream(gpu_lib):
    L, b = logits_of(500, 256, 9).cuda(), bias_of(256, 1).cuda()
    ws = torch.empty(gpu_lib.moe_group_route_workspace_size(500, 256), dtype=torch.uint8, device="cuda")
    first = gpu_lib.moe_group_route(L, b, 8, 8, 4, ws=ws)
    d = gpu_lib.moe_group_route_backward(L, first["topk_ids"], torch.ones(500, 8).cuda(), first["f"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = {k: torch.empty_like(v) for k, v in first.items()}
    d2 = torch.empty_like(d)
    one = torch.ones(500, 8).cuda()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        gpu_lib.moe_group_route(L, b, 8, 8, 4, ws=ws, **out)
        gpu_lib.moe_group_route_backward(L, out["topk_ids"], one, out["f"], d_logits=d2)
    for seed in (9, 10, 9):
        L.copy_(logits_of(500, 256, seed))
        graph.replay()
        torch.cuda.synchronize()
    assert all(torch.equal(out[k], first[k]) for k in out) and torch.equal(d, d2)
    ok(gpu_lib)


def test_logits_past_32_bit_offsets(gpu_lib):
    T, E = 2_200_000, 1024
    L = torch.zeros(T, E, device="cuda")
    L[-5:] = logits_of(5, E, 3).cuda()
    r = gpu_lib.moe_group_route(L, None, 8, 8, 4)
    part = gpu_lib.moe_group_route(L[-5:].contiguous(), None, 8, 8, 4)
    ok(gpu_lib)
    assert torch.equal(r["topk_ids"][-5:], part["topk_ids"]) and torch.equal(r["gates"][-5:], part["gates"])
    assert (r["topk_ids"][:-5] == torch.arange(8, device="cuda")).all() and r["counts"].sum().item() == 8 * T
    del L
    torch.cuda.empty_cache()


def test_many_ties_of_few_values(gpu_lib):
    # logits of a coarse grid: ties in every token, across lanes and groups, with and without equal biases
    g = torch.Generator().manual_seed(2)
    for E, groups in ((256, 8), (160, 8), (96, 32), (512, 4)):
        L = torch.randint(-4, 5, (60, E), generator=g).float() * 0.5
        for b in (None, torch.randint(0, 3, (E,), generator=g).float() * 0.125):
            for score in ("sigmoid", "softmax"):
                for best in (1, 2):
                    r = gpu_lib.moe_group_route(L.cuda(), None if b is None else b.cuda(), 6, groups, 3, score=score, best=best)
                    ok(gpu_lib)
                    want = O.route(L.double().numpy(), None if b is None else b.numpy(), 6, groups, 3, score, best, True, 1.0)
                    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])


@pytest.mark.parametrize("E", [4, 64])
def test_large_biases_that_cancel_in_a_groups_score(gpu_lib, E):
    """The first group's two best scores are near 1000 and -1000, where fp32 steps by 6e-5, and their sum is near 1: in 32 bits it is
    1 + 6e-5, above the other group's 1 + 4e-5, and exactly it is 1 + 3e-5, below."""
    per = E // 2
    L = np.full((3, E), -1.0, np.float32)
    bias = np.full(E, -2000.0, np.float32)
    L[:, 0], L[:, 1], L[:, per], L[:, per + 1] = 1.28e-4, 0.0, 1.6e-4, 0.0
    bias[[0, 1, per, per + 1]] = 1000.0, -1000.0, 0.0, 0.0
    want = O.route(L.astype(np.float64), bias.astype(np.float64), 2, 2, 1, "sigmoid", 2, True, 1.0)
    assert (want["ids"] >= per).all()
    r = gpu_lib.moe_group_route(torch.from_numpy(L).cuda(), torch.from_numpy(bias).cuda(), 2, 2, 1)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])


@pytest.mark.parametrize("E,groups,top_groups,k", [(256, 8, 4, 8), (160, 8, 3, 6), (96, 32, 5, 4), (64, 2, 1, 16), (66, 6, 2, 5), (40, 8, 7, 3), (1024, 4, 3, 16),
                                                   (32, 32, 9, 9), (296, 8, 3, 8), (200, 4, 2, 8), (992, 16, 5, 9), (900, 9, 4, 7), (35, 5, 2, 6),
                                                   (51, 17, 6, 5), (1023, 3, 2, 12), (144, 16, 8, 8), (1020, 17, 8, 10), (150, 3, 3, 10),
                                                   (7, 7, 2, 2), (1, 1, 1, 1)])
def test_near_ties_in_every_token(gpu_lib, E, groups, top_groups, k):
    """Logits and biases of a few values, off by some units in the last place: the order of most groups and experts is lost in 32 bits. With
    large biases too, the same for the experts of a group's place in all groups, so that the groups stay close."""
    g = torch.Generator().manual_seed(E)
    T, per = 150, E // groups
    for spread in (0.0, 0.2, 300.0):
        values, steps = torch.randn(5, generator=g), lambda *n: torch.randint(-3, 4, n, generator=g).float() * 2.0**-22
        L = values[torch.randint(0, 5, (T, E), generator=g)] * (1 + steps(T, E))
        L[torch.rand(T, E, generator=g) < 0.05] = -float("inf")
        b = (torch.randn(per, generator=g) * spread).repeat(groups) * (1 + steps(E) * 0.25)
        for score in ("sigmoid", "softmax"):
            for best in (1, 2):
                if best > per:
                    continue
                r = gpu_lib.moe_group_route(L.cuda(), b.cuda() if spread else None, k, groups, top_groups, score=score, best=best)
                ok(gpu_lib)
                want = O.route(L.double().numpy(), b.double().numpy() if spread else None, k, groups, top_groups, score, best, True, 1.0)
                np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])


def test_infinite_biases_choose_and_exclude(gpu_lib):
    """+inf: chosen whatever its score, groups of two such by index; -inf: behind all others; a sum of both: as masked."""
    L = logits_of(70, 64, 9)
    b = bias_of(64, 10)
    for plus, minus in (([5], []), ([5, 9, 20, 21, 40, 41, 56, 63], []), ([], list(range(8, 24))), ([3, 33], [0, 1, 60]),
                        (list(range(0, 64, 8)), [e for e in range(64) if e % 8]),            # +inf and -inf: every group's sum
                        ([0, 8, 16, 24, 32, 40], [e for e in range(48) if e % 8])):          # and of all but two
        bias = b.clone()
        bias[plus], bias[minus] = float("inf"), -float("inf")
        for best in (1, 2):
            r = gpu_lib.moe_group_route(L.cuda(), bias.cuda(), 6, 8, 3, best=best)
            ok(gpu_lib)
            want = O.route(L.double().numpy(), bias.double().numpy(), 6, 8, 3, "sigmoid", best, True, 1.0)
            np.testing.assert_array_equal(r["topk_ids"].cpu().numpy(), want["ids"])
