"""Host checks of routing by groups (no GPU): refusals before any CUDA call, and the oracle's gradient against differences."""
import ctypes

import numpy as np
import pytest

from oracle import group_route_oracle as O


@pytest.fixture(scope="module")
def lib():
    from top_routing_dispatch_moe_gb300 import build
    build.build()
    from top_routing_dispatch_moe_gb300 import moe
    return moe


def test_refusals_before_any_cuda_call(lib):
    raw = lib.raw_lib()
    P, n = ctypes.c_void_p, None
    ok, odd = P(0x1000), P(0x1004)
    INV, UNS, WS = lib.MOE_ERR_INVALID_ARG, lib.MOE_ERR_UNSUPPORTED, lib.MOE_ERR_WORKSPACE

    def call(fn, args, change, want):
        a = list(args)
        for i, v in change.items():
            a[i] = v
        assert fn(*a) == want, (fn, change, lib.moe_last_error_string())

    big = 1 << 30
    # logits, bias, T, E, k, groups, top_groups, score, best, renorm, scale, alpha, ids, gates, counts, f, P, aux, ws, bytes, stream
    args = [ok, n, 4, 64, 8, 8, 4, 0, 2, 1, 2.5, 0.01, ok, ok, ok, ok, ok, ok, ok, big, n]
    for change, want in (({7: 2}, UNS), ({7: -1}, UNS), ({2: -1}, INV), ({2: (1 << 30) + 1}, INV), ({3: 0}, INV), ({3: 1088, 5: 17}, INV), ({5: 7}, INV), ({5: 0}, INV),
                         ({3: 1024, 5: 64}, INV), ({6: 0}, INV), ({6: 9}, INV), ({8: 0}, INV), ({8: 3}, INV), ({5: 64}, INV),
                         ({4: 0}, INV), ({4: 17, 6: 8}, INV), ({4: 9, 6: 1}, INV), ({10: float("inf")}, INV), ({0: n}, INV),
                         ({12: n}, INV), ({17: n}, INV), ({18: n}, WS), ({18: odd}, WS), ({19: 16}, WS)):
        call(raw.moe_group_route, args, change, want)
    # x, w_packed, bias, T, h, E, k, dtype, groups, top_groups, score, best, renorm, scale, alpha, logits, ids, ... aux, ws, bytes, stream
    args = [ok, ok, n, 4, 64, 64, 8, lib.MOE_BF16, 8, 4, 1, 1, 0, 1.0, 0.01, n, ok, ok, ok, ok, ok, ok, ok, big, n]
    for change, want in (({7: 2}, UNS), ({10: 5}, UNS), ({4: 0}, INV), ({4: 60}, INV), ({8: 5}, INV), ({0: n}, INV), ({1: n}, INV),
                         ({0: odd}, INV), ({15: odd}, INV), ({16: n}, INV), ({22: n}, WS), ({23: 64}, WS)):
        call(raw.moe_group_router, args, change, want)
    # logits, ids, d_gates, f, T, E, k, score, renorm, scale, alpha, d_aux, d_logits, stream
    args = [ok, ok, ok, ok, 4, 64, 8, 0, 1, 1.0, 0.01, 1.0, ok, n]
    for change, want in (({7: 2}, UNS), ({4: -1}, INV), ({4: (1 << 30) + 1}, INV), ({5: 1025}, INV), ({6: 0}, INV), ({6: 17}, INV), ({9: float("nan")}, INV), ({0: n}, INV),
                         ({1: n}, INV), ({2: n}, INV), ({3: n}, INV), ({12: n}, INV), ({4: 0, 0: n, 12: n}, lib.MOE_OK)):
        call(raw.moe_group_route_backward, args, change, want)
    assert lib.moe_group_route_workspace_size(16384, 256) > 0
    assert lib.moe_group_route_workspace_size((1 << 30) + 1, 256) == 0
    assert lib.moe_group_route_workspace_size(-1, 256) == 0 and lib.moe_group_router_workspace_size(4, 0, 64, lib.MOE_BF16) == 0


def test_sizes_that_no_int_holds_are_refused(lib):
    """(ctypes takes a size modulo 2^32: 2^32 + 5 rows would be five.)"""
    lib._counts(1, (1 << 31) - 1)
    for n in (1 << 31, (1 << 32) + 5):
        with pytest.raises(lib.MoEError) as e:
            lib._counts(4, n)
        assert e.value.code == lib.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_the_oracles_gradient_is_that_of_differences(score, renorm):
    rng = np.random.default_rng(3)
    L = rng.normal(size=(3, 24)) * 1.5
    r = O.route(L, rng.normal(size=24) * 0.05, 4, 4, 2, score, 2, renorm, 2.5)
    dg = rng.normal(size=(3, 4))
    args = (r["ids"], dg, r["f"], score, renorm, 2.5)
    want = O.backward(L, *args, alpha=0.3, d_aux=0.7)
    eps = 1e-5
    for t, e in [(0, int(r["ids"][0, 0])), (1, int(r["ids"][1, 3])), (2, 5), (0, 23), (1, 0)]:
        hi, lo = L.copy(), L.copy()
        hi[t, e] += eps
        lo[t, e] -= eps
        got = (O.loss(hi, *args, alpha=0.3, d_aux=0.7) - O.loss(lo, *args, alpha=0.3, d_aux=0.7)) / (2 * eps)
        assert abs(got - want[t, e]) < 1e-8
