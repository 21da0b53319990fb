"""Host check (no GPU): the numbers of a Python call reach C as they are or are refused."""
import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from top_routing_dispatch_moe_gb300 import build
    build.build()
    from top_routing_dispatch_moe_gb300 import moe
    return moe


@pytest.mark.parametrize("n", [(1 << 32) + 2, -(1 << 32) + 2])
def test_every_number_of_a_call_is_looked_at(lib, n):
    """(2^32 + 2 groups would be two.)"""
    L, x, w, ids, gates, f = torch.zeros(0, 64), torch.zeros(0, 64), torch.zeros(0), torch.zeros(0, 4, dtype=torch.int32), torch.zeros(0, 4), torch.zeros(64)
    codes, scales, d_act = torch.zeros(0, 256, dtype=torch.int8), torch.zeros(0, 2), torch.zeros(0, 8)
    calls = [lambda **a: lib.moe_group_route(L, None, **{**dict(k=4, groups=4, top_groups=2), **a}),
             lambda **a: lib.moe_group_router(x, w, **{**dict(E=64, bias=None, k=4, groups=4, top_groups=2), **a})]
    for call in calls:
        for name in ("k", "groups", "top_groups", "best", "score"):
            with pytest.raises(lib.MoEError, match=f"a size of {n}") as e:
                call(**{name: n})
            assert e.value.code == lib.MOE_ERR_INVALID_ARG, name
    for call in (lambda: calls[1](E=n), lambda: lib.moe_group_route_backward(L, ids, gates, f, score=n), lambda: lib.moe_checkpoint8_save(d_act, E=n),
                 lambda: lib.moe_checkpoint8_swiglu_backward(codes, scales, d_act, E=n),
                 lambda: lib.moe_expert_up_gate_backward_checkpoint8(codes, scales, d_act, None, w, n, 8),
                 lambda: lib.moe_expert_up_gate_backward_checkpoint8(codes, scales, d_act, None, w, 8, n)):
        with pytest.raises(lib.MoEError, match=f"a size of {n}"):
            call()
