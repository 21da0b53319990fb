"""Host checks of the 8-bit entry points (no GPU): sizes as documented, and refusals before any CUDA call."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import int8_oracle as Q


@pytest.fixture(scope="module")
def lib():
    from top_routing_dispatch_moe_gb300 import build
    build.build()
    from top_routing_dispatch_moe_gb300 import moe
    return moe


def test_sizes(lib):
    raw = lib.raw_lib()
    assert raw.moe_int8_packed_weight_bytes(3, 130, 65) == 3 * 2 * 2 * 8192
    assert raw.moe_int8_packed_weight_bytes(1, 1, 1) == 8192
    assert raw.moe_int8_packed_expert_weights_bytes(2, 64, 65) == 2 * (2 * 1 + 1 * 2) * 8192
    assert lib.moe_int8_expert_ffn_workspace_size(4, 64, 64, 10) > lib.moe_int8_linear_workspace_size(4, 64, 64, 10) > 0
    for bad in ((0, 64, 64, 10), (1025, 64, 64, 10), (4, 0, 64, 10), (4, 64, 0, 10), (4, 64, (1 << 17) + 1, 10), (4, 64, 64, -1),
                (4, 64, 64, (1 << 28) + 1)):
        assert lib.moe_int8_linear_workspace_size(*bad) == 0
    assert lib.moe_int8_expert_ffn_workspace_size(4, 64, (1 << 16) + 1, 10) == 0


def test_refusals_before_any_cuda_call(lib):
    raw = lib.raw_lib()
    P, n = ctypes.c_void_p, None
    ok, odd, bad = P(0x1000), P(0x1008), P(0x1003)
    INV, UNS, WS, OK = lib.MOE_ERR_INVALID_ARG, lib.MOE_ERR_UNSUPPORTED, lib.MOE_ERR_WORKSPACE, lib.MOE_OK

    def call(fn, args, change, want):
        a = list(args)
        for i, v in change.items():
            a[i] = v
        assert fn(*a) == want, (fn, change, lib.moe_last_error_string())

    most = (1 << 17) + 1
    # x, ldx, x_rows, src, rows, K, dtype, codes, scales, stream
    args = [ok, 64, 4, n, 4, 64, lib.MOE_BF16, ok, ok, n]
    for change, want in (({6: 3}, UNS), ({4: -1}, INV), ({5: 0}, INV), ({5: most, 1: most}, INV), ({1: 63}, INV), ({2: 3}, INV), ({0: n}, INV),
                         ({7: n}, INV), ({8: n}, INV), ({0: bad}, INV), ({8: bad}, INV), ({4: 0, 7: n, 8: n}, OK)):
        call(raw.moe_int8_quantize, args, change, want)
    # codes, scales, rows, K, dtype, out, ldo, stream
    args = [ok, ok, 4, 64, lib.MOE_F16, ok, 64, n]
    for change, want in (({4: 5}, UNS), ({2: -1}, INV), ({3: 0}, INV), ({6: 63}, INV), ({0: n}, INV), ({1: n}, INV), ({5: n}, INV), ({5: bad}, INV),
                         ({2: 0, 0: n, 5: n}, OK)):
        call(raw.moe_int8_dequantize, args, change, want)
    # codes, G, N, K, packed, stream
    args = [ok, 2, 64, 64, ok, n]
    for change, want in (({1: 0}, INV), ({1: 1025}, INV), ({2: 0}, INV), ({3: most}, INV), ({0: n}, INV), ({4: n}, INV), ({4: odd}, INV)):
        call(raw.moe_int8_pack_weight, args, change, want)
    # gate, up, down, E, h, F, packed, stream
    args = [ok, ok, ok, 2, 64, 64, ok, n]
    for change, want in (({3: 0}, INV), ({4: most}, INV), ({5: (1 << 16) + 1}, INV), ({1: n}, INV), ({6: n}, INV), ({6: odd}, INV)):
        call(raw.moe_int8_pack_expert_weights, args, change, want)
    big = 1 << 30
    # x, ldx, x_rows, src, offsets, sched, packed, w_scales, G, N, K, rows, dtype, out, ldo, out_dtype, ws, bytes, stream
    args = [ok, 64, 4, n, ok, n, ok, ok, 2, 48, 64, 4, lib.MOE_BF16, ok, 48, lib.MOE_F32, ok, big, n]
    for change, want in (({12: 3}, UNS), ({15: -1}, UNS), ({8: 0}, INV), ({9: 0}, INV), ({10: 0}, INV), ({11: -1}, INV), ({1: 63}, INV), ({14: 47}, INV),
                         ({2: 3}, INV), ({4: n}, INV), ({5: ok}, INV), ({0: n}, INV), ({6: n}, INV), ({7: n}, INV), ({13: n}, INV), ({0: bad}, INV),
                         ({6: odd}, INV), ({13: bad}, INV), ({16: n}, WS), ({16: odd}, WS), ({17: 16}, WS), ({11: 0, 0: n, 13: n, 16: n}, OK)):
        call(raw.moe_int8_linear, args, change, want)
    # x, ldx, x_rows, src, offsets, sched, packed, gate, up, down scales, E, h, F, rows, dtype, out, ldo, out_dtype, ws, bytes, stream
    args = [ok, 64, 4, n, ok, n, ok, ok, ok, ok, 2, 64, 48, 4, lib.MOE_BF16, ok, 64, lib.MOE_BF16, ok, big, n]
    for change, want in (({14: 3}, UNS), ({10: 1025}, INV), ({11: 0}, INV), ({12: (1 << 16) + 1}, INV), ({1: 63}, INV), ({16: 63}, INV), ({5: ok}, INV),
                         ({7: n}, INV), ({8: n}, INV), ({9: n}, INV), ({9: bad}, INV), ({15: n}, INV), ({18: n}, WS), ({19: 2048}, WS)):
        call(raw.moe_int8_expert_ffn, args, change, want)


def test_the_binding_refuses_host_tensors_and_shapes(lib):
    x = torch.zeros(4, 64)
    with pytest.raises(lib.MoEError):
        lib.moe_int8_quantize(x)
    with pytest.raises(lib.MoEError):
        lib.moe_int8_pack_weight(torch.zeros(4, 64, dtype=torch.int8))
    with pytest.raises(lib.MoEError):
        lib.moe_int8_pack_expert_weights(*(torch.zeros(2, 8, 4, dtype=torch.int8),) * 3)


def test_the_oracle_rounds_ties_to_even():
    c, s = Q.quantize(np.array([[254.0, 1.0, 3.0, 5.0, -1.0, -3.0], [0.0] * 6, [1.0, np.inf, 0, 0, 0, 0]]))
    assert c.tolist() == [[127, 0, 2, 2, 0, -2], [0] * 6, [0] * 6]
    assert s[0] == 2.0 and s[1] == 0.0 and np.isnan(s[2])
