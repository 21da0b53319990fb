"""Host checks of the 4-bit entry points (no GPU): sizes as documented, and refusals before any CUDA call."""
import ctypes

import numpy as np
import pytest

from oracle import fp4_oracle as Q


@pytest.fixture(scope="module")
def lib():
    from top_routing_dispatch_moe_gb300 import build
    build.build()
    from top_routing_dispatch_moe_gb300 import moe
    return moe


def test_sizes(lib):
    assert [lib.moe_fp4_codes_pitch(k) for k in (0, 1, 32, 33, 999)] == [0, 16, 16, 32, 512]
    assert [lib.moe_fp4_scales_pitch(k, "nv") for k in (0, 1, 16, 17, 999)] == [0, 1, 1, 2, 63]
    assert [lib.moe_fp4_scales_pitch(k, "mx") for k in (0, 1, 32, 33, 999)] == [0, 1, 1, 2, 32]
    raw = lib.raw_lib()
    # 64-row blocks in pairs, 256 columns a stage: 8 KB of codes and, for 128 rows, 2 KB (nv) or 1 KB (mx) of scales
    assert raw.moe_fp4_packed_weight_bytes(3, 130, 300, 0) == 3 * 2 * (4 * 8192 + 2 * 2048)
    assert raw.moe_fp4_packed_weight_bytes(1, 1, 1, 1) == 2 * 8192 + 1024
    gu, down = 2 * 1 * (4 * 8192 + 2 * 1024), 2 * 1 * (2 * 8192 + 1024)
    assert raw.moe_fp4_packed_expert_weights_bytes(2, 96, 65, 1) == gu + down
    assert lib.moe_fp4_linear_workspace_size(4, 64, 0, "nv") > 0
    assert lib.moe_fp4_expert_ffn_workspace_size(4, 64, 64, 10, "mx") > lib.moe_fp4_linear_workspace_size(4, 64, 10, "mx")
    for bad in ((0, 64, 10), (1025, 64, 10), (4, 0, 10), (4, (1 << 20) + 1, 10), (4, 64, -1), (4, 64, (1 << 28) + 1)):
        assert lib.moe_fp4_linear_workspace_size(*bad, "nv") == 0
    with pytest.raises(lib.MoEError):
        lib.moe_fp4_scales_pitch(64, "int4")


def test_refusals_before_any_cuda_call(lib):
    raw = lib.raw_lib()
    P, n = ctypes.c_void_p, None
    ok, odd, bad = P(0x1000), P(0x1002), P(0x1003)
    INV, UNS, WS, OK = lib.MOE_ERR_INVALID_ARG, lib.MOE_ERR_UNSUPPORTED, lib.MOE_ERR_WORKSPACE, lib.MOE_OK

    def call(fn, args, change, want):
        a = list(args)
        for i, v in change.items():
            a[i] = v
        assert fn(*a) == want, (fn, change, lib.moe_last_error_string())

    # x, ldx, x_rows, src, rows, K, dtype, fmt, gscale, codes, scales, stream
    q, args = raw.moe_fp4_quantize, [ok, 64, 4, n, 4, 64, lib.MOE_BF16, 0, n, ok, ok, n]
    for change, want in (({6: 3}, UNS), ({7: 2}, UNS), ({4: -1}, INV), ({5: 0}, INV), ({5: (1 << 20) + 1, 1: 1 << 21}, INV),
                         ({1: 63}, INV), ({2: 3}, INV), ({0: n}, INV), ({9: n}, INV), ({10: n}, INV), ({9: odd}, INV),
                         ({0: bad}, INV), ({4: 0, 9: n, 10: n}, OK)):
        call(q, args, change, want)
    # codes, scales, rows, K, fmt, gscale, dtype, out, ldo, stream
    d, args = raw.moe_fp4_dequantize, [ok, ok, 4, 64, 1, n, lib.MOE_F16, ok, 64, n]
    for change, want in (({6: 5}, UNS), ({4: -1}, UNS), ({2: -1}, INV), ({3: 0}, INV), ({8: 63}, INV), ({0: n}, INV),
                         ({1: n}, INV), ({7: n}, INV), ({0: odd}, INV), ({7: bad}, INV), ({2: 0, 0: n, 7: n}, OK)):
        call(d, args, change, want)
    # codes, scales, G, N, K, fmt, packed, stream
    p, args = raw.moe_fp4_pack_weight, [ok, ok, 2, 64, 64, 0, ok, n]
    for change, want in (({5: 7}, UNS), ({2: 0}, INV), ({2: 1025}, INV), ({3: 0}, INV), ({4: 0}, INV), ({0: n}, INV),
                         ({1: n}, INV), ({6: n}, INV), ({0: odd}, INV), ({6: odd}, INV)):
        call(p, args, change, want)
    p, args = raw.moe_fp4_pack_expert_weights, [ok] * 6 + [2, 64, 64, 0, ok, n]
    for change, want in (({9: 7}, UNS), ({6: 0}, INV), ({7: 0}, INV), ({8: 0}, INV), ({0: n}, INV), ({5: n}, INV), ({4: odd}, INV)):
        call(p, args, change, want)
    # x, ldx, x_rows, src, offsets, tile_sched, packed, alpha, gscale, G, N, K, rows, fmt, dtype, out, ldo, out_dtype, ws, ws_bytes, stream
    big = 1 << 30
    lin, args = raw.moe_fp4_linear, [ok, 64, 4, n, ok, n, ok, n, n, 2, 32, 64, 4, 0, 1, ok, 32, 1, ok, big, n]
    for change, want in (({13: 2}, UNS), ({14: 3}, UNS), ({17: 3}, UNS), ({9: 0}, INV), ({9: 1025}, INV), ({10: 0}, INV),
                         ({11: 0}, INV), ({12: -1}, INV), ({1: 63}, INV), ({16: 31}, INV), ({2: 3}, INV), ({4: n}, INV),
                         ({5: ok}, INV), ({0: n}, INV), ({6: n}, INV), ({15: n}, INV), ({18: n}, INV), ({6: odd}, INV),
                         ({18: P(0x1010)}, INV), ({0: bad}, INV), ({15: bad}, INV), ({4: n, 5: odd}, INV), ({19: 64}, WS),
                         ({12: 0, 0: n, 6: n, 15: n, 18: n}, OK)):
        call(lin, args, change, want)
    # x, ldx, x_rows, src, offsets, tile_sched, packed, 3 alphas, gscale, act_gscale, E, h, F, rows, fmt, dtype, out, ldo, out_dtype, ws, ...
    ffn = raw.moe_fp4_expert_ffn
    args = [ok, 64, 4, n, ok, n, ok, n, n, n, n, n, 2, 64, 32, 4, 0, 1, ok, 64, 1, ok, big, n]
    for change, want in (({16: 2}, UNS), ({17: 3}, UNS), ({20: 3}, UNS), ({12: 0}, INV), ({13: 0}, INV), ({14: 0}, INV),
                         ({14: (1 << 20) + 1}, INV), ({15: -1}, INV), ({1: 63}, INV), ({19: 63}, INV), ({4: n}, INV),
                         ({5: ok}, INV), ({0: n}, INV), ({6: n}, INV), ({18: n}, INV), ({21: n}, INV), ({22: 64}, WS),
                         ({15: 0, 0: n, 6: n, 18: n, 21: n}, OK)):
        call(ffn, args, change, want)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_the_oracle_on_known_blocks(fmt):
    """Values that the formats hold exactly come back; the largest value of a block picks its scale; ties go to even."""
    b = Q.BLOCK[fmt]
    grid = np.concatenate([Q.E2M1, -Q.E2M1])
    x = np.resize(grid, (3, 2 * b)) * np.array([[1.0], [0.25], [64.0]])
    code, byte = Q.quantize(x, fmt)
    np.testing.assert_array_equal(Q.dequantize(code, byte, fmt), x)
    np.testing.assert_array_equal(Q.scale_of(byte, fmt), np.repeat([[1.0], [0.25], [64.0]], 2, 1))
    t = np.zeros((1, b))
    t[0, :8] = 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0
    code, byte = Q.quantize(t, fmt)
    np.testing.assert_array_equal(Q.dequantize(code, byte, fmt)[0, :8], [0, 1, 1, 2, 2, 4, 4, 6])
    x = np.random.default_rng(1).normal(size=(64, 5 * b + 3))
    v = Q.dequantize(*Q.quantize(x, fmt), fmt)
    amax = np.abs(np.pad(x, ((0, 0), (0, b - 3))).reshape(64, -1, b)).max(-1)
    # half the widest step (2 of 6) of the largest value, and what saturates or a scale's own rounding adds
    assert (np.abs(v - x) <= np.repeat(amax, b, 1)[:, : x.shape[1]] * (0.25 if fmt == "mx" else 0.18)).all()
