"""Activation checkpoints in 8 bits on the GPU: codes and scales exactly, the SwiGLU backward against its formula in 64 bits and against
differences, and the layer's backward from them."""
import numpy as np
import pytest
import torch

from oracle import int8_oracle as Q

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BF16 = 2.0**-8                                            # half a step, relative


def f64(t):
    return t.double().cpu().numpy()


def ok(moe):
    torch.cuda.synchronize()
    assert moe.moe_check_device_error() == moe.MOE_OK, moe.moe_last_error_string()


def blocks(x):
    """codes [rows, C] and scales [rows, blocks] of x [rows, C] in float64."""
    rows, C = x.shape
    pad = np.pad(x, ((0, 0), (0, -C % 128))).reshape(rows, -1, 128)
    c, s = Q.quantize(pad)
    return c.reshape(rows, -1)[:, :C], s


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,C", [(1, 1), (1, 128), (3, 127), (5, 129), (4, 256), (17, 999), (33, 1000), (9, 2048), (130, 640), (2, 20000)])
def test_save_and_load(gpu_lib, dtype, rows, C):
    x = (torch.randn(rows, C, generator=torch.Generator().manual_seed(rows + C)) * 3).to(DT[dtype]).cuda()
    c, s = gpu_lib.moe_checkpoint8_save(x)
    ok(gpu_lib)
    code, scale = blocks(f64(x))
    np.testing.assert_array_equal(c.cpu().numpy(), code)
    np.testing.assert_array_equal(f64(s), scale)
    for out in ("fp32", dtype):
        y = gpu_lib.moe_checkpoint8_load(c, s, dtype=DT[out])
        assert torch.equal(y, (c.float() * s.repeat_interleave(128, 1)[:, :C]).to(DT[out]))
    # strides on both sides
    wide = torch.zeros(rows, C + 5, dtype=DT[dtype], device="cuda")
    wide[:, 3:3 + C] = x
    c2, s2 = gpu_lib.moe_checkpoint8_save(wide[:, 3:3 + C])
    assert torch.equal(c2, c) and torch.equal(s2, s)
    gpu_lib.moe_checkpoint8_load(c, s, out=wide[:, 1:1 + C])
    assert torch.equal(wide[:, 1:1 + C], y) and (wide[:, 0] == 0).all() and (wide[:, C + 3:] == 0).all()
    ok(gpu_lib)


def test_bad_and_empty_blocks(gpu_lib):
    x = torch.randn(4, 384, generator=torch.Generator().manual_seed(1))
    x[0, :128] = 0.0
    x[1, 130] = float("nan")
    x[2, 383] = -float("inf")
    x[3, 128:256] *= 2.0**-100
    for C in (384, 383):
        v = x[:, :C].contiguous()
        c, s = gpu_lib.moe_checkpoint8_save(v.cuda())
        ok(gpu_lib)
        code, scale = blocks(v.double().numpy())
        np.testing.assert_array_equal(c.cpu().numpy(), code)
        np.testing.assert_array_equal(f64(s), scale)
    assert gpu_lib.moe_checkpoint8_save(torch.empty(0, 64).cuda())[0].shape == (0, 64)


def swiglu_backward(g, u, da):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-g))
    return da * u * s * (1.0 + g * (1.0 - s)), da * g * s, g * s * u


def split(moe, gu, F):
    """g and u [rows, F] of a [rows, gu_cols(F)] array."""
    v = gu.reshape(gu.shape[0], -1, 2, 128)
    return v[:, :, 0].reshape(gu.shape[0], -1)[:, :F], v[:, :, 1].reshape(gu.shape[0], -1)[:, :F]


@pytest.mark.parametrize("rows,F,scale", [(1, 8, 1.0), (3, 120, 1.0), (5, 128, 30.0), (17, 136, 1.0), (33, 1000, 3.0), (130, 384, 1.0), (2, 14336, 1.0)])
def test_swiglu_backward(gpu_lib, rows, F, scale):
    gen = torch.Generator().manual_seed(rows * F)
    cols = gpu_lib.gu_cols(F)
    gu = torch.zeros(rows, cols // 256, 2, 128)
    gu.view(rows, -1, 256)
    full = torch.randn(rows, cols // 256, 2, 128, generator=gen) * scale
    for i in range(cols // 256):
        n = min(128, F - 128 * i)
        gu[:, i, :, :n] = full[:, i, :, :n]
    gu = gu.view(rows, cols).bfloat16().cuda()
    da = torch.randn(rows, F, generator=gen).bfloat16().cuda()
    c, s = gpu_lib.moe_checkpoint8_save(gu)
    d_gu, act = gpu_lib.moe_checkpoint8_swiglu_backward(c, s, da)
    ok(gpu_lib)
    v = (c.float() * s.repeat_interleave(128, 1)).double().cpu().numpy()
    g, u = split(gpu_lib, v, F)
    want = swiglu_backward(g, u, f64(da))
    got = (*split(gpu_lib, f64(d_gu), F), f64(act))
    # bf16's rounding; the quick exponential and quotient, off by 2^-20 and one half step for each unit of |g|, act on s and 1 - s: d_g
    # is a sum of da u s and da u s g (1 - s)
    span = 16 + np.abs(g)
    s_ = 1.0 / (1.0 + np.exp(-np.clip(g, -700, 700)))
    mags = (np.abs(f64(da) * u * s_) * (1 + np.abs(g)), np.abs(want[1]), np.abs(want[2]))
    for w, y, m in zip(want, got, mags):
        assert (np.abs(y - w) <= BF16 * np.abs(w) * 1.001 + span * 2.0**-24 * 4 * m + 1e-36).all()
    pad = f64(d_gu).reshape(rows, -1, 2, 128)
    if F % 128:
        assert (pad[:, -1, :, F % 128:] == 0).all()


def test_gradient_is_that_of_differences():
    rng = np.random.default_rng(0)
    g, u, da = rng.normal(size=(3, 40)) * 3
    d_g, d_u, _ = swiglu_backward(g, u, da)
    e = 1e-6
    act = lambda g, u: swiglu_backward(g, u, 0 * g)[2]
    np.testing.assert_allclose((act(g + e, u) - act(g - e, u)) / (2 * e) * da, d_g, atol=1e-8)
    np.testing.assert_allclose((act(g, u + e) - act(g, u - e)) / (2 * e) * da, d_u, atol=1e-8)


def test_infinite_gates_stay_in_their_block(gpu_lib):
    gu = torch.zeros(2, 256)
    gu[0, :128] = -300.0
    gu[0, 128:] = 2.0
    gu[1, 5] = float("inf")
    da = torch.ones(2, 128).bfloat16().cuda()
    c, s = gpu_lib.moe_checkpoint8_save(gu.bfloat16().cuda())
    d_gu, act = gpu_lib.moe_checkpoint8_swiglu_backward(c, s, da)
    ok(gpu_lib)
    assert (d_gu[0] == 0).all() and (act[0] == 0).all() and act[1].isnan().all()


@pytest.mark.parametrize("capacity", [0, 40])
def test_only_the_schedules_rows(gpu_lib, capacity):
    T, E, k, h, F = 300, 6, 2, 64, 72
    x = torch.randn(T, h, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i))[:k] for i in range(T)]).int().cuda()
    d = gpu_lib.moe_dispatch(x, ids, E, capacity)
    rows, cols = d["rows"], gpu_lib.gu_cols(F)
    gu = torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    da = torch.randn(rows, F, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    c, s = gpu_lib.moe_checkpoint8_save(gu)
    c2, s2 = torch.full_like(c, 99), torch.full_like(s, 99.0)
    gpu_lib.moe_checkpoint8_save(gu, tile_sched=d["tile_sched"], E=E, codes=c2, scales=s2)
    d_gu, act = gpu_lib.moe_checkpoint8_swiglu_backward(c, s, da)
    d2, a2 = torch.full_like(d_gu, 7.0), torch.full_like(act, 7.0)
    gpu_lib.moe_checkpoint8_swiglu_backward(c, s, da, tile_sched=d["tile_sched"], E=E, d_gu=d2, act=a2)
    ok(gpu_lib)
    live = torch.zeros(rows, dtype=torch.bool)
    off, kept = d["offsets"].tolist(), d["kept_counts"].tolist()
    for e in range(E):
        live[off[e]:off[e] + kept[e]] = True
    live = live.cuda()
    assert torch.equal(c2[live], c[live]) and (c2[~live] == 99).all() and torch.equal(s2[live], s[live]) and (s2[~live] == 99).all()
    assert torch.equal(d2[live], d_gu[live]) and (d2[~live] == 7).all() and torch.equal(a2[live], act[live]) and (a2[~live] == 7).all()
    for call in (lambda: gpu_lib.moe_checkpoint8_save(gu, tile_sched=d["tile_sched"], E=E + 1, codes=c2, scales=s2),
                 lambda: gpu_lib.moe_checkpoint8_swiglu_backward(c, s, da, tile_sched=d["tile_sched"], E=E - 1, d_gu=d2, act=a2)):
        call()
        torch.cuda.synchronize()
        assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_ERR_INVALID_ARG


def test_the_experts_backward_from_a_checkpoint(gpu_lib):
    T, E, k, h, F = 200, 4, 2, 128, 200
    gen = torch.Generator().manual_seed(3)
    mk = lambda *s: (torch.randn(*s, generator=gen) / s[-1] ** 0.5).bfloat16().cuda()
    x = torch.randn(T, h, generator=gen).bfloat16().cuda()
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(T)]).int().cuda()
    wg, wu, wd = mk(E, F, h), mk(E, F, h), mk(E, h, F)
    packed, packed_bwd = gpu_lib.moe_pack_expert_weights(wg, wu, wd), gpu_lib.moe_pack_expert_weights_backward(wg, wu, wd)
    d = gpu_lib.moe_dispatch(x, ids, E)
    sched = d["tile_sched"]
    _, gu, _, _ = gpu_lib.moe_expert_up_gate_save(d["buf"], sched, packed, E, F)
    codes, scales = gpu_lib.moe_checkpoint8_save(gu, tile_sched=sched, E=E)
    da = torch.randn(d["rows"], F, generator=gen).bfloat16().cuda()
    d_gu, act, d_buf = gpu_lib.moe_expert_up_gate_backward_checkpoint8(codes, scales, da, sched, packed_bwd, E, h)
    kept = gpu_lib.moe_checkpoint8_load(codes, scales)
    d_gu2, d_buf2 = gpu_lib.moe_expert_up_gate_backward_saved(gu, da, sched, packed_bwd, E, h)
    ok(gpu_lib)
    alone = gpu_lib.moe_checkpoint8_swiglu_backward(codes, scales, da)
    assert torch.equal(alone[0], d_gu) and torch.equal(alone[1], act)
    # the checkpoint is within half a step, amax / 254 of its block, of what it keeps (and bf16's rounding of the loaded value)
    v = f64(gu).reshape(d["rows"], -1, 128)
    assert (np.abs(f64(kept).reshape(v.shape) - v) <= np.abs(v).max(2, keepdims=True) / 254 * 1.001 + BF16 * np.abs(v)).all()
    # d_buf is the product of the d_gu it came with
    off = d["offsets"].tolist()
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        g, u = split(gpu_lib, f64(d_gu)[lo:hi], F)
        want = g @ f64(wg)[e] + u @ f64(wu)[e]
        mag = np.abs(g) @ np.abs(f64(wg)[e]) + np.abs(u) @ np.abs(f64(wu)[e])
        assert (np.abs(f64(d_buf)[lo:hi] - want) <= BF16 * np.abs(want) * 1.001 + 2 * F * 2.0**-24 * mag).all()


def test_captured(gpu_lib):
    gu = torch.randn(300, 512, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    da = torch.randn(300, 256, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    want = gpu_lib.moe_checkpoint8_swiglu_backward(*gpu_lib.moe_checkpoint8_save(gu), da)
    c, s = torch.empty(300, 512, dtype=torch.int8, device="cuda"), torch.empty(300, 4, device="cuda")
    d_gu, act = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        gpu_lib.moe_checkpoint8_save(gu, codes=c, scales=s)
        gpu_lib.moe_checkpoint8_swiglu_backward(c, s, da, d_gu=d_gu, act=act)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(d_gu, want[0]) and torch.equal(act, want[1])
    ok(gpu_lib)


def test_past_32_bit_offsets(gpu_lib):
    rows, F = 76000, 14336                                # 76000 x 28672 values
    gu = torch.zeros(rows, 2 * F, dtype=torch.bfloat16, device="cuda")
    gu[-3:] = torch.randn(3, 2 * F, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    da = torch.ones(rows, F, dtype=torch.bfloat16, device="cuda")
    c, s = gpu_lib.moe_checkpoint8_save(gu)
    d_gu, act = gpu_lib.moe_checkpoint8_swiglu_backward(c, s, da)
    ok(gpu_lib)
    c3, s3 = gpu_lib.moe_checkpoint8_save(gu[-3:])
    d3, a3 = gpu_lib.moe_checkpoint8_swiglu_backward(c3, s3, da[-3:])
    assert torch.equal(c[-3:], c3) and torch.equal(s[-3:], s3) and torch.equal(d_gu[-3:], d3) and torch.equal(act[-3:], a3)
    assert (c[:-3] == 0).all() and (act[40000] == 0).all()
    assert torch.equal(gpu_lib.moe_checkpoint8_load(c, s)[-3:], gpu_lib.moe_checkpoint8_load(c3, s3))
    del gu, da, c, s, d_gu, act
    torch.cuda.empty_cache()
