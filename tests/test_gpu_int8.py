"""The 8-bit expert operators on the GPU against the float64 oracle: codes exactly, products within the roundings that follow the
exact sums, the FFN within the steps that activations next to a border may take the other way."""
import numpy as np
import pytest
import torch

from oracle import int8_oracle as Q

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}
F32 = HALF_STEP["fp32"]


def data(shape, dtype="bf16", seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).cuda()


def f64(t):
    return t.double().cpu().numpy()


def ok(moe):
    torch.cuda.synchronize()
    assert moe.moe_check_device_error() == moe.MOE_OK, moe.moe_last_error_string()


def weight(G, N, K, seed=1):
    """Codes [G, N, K] with -128 among them, and scales [G, N]."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(-128, 128, (G, N, K), generator=g, dtype=torch.int16).to(torch.int8)
    return c.cuda(), (torch.rand(G, N, generator=g) * 2e-3 + 1e-4).cuda()


def offsets_of(rows, G, seed=0, kind="random"):
    g = np.random.default_rng(seed)
    if kind == "one":                                    # all rows in one group
        n = np.zeros(G, np.int64)
        n[g.integers(G)] = rows
    else:
        n = g.multinomial(rows, g.dirichlet(np.full(G, 0.5)))
    return np.concatenate([[0], np.cumsum(n)])


def dev(offsets):
    return torch.from_numpy(np.asarray(offsets, np.int32)).cuda()


def near(got, want, dtype, extra=0.0):
    """got (of dtype) is want after the three fp32 roundings of (sum * scale) * scale and the type's own; `extra`: absolute."""
    got = f64(got)
    tol = (3 * F32 + HALF_STEP[dtype]) * np.abs(want) * (1 + 1e-6) + extra + (2.0**-25 if dtype == "fp16" else 0.0)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    bad = np.abs(got - want) > tol
    assert not bad[~np.isnan(want)].any(), (int(bad.sum()), float(np.nanmax(np.abs(got - want) / (np.abs(want) + 1e-30))))


# ------------------------------------------------------------------------------------------ rows there and back


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 7168), (3, 15), (5, 16), (7, 31), (129, 64), (33, 100), (17, 999), (9, 2048), (4, 2064),
                                    (5, 4096), (3, 8208), (2, 16384), (2, 16400), (3, 20001), (70, 768)])
def test_quantize_is_the_definition(gpu_lib, dtype, rows, K):
    x = data((rows, K), dtype, rows * 7919 + K, 3.0)
    c, s = gpu_lib.moe_int8_quantize(x)
    ok(gpu_lib)
    code, scale = Q.quantize(f64(x))
    np.testing.assert_array_equal(c.cpu().numpy(), code)
    np.testing.assert_array_equal(f64(s), scale)
    for out in ("fp32", dtype):
        y = gpu_lib.moe_int8_dequantize(c, s, dtype=DT[out])
        want = (c.float() * s.unsqueeze(1)).to(DT[out])      # one fp32 product, one rounding
        assert torch.equal(y, want)
    ok(gpu_lib)


@pytest.mark.parametrize("K", [64, 999])
def test_values_on_and_next_to_a_border(gpu_lib, K):
    # amax = 254 * 2^e: every odd multiple of half a step is a tie; and fp32 neighbours of ties
    base = np.arange(K) % 127 + 0.5
    x = np.stack([base * 2.0, np.nextafter(np.float32(base * 2), np.float32(1e9)), np.nextafter(np.float32(base * 2), np.float32(-1e9)), -base * 2.0,
                  base * 3.0, np.nextafter(np.float32(base * 3), np.float32(1e9))]).astype(np.float32)
    x[:4, 0] = 254.0
    x[4:, 0] = 381.0
    x *= np.float32(2.0) ** np.array([0, 3, -20, 60, -60, 100], np.float32)[:, None]
    t = torch.from_numpy(x).cuda()
    c, s = gpu_lib.moe_int8_quantize(t)
    ok(gpu_lib)
    code, scale = Q.quantize(x)
    np.testing.assert_array_equal(c.cpu().numpy(), code)
    np.testing.assert_array_equal(f64(s), scale)


def test_zero_tiny_infinite_and_nan_rows(gpu_lib):
    x = torch.randn(8, 96, generator=torch.Generator().manual_seed(0))
    x[0] = 0.0
    x[1] *= 2.0**-110
    x[2, 5] = float("inf")
    x[3, 95] = float("nan")
    x[4] = torch.nan_to_num(x[4]) * 1e38
    x[5] = 0.0
    x[5, 17] = 2.0**-96
    for K in (96, 95):
        v = x[:, :K].contiguous()
        if K == 95:
            v[3, 94] = float("nan")
        c, s = gpu_lib.moe_int8_quantize(v.cuda())
        ok(gpu_lib)
        code, scale = Q.quantize(v.double().numpy())
        np.testing.assert_array_equal(c.cpu().numpy(), code)
        np.testing.assert_array_equal(f64(s), scale)
        y = gpu_lib.moe_int8_dequantize(c, s, dtype=torch.float32)
        # (the fourth row's 4.1e38 is an infinity in fp32)
        finite = torch.isfinite(v).all(1)
        assert finite.tolist() == [True, True, False, False, False, True, True, True]
        assert y[~finite].isnan().all() and (y[:2] == 0).all() and torch.isfinite(y[finite]).all()


def test_strides_gathered_rows_and_bounds(gpu_lib):
    big = data((20, 300), "bf16", 3)
    for x in (big[:, 8:136], big[:, 1:130], big[::2, :64], big.t().contiguous().t()[:, :1]):
        c, s = gpu_lib.moe_int8_quantize(x)
        ok(gpu_lib)
        code, scale = Q.quantize(f64(x))
        np.testing.assert_array_equal(c.cpu().numpy(), code)
        out = torch.full((x.shape[0], 200), 7.0, dtype=torch.bfloat16, device="cuda")
        for at in (0, 1):
            view = out[:, at:at + x.shape[1]]
            gpu_lib.moe_int8_dequantize(c, s, out=view)
            assert torch.equal(view, (c.float() * s.unsqueeze(1)).bfloat16())
        assert (out[:, x.shape[1] + 1:] == 7.0).all()
    src = torch.tensor([3, -1, 0, 3, 19], dtype=torch.int32, device="cuda")
    c, s = gpu_lib.moe_int8_quantize(big, src=src)
    ok(gpu_lib)
    rows = f64(big)[[3, 0, 0, 3, 19]]
    rows[1] = 0.0
    code, scale = Q.quantize(rows)
    np.testing.assert_array_equal(c.cpu().numpy(), code)
    src[2] = 20
    c, _ = gpu_lib.moe_int8_quantize(big, src=src)
    torch.cuda.synchronize()
    assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_ERR_INVALID_ARG
    assert (c[2] == 0).all()
    assert gpu_lib.moe_int8_quantize(big[:0])[0].shape == (0, 300)


# ------------------------------------------------------------------------------------------ products


LINEAR = [  # G, rows, N, K, kind
    (1, 1, 1, 1, "random"), (1, 1, 128, 64, "random"), (3, 2, 33, 70, "random"), (1, 9, 130, 128, "random"), (5, 40, 256, 200, "random"),
    (7, 300, 257, 136, "random"), (2, 33, 96, 1000, "one"), (16, 64, 384, 512, "random"), (3, 700, 512, 320, "random"), (1, 257, 640, 64, "one"),
    (128, 200, 64, 64, "random"), (1024, 1500, 32, 64, "random"), (4, 1300, 300, 2048, "random"), (2, 600, 1001, 1044, "one"), (1, 31, 100, 16500, "one")]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("G,rows,N,K,kind", LINEAR)
def test_linear(gpu_lib, dtype, G, rows, N, K, kind):
    x = data((rows, K), dtype, G + rows)
    w, ws = weight(G, N, K)
    off = offsets_of(rows, G, rows, kind)
    packed = gpu_lib.moe_int8_pack_weight(w)
    y = gpu_lib.moe_int8_linear(x, dev(off), packed, ws)
    ok(gpu_lib)
    c, s = Q.quantize(f64(x))
    want = Q.linear(c, s, off, w.cpu().numpy(), f64(ws))
    # past 2^24 the sums of whole numbers round: K / 16 partial sums, each off by half a step of the largest
    most = np.abs(c).sum(1).max() * 128.0
    extra = 0.0 if most < 2**24 else (K / 16 + 1) * most * F32 * np.nanmax(s) * f64(ws).max()
    near(y, want, dtype, extra)


def test_linear_of_the_largest_codes(gpu_lib):
    # the largest sums: 127 * 128 * K, past 2^24 in every channel
    K, rows = 4096, 70
    x = torch.ones(rows, K).cuda()
    x[1::2] = -1.0
    w = torch.full((1, 160, K), -128, dtype=torch.int8, device="cuda")
    ws = torch.full((1, 160), 1.0, device="cuda")
    for n in (3, rows):
        y = gpu_lib.moe_int8_linear(x[:n], dev([0, n]), gpu_lib.moe_int8_pack_weight(w), ws)
        ok(gpu_lib)
        # every partial sum is a multiple of 128 * 127 * 16 below 2^24 of those: exact
        want = -128.0 * 127 * K * f64(torch.tensor([1.0 / 127.0]))
        np.testing.assert_allclose(f64(y), np.where(np.arange(n) % 2, -want, want)[:, None] * np.ones((1, 160)), rtol=4 * F32)


@pytest.mark.parametrize("rows", [5, 400])
def test_rows_of_no_group_strided_output_and_other_type(gpu_lib, rows):
    x = data((rows, 192), "bf16", 9)
    w, ws = weight(3, 70, 192)
    off = np.array([1, 2, 2, rows - 1])
    out = torch.full((rows, 90), 5.0, device="cuda")
    gpu_lib.moe_int8_linear(x, dev(off), gpu_lib.moe_int8_pack_weight(w), ws, out=out[:, 3:73])
    ok(gpu_lib)
    c, s = Q.quantize(f64(x))
    want = Q.linear(c, s, off, w.cpu().numpy(), f64(ws))
    near(out[1:rows - 1, 3:73], want[1:rows - 1], "fp32")
    assert (out[0] == 5).all() and (out[-1] == 5).all() and (out[:, :3] == 5).all() and (out[:, 73:] == 5).all()


@pytest.mark.parametrize("rows", [4, 300])
def test_a_bad_row_leaves_the_others(gpu_lib, rows):
    x = data((rows, 128), "fp32", 2)
    x[1, 7] = float("inf")
    x[2] = 0.0
    w, ws = weight(2, 64, 128)
    off = [0, rows // 2, rows]
    y = gpu_lib.moe_int8_linear(x, dev(off), gpu_lib.moe_int8_pack_weight(w), ws)
    ok(gpu_lib)
    c, s = Q.quantize(f64(x))
    near(y, Q.linear(c, s, off, w.cpu().numpy(), f64(ws)), "fp32")
    assert y[1].isnan().all() and (y[2] == 0).all()


def test_offsets_that_fall_or_leave_the_rows_are_reported(gpu_lib):
    for rows in (6, 400):
        x = data((rows, 64))
        w, ws = weight(3, 64, 64)
        packed = gpu_lib.moe_int8_pack_weight(w)
        for off in ([0, 4, 2, rows], [-1, 1, 2, rows], [0, 1, 2, rows + 1]):
            out = torch.full((rows, 64), 3.0, dtype=torch.bfloat16, device="cuda")
            gpu_lib.moe_int8_linear(x, dev(off), packed, ws, out=out)
            torch.cuda.synchronize()
            assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_ERR_INVALID_ARG
            assert (out == 3).all()


@pytest.mark.parametrize("T,capacity", [(3, 0), (200, 0), (200, 40), (700, 0)])
def test_the_dispatchs_schedule(gpu_lib, T, capacity):
    E, k, h, F = 6, 2, 128, 96
    x = data((T, h), "bf16", 4)
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(i))[:k] for i in range(T)]).int().cuda()
    d = gpu_lib.moe_dispatch(x, ids, E, capacity)
    gate, gs = weight(E, F, h, 5)
    up, us = weight(E, F, h, 6)
    down, ds = weight(E, h, F, 7)
    packed = gpu_lib.moe_int8_pack_expert_weights(gate, up, down)
    rows = d["rows"]
    out = torch.zeros((rows, h), dtype=torch.bfloat16, device="cuda")
    gpu_lib.moe_int8_expert_ffn(x, None, packed, gs, us, ds, src=d["src_token"], tile_sched=d["tile_sched"], out=out)
    again = torch.zeros_like(out)
    gpu_lib.moe_int8_expert_ffn(d["buf"], None, packed, gs, us, ds, tile_sched=d["tile_sched"], out=again)
    ok(gpu_lib)
    assert torch.equal(out, again)
    if not capacity:
        third = gpu_lib.moe_int8_expert_ffn(d["buf"], d["offsets"], packed, gs, us, ds)
        assert torch.equal(out, third)
    y = gpu_lib.moe_int8_linear(d["buf"], None, gpu_lib.moe_int8_pack_weight(gate), gs, tile_sched=d["tile_sched"], out=torch.zeros((rows, F), dtype=torch.bfloat16, device="cuda"))
    c, s = Q.quantize(f64(d["buf"]))
    off, kept = d["offsets"].cpu().numpy(), d["kept_counts"].cpu().numpy()
    for e in range(E):
        lo, hi = off[e], off[e] + kept[e]
        near(y[lo:hi], (c[lo:hi].astype(float) @ gate[e].cpu().numpy().astype(float).T) * s[lo:hi, None] * f64(gs)[e], "bf16")
        assert (out[hi:off[e + 1]] == 0).all() and (y[hi:off[e + 1]] == 0).all()
    # a schedule of other groups, and one whose rows are not the call's
    other, os_ = weight(5, F, h, 8)
    gpu_lib.moe_int8_linear(d["buf"], None, gpu_lib.moe_int8_pack_weight(other), os_, tile_sched=d["tile_sched"])
    torch.cuda.synchronize()
    assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_ERR_INVALID_ARG


FFN = [  # E, rows, h, F, kind
    (1, 1, 64, 32, "random"), (4, 3, 128, 96, "random"), (8, 20, 256, 192, "random"), (3, 300, 136, 200, "random"), (2, 700, 256, 512, "one"),
    (16, 900, 512, 320, "random"), (5, 33, 72, 1000, "random"), (2, 40, 7168, 64, "random"), (64, 500, 128, 64, "random")]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("E,rows,h,F,kind", FFN)
def test_expert_ffn(gpu_lib, dtype, E, rows, h, F, kind):
    x = data((rows, h), dtype, E * rows)
    gate, gs = weight(E, F, h, 2)
    up, us = weight(E, F, h, 3)
    down, ds = weight(E, h, F, 4)
    gs, us = gs * 0.05, us * 0.05                          # gates of a few units
    off = offsets_of(rows, E, rows, kind)
    y = gpu_lib.moe_int8_expert_ffn(x, dev(off), gpu_lib.moe_int8_pack_expert_weights(gate, up, down), gs, us, ds)
    ok(gpu_lib)
    a = Q.act(f64(x), off, gate.cpu().numpy(), f64(gs), up.cpu().numpy(), f64(us))
    # act is within 16 half steps of fp32 and one for each unit of the gate, so its codes are those of `a` but where a * 127 / amax
    # lies within 127 * that of a border; such a code may be one off
    amax = np.abs(a).max(1, keepdims=True)
    q = a * 127.0 / amax
    codes = np.rint(q)
    slack = 127.0 * 64 * F32 + 1e-9
    open_ = (np.abs(np.abs(q - np.floor(q)) - 0.5) < slack)
    scales = amax[:, 0] / 127.0
    want = Q.linear(codes, scales, off, down.cpu().numpy(), f64(ds))
    lim = np.zeros_like(want)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        lim[lo:hi] = (open_[lo:hi].astype(float) @ np.abs(down[e].cpu().numpy().astype(float)).T) * scales[lo:hi, None] * f64(ds)[e][None]
    # the scale itself carries act's error: 64 half steps of the sum of magnitudes
    mag = Q.linear(np.abs(codes), scales, off, np.abs(down.cpu().numpy().astype(np.int64)), f64(ds))
    near(y, want, dtype, lim + 64 * F32 * mag)


def test_gates_far_from_zero(gpu_lib):
    # gates near -200, 0 and 200: exp(-g) overflows on one side, and silu is 0 or g there
    h = F = 64
    x = torch.zeros(12, h)
    x[:, 0] = 1.0
    gate = torch.zeros(1, F, h, dtype=torch.int8)
    gate[0, :, 0] = torch.arange(F) * 4 - 128
    one = torch.zeros(1, F, h, dtype=torch.int8)
    one[0, :, 0] = 1
    down = torch.zeros(1, h, F, dtype=torch.int8)
    down[0] = torch.eye(h, dtype=torch.int8)
    gs, us, ds = torch.full((1, F), 1.6), torch.ones(1, F), torch.ones(1, h)
    for n in (2, 12):
        y = gpu_lib.moe_int8_expert_ffn(x[:n].cuda(), dev([0, n]), gpu_lib.moe_int8_pack_expert_weights(gate.cuda(), one.cuda(), down.cuda()), gs.cuda(), us.cuda(), ds.cuda())
        ok(gpu_lib)
        a = Q.act(x[:n].double().numpy(), [0, n], gate.numpy(), gs.double().numpy(), one.numpy(), us.double().numpy())
        step = np.abs(a).max() / 127
        assert torch.isfinite(y).all() and np.abs(f64(y) - a).max() <= step * 0.501


def test_captured_on_streams_with_changing_rows(gpu_lib):
    E, rows, h, F = 4, 500, 128, 96
    x = data((rows, h), "bf16", 1)
    gate, gs = weight(E, F, h, 2)
    up, us = weight(E, F, h, 3)
    down, ds = weight(E, h, F, 4)
    packed = gpu_lib.moe_int8_pack_expert_weights(gate, up, down)
    offs = [offsets_of(rows, E, i) for i in range(3)]
    want = [gpu_lib.moe_int8_expert_ffn(x, dev(o), packed, gs, us, ds) for o in offs]
    ok(gpu_lib)
    off = dev(offs[0])
    out = torch.empty((rows, h), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(gpu_lib.moe_int8_expert_ffn_workspace_size(E, h, F, rows), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        gpu_lib.moe_int8_expert_ffn(x, off, packed, gs, us, ds, out=out, ws=ws)
    for i in (0, 1, 2, 1):
        off.copy_(dev(offs[i]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    # two streams, each with its own workspace, at once
    outs = []
    for i in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        outs.append(gpu_lib.moe_int8_expert_ffn(x, dev(offs[i]), packed, gs, us, ds, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    ok(gpu_lib)


# ------------------------------------------------------------------------------------------ edges


@pytest.mark.parametrize("G,rows", [(1, 3), (6, 40), (2, 100), (2, 250), (2, 700), (20, 1000), (20, 2400)])
def test_waits_that_run_out_are_reported(gpu_lib, G, rows):
    """Every tile shape of the product, with a single poll for each wait: one that runs out is reported and leaves the device usable, and
    a call that reports none is whole. (A poll itself waits, as long as the chip sees fit.)"""
    K, N = 4096, 300
    x = data((rows, K), "bf16", 1)
    w, ws = weight(G, N, K)
    packed = gpu_lib.moe_int8_pack_weight(w)
    off = dev(np.linspace(0, rows, G + 1).astype(int))
    want = gpu_lib.moe_int8_linear(x, off, packed, ws)
    ok(gpu_lib)
    gpu_lib.moe_set_wait_limit(1)
    try:
        for _ in range(3):
            y = gpu_lib.moe_int8_linear(x, off, packed, ws)
            torch.cuda.synchronize()
            status = gpu_lib.moe_check_device_error()
            assert status == gpu_lib.MOE_ERR_TIMEOUT or (status == gpu_lib.MOE_OK and torch.equal(y, want))
    finally:
        gpu_lib.moe_set_wait_limit(0)
    assert torch.equal(gpu_lib.moe_int8_linear(x, off, packed, ws), want)
    ok(gpu_lib)


@pytest.mark.parametrize("rows", [6, 70, 500])
def test_a_bad_row_of_the_ffn_leaves_the_others(gpu_lib, rows):
    E, h, F = 2, 128, 96
    x = data((rows, h), "bf16", 3)
    gate, gs = weight(E, F, h, 2)
    up, us = weight(E, F, h, 3)
    down, ds = weight(E, h, F, 4)
    packed = gpu_lib.moe_int8_pack_expert_weights(gate, up, down)
    off = dev([0, rows // 2, rows])
    good = gpu_lib.moe_int8_expert_ffn(x, off, packed, gs, us, ds)
    x[1, 5] = float("nan")
    x[rows - 1, 0] = float("inf")
    x[2] = 0.0
    bad = gpu_lib.moe_int8_expert_ffn(x, off, packed, gs, us, ds)
    ok(gpu_lib)
    keep = torch.ones(rows, dtype=torch.bool)
    keep[[1, 2, rows - 1]] = False
    assert torch.equal(bad[keep], good[keep]) and bad[1].isnan().all() and bad[rows - 1].isnan().all() and (bad[2] == 0).all()


def test_a_rows_result_does_not_depend_on_the_batch(gpu_lib):
    """Sums below 2^24 are exact, so the kernels of few and of many rows give the same bits."""
    K, N = 512, 200
    x = data((900, K), "bf16", 5)
    w, ws = weight(1, N, K)
    packed = gpu_lib.moe_int8_pack_weight(w)
    whole = gpu_lib.moe_int8_linear(x, dev([0, 900]), packed, ws, out_dtype=torch.float32)
    for n in (1, 5, 8, 9, 16, 17, 33, 64, 100, 129, 256, 257):
        part = gpu_lib.moe_int8_linear(x[:n], dev([0, n]), packed, ws, out_dtype=torch.float32)
        assert torch.equal(part, whole[:n]), n
    ok(gpu_lib)


def test_outputs_and_rows_past_32_bit_offsets(gpu_lib):
    # 40000 x 60000 outputs; 140000 x 16384 values of rows
    K, N, rows = 64, 60000, 40000
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-300:] = data((300, K), "bf16", 7)
    w, ws = weight(1, N, K)
    y = gpu_lib.moe_int8_linear(x, dev([0, rows]), gpu_lib.moe_int8_pack_weight(w), ws)
    ok(gpu_lib)
    assert (y[:1000] == 0).all()
    part = gpu_lib.moe_int8_linear(x[-300:], dev([0, 300]), gpu_lib.moe_int8_pack_weight(w), ws)
    assert torch.equal(y[-300:], part)
    del y, x
    x = torch.zeros(140000, 16384, dtype=torch.bfloat16, device="cuda")
    x[-2:] = data((2, 16384), "bf16", 8)
    c, s = gpu_lib.moe_int8_quantize(x)
    d = gpu_lib.moe_int8_dequantize(c, s)
    ok(gpu_lib)
    code, scale = Q.quantize(f64(x[-2:]))
    np.testing.assert_array_equal(c[-2:].cpu().numpy(), code)
    assert torch.equal(d[-2:], (c[-2:].float() * s[-2:, None]).bfloat16()) and (s[:-2] == 0).all() and (d[70000] == 0).all()


def test_a_schedule_past_the_rows_is_cut(gpu_lib):
    w, ws = weight(1, 96, 64)
    x = data((40, 64))
    full = torch.full((60, 96), 5.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.moe_int8_linear(x, None, gpu_lib.moe_int8_pack_weight(w), ws, tile_sched=gpu_lib.moe_dense_tile_sched(128), out=full[:40])
    ok(gpu_lib)
    assert torch.equal(full[:40], gpu_lib.moe_int8_linear(x, dev([0, 40]), gpu_lib.moe_int8_pack_weight(w), ws)) and (full[40:] == 5).all()
    out = torch.full((40, 96), 5.0, dtype=torch.bfloat16, device="cuda")
    gpu_lib.moe_int8_linear(x, None, gpu_lib.moe_int8_pack_weight(w), ws, tile_sched=gpu_lib.moe_dense_tile_sched(128 * 20), out=out)
    torch.cuda.synchronize()
    assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_ERR_INVALID_ARG and (out == 5).all()


def test_no_rows_and_groups_without_rows(gpu_lib):
    w, ws = weight(4, 40, 64)
    packed = gpu_lib.moe_int8_pack_weight(w)
    assert gpu_lib.moe_int8_linear(data((0, 64)), dev([0] * 5), packed, ws).shape == (0, 40)
    for rows in (3, 300):
        out = torch.full((rows, 40), 2.0, dtype=torch.bfloat16, device="cuda")
        gpu_lib.moe_int8_linear(data((rows, 64)), dev([0] * 5), packed, ws, out=out)
        ok(gpu_lib)
        assert (out == 2).all()
        y = gpu_lib.moe_int8_linear(data((rows, 64)), dev([0, 0, rows, rows, rows]), packed, ws)
        assert torch.equal(y, gpu_lib.moe_int8_linear(data((rows, 64)), dev([0, rows]), gpu_lib.moe_int8_pack_weight(w[1:2]), ws[1:2]))
    none = torch.full((7,), -1, dtype=torch.int32, device="cuda")
    y = gpu_lib.moe_int8_linear(data((0, 64)), dev([0, 2, 4, 5, 7]), packed, ws, src=none)
    ok(gpu_lib)
    assert (y == 0).all()


# few rows a group, one SM's worth of tiles, and every tile of pairs: 64, 128 and 256 rows
@pytest.mark.parametrize("x_rows,rows,G,N,K", [(1, 5, 3, 40, 64), (7, 100, 20, 130, 200), (64, 512, 33, 257, 1044), (33, 700, 2, 520, 96),
                                               (200, 6000, 64, 384, 160), (100, 12000, 64, 384, 64), (500, 3000, 5, 700, 320),
                                               (2999, 3000, 3, 700, 70)])
def test_rows_that_several_of_the_call_name(gpu_lib, x_rows, rows, G, N, K):
    """x quantised once and its rows fetched by src: bit for bit the call on the rows written out, -1 among them."""
    w, ws = weight(G, N, K, 3)
    packed = gpu_lib.moe_int8_pack_weight(w)
    gen = np.random.default_rng(rows)
    src = gen.integers(-1, x_rows, rows).astype(np.int32)
    src[gen.integers(rows)] = x_rows - 1
    off = dev(offsets_of(rows, G, rows))
    for dtype, wide in (("bf16", False), ("fp32", True)):
        x = data((x_rows, K + 8), dtype, 2)[:, :K] if wide else data((x_rows, K), dtype, 2)
        whole = torch.where(dev(src)[:, None] < 0, torch.zeros((), dtype=x.dtype, device="cuda"), x[dev(src).clamp(min=0).long()])
        got = gpu_lib.moe_int8_linear(x, off, packed, ws, src=dev(src))
        want = gpu_lib.moe_int8_linear(whole, off, packed, ws)
        ok(gpu_lib)
        assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [20, 600, 6000])
def test_a_wrong_row_among_those_named(gpu_lib, rows):
    """Reported and taken as zeros; a row with an infinity is NaN wherever it is named, and nowhere else."""
    G, N, K, x_rows = 6, 200, 128, 10
    w, ws = weight(G, N, K, 4)
    packed = gpu_lib.moe_int8_pack_weight(w)
    x = data((x_rows, K), "bf16", 5)
    x[3, 17] = float("inf")
    src = torch.arange(rows, dtype=torch.int32, device="cuda") % x_rows
    off = dev(offsets_of(rows, G, 6))
    y = gpu_lib.moe_int8_linear(x, off, packed, ws, src=src)
    ok(gpu_lib)
    assert torch.equal(torch.isnan(y).any(1), src == 3) and torch.equal(torch.isnan(y).all(1), src == 3)
    for bad in (x_rows, -2, 2**31 - 1, -(2**31)):
        other = src.clone()
        other[rows // 2] = bad
        z = gpu_lib.moe_int8_linear(x, off, packed, ws, src=other)
        torch.cuda.synchronize()
        assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_ERR_INVALID_ARG
        assert (z[rows // 2] == 0).all()
        z[rows // 2] = y[rows // 2]
        assert torch.equal(z.nan_to_num(), y.nan_to_num())


@pytest.mark.parametrize("dtype,bits", [("bf16", 7), ("fp16", 10)])
def test_every_quotient_of_16_bit_numbers(gpu_lib, dtype, bits):
    """Codes of all significands under all largest ones, over the exponents that give codes other than 0: by whole numbers, ties to even."""
    n, one = 1 << bits, 1 << bits
    X = np.concatenate([np.arange(one, 2 * one, dtype=np.int64)] * 10)             # x = X 2^-d of the largest's exponent
    d = np.repeat(np.arange(10), n)
    for exponent in ((-60, 0, 120) if dtype == "bf16" else (-4, 0, 15)):
        for A0 in range(one, 2 * one, 128):
            A = np.arange(A0, A0 + 128, dtype=np.int64)[:, None]
            keep = (X[None] <= A) | (d[None] > 0)                                # below the largest
            num, den = 127 * X[None], A << d[None]
            q, r = num // den, num % den
            q += (2 * r > den) | ((2 * r == den) & (q & 1 == 1))
            x = np.where(keep, X * 2.0 ** -d, 0.0)
            x[:, 1::2] *= -1
            x = np.concatenate([A.astype(float), x], 1) * 2.0 ** (exponent - bits)
            t = torch.from_numpy(x).to(DT[dtype]).cuda()
            # (fp16's lowest exponent: what is subnormal loses bits, and counts with the bits it has)
            exact = t.double().cpu().numpy() == x
            want = np.concatenate([np.full((128, 1), 127), np.where(keep, q, 0) * np.where(np.arange(len(X)) % 2, -1, 1)], 1)
            c, _ = gpu_lib.moe_int8_quantize(t)
            assert exact[:, : 2 * n].all()
            np.testing.assert_array_equal(c.cpu().numpy()[exact], want[exact])
            codes, _ = gpu_lib.moe_checkpoint8_save(torch.cat([t[:, :1], t[:, 1:128]], 1).contiguous())
            np.testing.assert_array_equal(codes.cpu().numpy()[exact[:, :128]], want[:, :128][exact[:, :128]])
    ok(gpu_lib)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(40, 33), (19, 47), (35, 2033), (18, 2047), (35, 3001), (33, 4081), (17, 4097), (16, 17), (3, 9999)])
def test_rows_that_start_on_no_boundary(gpu_lib, dtype, rows, K):
    """Contiguous matrices whose rows begin and end within 16-byte pieces, there and back; the same with row strides, which go another way;
    with what lies around left alone."""
    x = data((rows, K), dtype, K, 2.0)
    code, scale = Q.quantize(f64(x))
    room = torch.full((rows * K + 64,), 77, dtype=torch.int8, device="cuda")
    codes = room[16: 16 + rows * K].view(rows, K)
    c, s = gpu_lib.moe_int8_quantize(x, codes=codes)
    wide = torch.zeros((rows, K + 3), dtype=x.dtype, device="cuda")
    wide[:, :K] = x
    c2, s2 = gpu_lib.moe_int8_quantize(wide[:, :K])
    ok(gpu_lib)
    np.testing.assert_array_equal(c.cpu().numpy(), code)
    np.testing.assert_array_equal(f64(s), scale)
    assert torch.equal(c, c2) and torch.equal(s, s2)
    assert (room[:16] == 77).all() and (room[16 + rows * K:] == 77).all()
    back = torch.full((rows * K + 64,), 5.0, dtype=x.dtype, device="cuda")
    out = back[32: 32 + rows * K].view(rows, K)
    gpu_lib.moe_int8_dequantize(codes, s, out=out)
    strided = gpu_lib.moe_int8_dequantize(codes, s, out=wide[:, :K])
    ok(gpu_lib)
    want = (c.float() * s.unsqueeze(1)).to(x.dtype)
    assert torch.equal(out, want) and torch.equal(strided, want)
    assert (back[:32] == 5).all() and (back[32 + rows * K:] == 5).all() and (wide[:, K:] == 0).all()


# 8, 4 and 2 CTAs to a tile (by its columns and the number of tiles), groups without rows, tiles of one row to sixteen, ragged columns
@pytest.mark.parametrize("G,rows,N,K", [(1, 1, 96, 6528), (2, 16, 96, 6528), (2, 2, 32, 2720), (3, 7, 130, 4099), (1, 16, 128, 1024), (1, 40, 257, 3000),
                                       (2, 30, 64, 16384), (5, 9, 384, 2048), (1, 16, 2000, 1500), (40, 12, 70, 5000), (1, 33, 1, 131072)])
def test_long_rows_by_few_channels(gpu_lib, G, rows, N, K):
    w, ws = weight(G, N, K, 5)
    packed = gpu_lib.moe_int8_pack_weight(w)
    off = offsets_of(rows, G, G)
    for dtype in ("bf16", "fp32"):
        x = data((rows, K), dtype, 6)
        y = gpu_lib.moe_int8_linear(x, dev(off), packed, ws)
        again = gpu_lib.moe_int8_linear(x, dev(off), packed, ws)
        ok(gpu_lib)
        c, s = Q.quantize(f64(x))
        want = np.concatenate([(c[a:b].astype(float) @ w[g].cpu().numpy().astype(float).T) * s[a:b, None] * f64(ws)[g] for g, (a, b) in
                               enumerate(zip(off[:-1], off[1:]))])
        assert torch.equal(y, again)
        near(y, want, dtype)


@pytest.mark.parametrize("T", [1, 9])
def test_an_ffn_of_few_channels_and_long_rows(gpu_lib, T):
    E, h, F = 2, 96, 6528
    gate, gs = weight(E, F, h, 1)
    up, us = weight(E, F, h, 2)
    down, ds = weight(E, h, F, 3)
    packed = gpu_lib.moe_int8_pack_expert_weights(gate, up, down)
    x = data((T, h), "bf16", T)
    off = dev([0, T // 2, T])
    y = gpu_lib.moe_int8_expert_ffn(x, off, packed, gs, us, ds)
    # of its parts: the two products and the activation in fp32, quantised by rows
    g = gpu_lib.moe_int8_linear(x, off, gpu_lib.moe_int8_pack_weight(gate), gs, out_dtype=torch.float32)
    u = gpu_lib.moe_int8_linear(x, off, gpu_lib.moe_int8_pack_weight(up), us, out_dtype=torch.float32)
    act = torch.nn.functional.silu(g.double()) * u.double()
    want = gpu_lib.moe_int8_linear(act.float(), off, gpu_lib.moe_int8_pack_weight(down), ds, out_dtype=torch.float32).double()
    ok(gpu_lib)
    # an activation in another last bit moves a code by one step at most: 6528 of them, a hundredth near a border at the very most
    step = act.abs().amax(1, keepdim=True) / 127 * 128 * ds.double().max()
    assert ((y.double() - want).abs() <= want.abs() * HALF_STEP["bf16"] + 65 * step).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 16), (300, 16), (77, 32), (1000, 48), (33, 64), (5, 112), (129, 128), (64, 144), (17, 240), (40, 256), (9, 272)])
def test_short_rows(gpu_lib, dtype, rows, K):
    """Several rows to a warp; an infinite row and one of zeros between others, rows named by src, and as a product's operand."""
    x = data((rows, K), dtype, K, 2.0)
    if rows > 4:
        x[1, K - 1], x[3] = float("inf"), 0.0
    src = torch.randint(-1, rows, (2 * rows + 1,), generator=torch.Generator().manual_seed(K)).int().cuda()
    code, scale = Q.quantize(f64(x))
    c, s = gpu_lib.moe_int8_quantize(x)
    cs, ss = gpu_lib.moe_int8_quantize(x, src=src)
    ok(gpu_lib)
    np.testing.assert_array_equal(c.cpu().numpy(), code)
    np.testing.assert_array_equal(f64(s), scale)
    at, none = src.clamp(min=0).long(), src < 0
    assert torch.equal(cs, torch.where(none[:, None], 0, c[at]).to(torch.int8))
    np.testing.assert_array_equal(f64(ss), f64(torch.where(none, 0.0, s[at])))
    w, ws = weight(1, 24, K, 3)
    y = gpu_lib.moe_int8_linear(x, dev([0, rows]), gpu_lib.moe_int8_pack_weight(w), ws)
    near(y, (code.astype(float) @ w[0].cpu().numpy().astype(float).T) * scale[:, None] * f64(ws)[0], dtype)
    ok(gpu_lib)
