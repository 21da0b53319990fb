"""The 4-bit expert operators on the GPU against the float64 oracle: codes and scales exactly, products and the FFN
within bounds that count the fp32 sums, the output's rounding and the activations that lie at a rounding tie."""
import numpy as np
import pytest
import torch

from oracle import fp4_oracle as Q

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
HALF_STEP = {k: torch.finfo(v).eps / 2 for k, v in DT.items()}


def data(shape, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).cuda()


def f64(t):
    return t.double().cpu().numpy()


def ok(moe):
    torch.cuda.synchronize()
    assert moe.moe_check_device_error() == moe.MOE_OK, moe.moe_last_error_string()


def weight(moe, G, N, K, fmt, seed, gscale=None):
    w = data((G * N, K), "bf16", seed, K**-0.5)
    c, s = moe.moe_fp4_quantize(w, fmt, gscale=gscale)
    v = Q.dequantize(Q.unpack_codes(c.cpu().numpy(), K), s.cpu().numpy(), fmt).reshape(G, N, K)
    return c.view(G, N, -1), s.view(G, N, -1), v


# ------------------------------------------------------------------------------------------ quantisation


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 7168), (3, 15), (5, 16), (7, 31), (2, 33), (129, 64), (33, 100), (17, 999),
                                    (300, 512), (4, 1040), (70, 2048)])
def test_quantize_is_the_definition(gpu_lib, fmt, dtype, rows, K):
    x = data((rows, K), dtype, rows * 7919 + K, 3.0)
    c, s = gpu_lib.moe_fp4_quantize(x, fmt)
    ok(gpu_lib)
    code, byte = Q.quantize(f64(x), fmt)
    np.testing.assert_array_equal(s.cpu().numpy(), byte)
    np.testing.assert_array_equal(Q.unpack_codes(c.cpu().numpy(), K), code)
    for out in ("fp32", dtype):
        y = gpu_lib.moe_fp4_dequantize(c, s, K, fmt, dtype=DT[out])
        want = torch.from_numpy(Q.dequantize(code, byte, fmt)).to(DT[out])
        assert torch.equal(y.cpu(), want)
    ok(gpu_lib)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_quantize_with_a_multiplier(gpu_lib, fmt):
    # a power of two times bf16 is exact, and so is the quotient on the way back: the definition to the bit
    x = data((65, 96), "bf16", 5)
    g = torch.tensor([0.0625], device="cuda")
    c, s = gpu_lib.moe_fp4_quantize(x, fmt, gscale=g)
    y = gpu_lib.moe_fp4_dequantize(c, s, 96, fmt, gscale=g, dtype=torch.float32)
    code, byte = Q.quantize(f64(x) * 0.0625, fmt)
    np.testing.assert_array_equal(s.cpu().numpy(), byte)
    np.testing.assert_array_equal(Q.unpack_codes(c.cpu().numpy(), 96), code)
    np.testing.assert_array_equal(f64(y), Q.dequantize(code, byte, fmt) / 0.0625)
    # any other: the way back is the rounded quotient, one half step of fp32
    g.fill_(58.35)
    y = gpu_lib.moe_fp4_dequantize(c, s, 96, fmt, gscale=g, dtype=torch.float32)
    want = Q.dequantize(code, byte, fmt) / float(g)
    assert (np.abs(f64(y) - want) <= 2.0**-24 * np.abs(want)).all()
    ok(gpu_lib)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("g", [58.35, -0.7, 1e-3])
def test_quantize_with_any_multiplier(gpu_lib, fmt, dtype, g):
    """Codes and scales are those of x * g rounded to fp32, by the row-major kernel and element by element."""
    x = data((300, 999), dtype, 5)
    mult = torch.tensor([g], device="cuda")
    c, s = gpu_lib.moe_fp4_quantize(x, fmt, gscale=mult)
    ok(gpu_lib)
    code, byte = Q.quantize(np.float64(np.float32(f64(x) * float(mult))), fmt)
    np.testing.assert_array_equal(s.cpu().numpy(), byte)
    np.testing.assert_array_equal(Q.unpack_codes(c.cpu().numpy(), 999), code)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("g", [1e-40, -1e-39, 1e-30, 1e16, -3e38])
def test_dequantize_with_a_multiplier_at_the_ends_of_the_range(gpu_lib, fmt, g):
    """The quotient code * scale / g rounded to fp32, where 1 / g is infinite or below the normal range too: zeros stay 0."""
    x = data((40, 96), "fp32", 5)
    x[::3] = 0.0
    x[1::3] *= 2.0**-60
    c, s = gpu_lib.moe_fp4_quantize(x, fmt)
    mult = torch.tensor([g], device="cuda")
    y = gpu_lib.moe_fp4_dequantize(c, s, 96, fmt, gscale=mult, dtype=torch.float32)
    ok(gpu_lib)
    with np.errstate(over="ignore"):
        want = np.float32(f64(gpu_lib.moe_fp4_dequantize(c, s, 96, fmt, dtype=torch.float32)) / float(mult))
    assert (want[::3] == 0).all()
    np.testing.assert_array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_at_the_edges(gpu_lib, fmt, dtype):
    """Zeros, values at ties, the type's largest and smallest, infinities and NaN, each in blocks of their own."""
    fi = torch.finfo(DT[dtype])
    x = torch.zeros((12, 64), dtype=torch.float64)
    x[1, :] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]).repeat(8) * torch.tensor([1.0, -1.0]).repeat(32)
    x[2, 0], x[2, 40] = fi.max, -fi.max
    x[3, :] = fi.tiny
    x[4, 3] = fi.smallest_normal * fi.eps
    x[5, 0], x[5, 1], x[5, 63] = float("inf"), -1.0, float("-inf")
    x[6, 5], x[6, 6] = float("nan"), 2.0
    x[7, :] = 6 * 448.0 * 1.5
    x[8, :] = 2.0**-10 * 6
    x[9, :] = -0.0
    x[10, 0], x[10, 1] = fi.max, 1.0
    x[11, 16] = 6 * 17 / 16            # amax / 6 half way between two e4m3 values
    x = x.to(DT[dtype]).cuda()
    c, s = gpu_lib.moe_fp4_quantize(x, fmt)
    ok(gpu_lib)
    code, byte = Q.quantize(f64(x), fmt)
    np.testing.assert_array_equal(s.cpu().numpy(), byte)
    np.testing.assert_array_equal(Q.unpack_codes(c.cpu().numpy(), 64), code)
    y = gpu_lib.moe_fp4_dequantize(c, s, 64, fmt, dtype=torch.float32)
    with np.errstate(over="ignore"):
        want = Q.dequantize(code, byte, fmt).astype(np.float32)
    np.testing.assert_array_equal(f64(y), want.astype(np.float64))


def test_quantize_rows_by_index_and_strides(gpu_lib):
    base = data((50, 300), "bf16", 9)
    x = base[:, 7:207]                                       # rows 600 bytes apart, starting on 14
    src = torch.tensor([3, -1, 49, 0, 3, 11], dtype=torch.int32, device="cuda")
    c, s = gpu_lib.moe_fp4_quantize(x, "nv", src=src)
    want = np.where(src.cpu().numpy()[:, None] >= 0, f64(x)[src.cpu().numpy().clip(0)], 0.0)
    code, byte = Q.quantize(want, "nv")
    np.testing.assert_array_equal(s.cpu().numpy(), byte)
    np.testing.assert_array_equal(Q.unpack_codes(c.cpu().numpy(), 200), code)
    out = torch.full((6, 256), 7.0, device="cuda")[:, 5:205]
    gpu_lib.moe_fp4_dequantize(c, s, 200, "nv", out=out)
    np.testing.assert_array_equal(f64(out), Q.dequantize(code, byte, "nv"))
    assert (out._base[:, :5] == 7).all() and (out._base[:, 205:] == 7).all()
    ok(gpu_lib)
    # an index outside x: a row of zeros, and reported
    src[2] = 50
    c, s = gpu_lib.moe_fp4_quantize(x, "nv", src=src)
    torch.cuda.synchronize()
    assert gpu_lib.moe_check_device_error() == gpu_lib.MOE_ERR_INVALID_ARG
    assert (Q.unpack_codes(c.cpu().numpy(), 200)[2] == 0).all()
    ok(gpu_lib)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_offsets_past_32_bits(gpu_lib, fmt):
    """2.2e9 values: the last rows are those of a call of their own, there and back, and through the product."""
    moe = gpu_lib
    rows, K, N = 1 << 20, 2080, 40
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    x[-300:] = data((300, K), "bf16", 3)
    c, s = moe.moe_fp4_quantize(x, fmt)
    c1, s1 = moe.moe_fp4_quantize(x[-300:], fmt)
    assert torch.equal(c[-300:], c1) and torch.equal(s[-300:], s1)
    y = moe.moe_fp4_dequantize(c, s, K, fmt)
    assert torch.equal(y[-300:], moe.moe_fp4_dequantize(c1, s1, K, fmt))
    ok(moe)
    del y, c, s
    wc, wsc, _ = weight(moe, 2, N, K, fmt, 5)
    packed = moe.moe_fp4_pack_weight(wc, wsc, K, fmt)
    off = torch.tensor([0, rows - 200, rows], dtype=torch.int32, device="cuda")
    y = moe.moe_fp4_linear(x, off, packed, N, fmt)
    off = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    assert torch.equal(y[-300:], moe.moe_fp4_linear(x[-300:].contiguous(), off, packed, N, fmt))
    ok(moe)


# ----------------------------------------------------------------------------------------------- product


def check_linear(moe, counts, N, K, fmt, dtype, out_dtype=None, alpha=None, gscale=None, src=None, x_rows=None, seed=1):
    out_dtype = out_dtype or dtype
    G, rows = len(counts), int(sum(counts))
    x = data((x_rows if x_rows is not None else rows, K), dtype, seed)
    c, s, w = weight(moe, G, N, K, fmt, seed + 1)
    packed = moe.moe_fp4_pack_weight(c, s, K, fmt)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = moe.moe_fp4_linear(x, torch.from_numpy(off).cuda(), packed, N, fmt, alpha=alpha, gscale=gscale, src=src,
                           out_dtype=DT[out_dtype])
    ok(moe)
    xx = f64(x) if src is None else np.where(src.cpu().numpy()[:, None] >= 0, f64(x)[src.cpu().numpy().clip(0)], 0.0)
    a = Q.dequantize(*Q.quantize(xx * (1.0 if gscale is None else float(gscale)), fmt), fmt)
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        al = 1.0 if alpha is None else float(alpha[g])
        want = a[lo:hi] @ w[g].T * al
        bound = Q.product_bound(a[lo:hi] * al, w[g], want, HALF_STEP[out_dtype])
        assert (np.abs(f64(y[lo:hi]) - want) <= bound).all(), (g, np.abs(f64(y[lo:hi]) - want).max())


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 64, 64), ([1], 1, 1), ([0, 1, 0], 128, 256), ([3, 0, 130, 1], 192, 320), ([128, 129, 127], 200, 512),
    ([5], 1000, 33), ([33, 64, 96, 97], 65, 1000), ([300], 448, 2048), ([1] * 40, 256, 768), ([0, 0], 64, 64),
    ([700, 1], 640, 192)])
def test_linear(gpu_lib, fmt, counts, N, K):
    check_linear(gpu_lib, counts, N, K, fmt, "bf16")


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32"), ("fp32", "bf16")])
def test_linear_types_multipliers_and_rows_by_index(gpu_lib, fmt, dtype, out_dtype):
    src = torch.tensor([4, 0, 0, -1, 9, 8, 7, 1, 2, 2, 9], dtype=torch.int32, device="cuda")
    check_linear(gpu_lib, [4, 0, 7], 96, 160, fmt, dtype, out_dtype, alpha=torch.tensor([0.5, 9.0, -3.0], device="cuda"),
                 gscale=torch.tensor([8.0], device="cuda"), src=src, x_rows=10)


@pytest.mark.parametrize("fmt,dtype", [("nv", "bf16"), ("mx", "fp32")])
@pytest.mark.parametrize("counts,N,K", [([866, 1729, 5], 2100, 256), ([3000, 5995, 5], 1300, 128), ([6666, 13329, 5], 600, 64),
                                        ([200] * 23 + [131], 1304, 1100), ([300, 5401], 2240, 1344), ([5000], 1000, 2048)])
def test_linear_of_many_tiles(gpu_lib, counts, N, K, fmt, dtype):
    """Enough tiles for each tile width and for pairs of SMs, and more tiles than SMs: the accumulators and the ring wrap
    around, groups end on half a pair, and the output is stored in whole boxes and row by row."""
    check_linear(gpu_lib, counts, N, K, fmt, dtype)


def ragged(G, most, seed):
    """Rows of G groups, a fifth of them empty."""
    n = np.random.default_rng(seed).integers(0, most, G)
    n[::5] = 0
    return [int(v) for v in n]


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("G,most,N,K", [(129, 9, 48, 64), (449, 5, 48, 96), (1024, 4, 40, 64),     # one SM to a tile
                                        (45, 700, 700, 512), (70, 600, 1100, 300)])                # pairs of SMs
def test_linear_of_many_groups(gpu_lib, fmt, G, most, N, K):
    """More groups than the threads' and warps' shares of the scans over them, by offsets, and the same bits by a schedule."""
    moe = gpu_lib
    counts = ragged(G, most, G)
    check_linear(moe, counts, N, K, fmt, "bf16", "fp32")
    x = data((sum(counts), K), "bf16", 1)
    c, s, _ = weight(moe, G, N, K, fmt, 2)
    packed = moe.moe_fp4_pack_weight(c, s, K, fmt)
    at = [0] + [int(v) for v in np.cumsum(counts)]
    y = moe.moe_fp4_linear(x, torch.tensor(at, dtype=torch.int32, device="cuda"), packed, N, fmt)
    z = moe.moe_fp4_linear(x, None, packed, N, fmt, G=G, tile_sched=tile_sched(list(zip(at, at[1:]))))
    ok(moe)
    assert torch.equal(y, z)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_linear_of_many_groups_and_rows_used_many_times(gpu_lib, fmt):
    counts = ragged(300, 40, 3)
    src = torch.randint(-1, 600, (sum(counts),), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    check_linear(gpu_lib, counts, 48, 1100, fmt, "bf16", src=src, x_rows=600)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_expert_ffn_of_many_experts(gpu_lib, fmt):
    check_ffn(gpu_lib, ragged(200, 9, 4), 64, 96, fmt, "bf16", T=100)


def test_linear_keeps_other_rows_and_columns(gpu_lib):
    moe = gpu_lib
    c, s, w = weight(moe, 2, 40, 64, "nv", 3)
    packed = moe.moe_fp4_pack_weight(c, s, 64, "nv")
    x = data((20, 64), "bf16", 4)
    full = torch.full((20, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([2, 6, 13], dtype=torch.int32, device="cuda")
    moe.moe_fp4_linear(x, off, packed, 40, "nv", out=full[:, 3:43])
    ok(moe)
    assert (full[:2] == 5).all() and (full[13:] == 5).all() and (full[:, :3] == 5).all() and (full[:, 43:] == 5).all()
    a = Q.dequantize(*Q.quantize(f64(x), "nv"), "nv")
    for g, lo, hi in ((0, 2, 6), (1, 6, 13)):
        want = a[lo:hi] @ w[g].T
        assert (np.abs(f64(full[lo:hi, 3:43]) - want) <= Q.product_bound(a[lo:hi], w[g], want, 2.0**-8)).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,ldo", [(45, 48), (1, 8), (37, 40), (75, 80), (97, 104), (127, 128), (2045, 2048), (1990, 2000)])
@pytest.mark.parametrize("rows", [200, 2600])
def test_linear_writes_its_columns_alone(gpu_lib, dtype, N, ldo, rows):
    """Outputs of any width in rows that start on 16 bytes, one SM and pairs of SMs to a tile: the columns beside them stay."""
    moe = gpu_lib
    c, s, w = weight(moe, 2, N, 192, "mx", 3)
    packed = moe.moe_fp4_pack_weight(c, s, 192, "mx")
    x = data((rows, 192), "bf16", 4)
    full = torch.full((rows, ldo), 5.0, dtype=DT[dtype], device="cuda")
    off = torch.tensor([0, rows - 130, rows], dtype=torch.int32, device="cuda")
    moe.moe_fp4_linear(x, off, packed, N, "mx", out=full[:, :N])
    ok(moe)
    assert (full[:, N:] == 5).all()
    a = Q.dequantize(*Q.quantize(f64(x), "mx"), "mx")
    for g, lo, hi in ((0, 0, rows - 130), (1, rows - 130, rows)):
        want = a[lo:hi] @ w[g].T
        bound = Q.product_bound(a[lo:hi], w[g], want, HALF_STEP[dtype]) + (2.0**-25 if dtype == "fp16" else 0.0)
        assert (np.abs(f64(full[lo:hi, :N]) - want) <= bound).all()


@pytest.mark.parametrize("off", [[0, 5, 3, 20], [-1, 5, 6, 20], [0, 5, 6, 21]])
def test_bad_offsets_are_reported_and_nothing_is_written(gpu_lib, off):
    moe = gpu_lib
    c, s, _ = weight(moe, 3, 32, 64, "mx", 3)
    packed = moe.moe_fp4_pack_weight(c, s, 64, "mx")
    out = torch.full((20, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_fp4_linear(data((20, 64), "bf16"), torch.tensor(off, dtype=torch.int32, device="cuda"), packed, 32, "mx", out=out)
    torch.cuda.synchronize()
    assert moe.moe_check_device_error() == moe.MOE_ERR_INVALID_ARG
    assert (out == 5).all()
    ok(moe)


def test_a_nan_row_stays_in_its_row(gpu_lib):
    moe = gpu_lib
    c, s, _ = weight(moe, 1, 64, 128, "nv", 3)
    packed = moe.moe_fp4_pack_weight(c, s, 128, "nv")
    x = data((150, 128), "bf16", 8)
    off = torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    y0 = moe.moe_fp4_linear(x, off, packed, 64, "nv")
    x[77, 5] = float("nan")
    y1 = moe.moe_fp4_linear(x, off, packed, 64, "nv")
    ok(moe)
    assert torch.isnan(y1[77]).all()
    keep = [i for i in range(150) if i != 77]
    assert torch.equal(y0[keep], y1[keep])


@pytest.mark.parametrize("counts,N", [([3, 2], 96), ([900, 1000], 2304)])
def test_a_wait_that_runs_out_is_reported(gpu_lib, counts, N):
    """With one poll to a wait the roles give up (the epilogue waits for 32768 columns of products): the call reports
    MOE_ERR_TIMEOUT, and the next one is whole again (one SM and a pair of SMs to a tile)."""
    moe = gpu_lib
    K = 32768
    g = torch.Generator("cuda").manual_seed(1)
    c = torch.randint(0, 256, (2, N, K // 2), dtype=torch.uint8, device="cuda", generator=g)
    packed = moe.moe_fp4_pack_weight(c, torch.full((2, N, K // 16), 0x28, dtype=torch.uint8, device="cuda"), K, "nv")
    x = torch.randn((sum(counts), K), device="cuda", generator=g).bfloat16()
    off = torch.tensor([0, counts[0], sum(counts)], dtype=torch.int32, device="cuda")
    want = moe.moe_fp4_linear(x, off, packed, N, "nv")
    ok(moe)
    moe.moe_set_wait_limit(1)
    try:
        moe.moe_fp4_linear(x, off, packed, N, "nv")
        torch.cuda.synchronize()
        assert moe.moe_check_device_error() == moe.MOE_ERR_TIMEOUT
    finally:
        moe.moe_set_wait_limit(0)
    assert torch.equal(moe.moe_fp4_linear(x, off, packed, N, "nv"), want)
    ok(moe)


@pytest.mark.parametrize("G", [1, 5])
def test_another_calls_schedule_is_reported(gpu_lib, G):
    """A tile schedule of another number of groups, or of more rows than the call has, computes nothing."""
    moe = gpu_lib
    c, s, _ = weight(moe, 5, 32, 64, "mx", 3)
    packed = moe.moe_fp4_pack_weight(c, s, 64, "mx")
    sched = moe.moe_dense_tile_sched(128 * 20)
    out = torch.full((40, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_fp4_linear(data((40, 64), "bf16"), None, packed, 32, "mx", G=G, tile_sched=sched, out=out)
    torch.cuda.synchronize()
    assert moe.moe_check_device_error() == moe.MOE_ERR_INVALID_ARG
    assert (out == 5).all()
    ok(moe)


def test_a_schedule_past_the_rows_is_cut(gpu_lib):
    """A tile schedule whose tile ends past the call's rows: the rows there are, and nothing after them."""
    moe = gpu_lib
    c, s, w = weight(moe, 1, 32, 64, "mx", 3)
    packed = moe.moe_fp4_pack_weight(c, s, 64, "mx")
    x = data((40, 64), "bf16")
    full = torch.full((60, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_fp4_linear(x, None, packed, 32, "mx", G=1, tile_sched=moe.moe_dense_tile_sched(128), out=full[:40])
    ok(moe)
    assert (full[40:] == 5).all()
    a = Q.dequantize(*Q.quantize(f64(x), "mx"), "mx")
    want = a @ w[0].T
    assert (np.abs(f64(full[:40]) - want) <= Q.product_bound(a, w[0], want, 2.0**-8)).all()


def tile_sched(groups, first=None):
    """The tile schedule of groups of rows [(begin, end)]; first: other words in the place of its tiles before each group."""
    tiles = [(g, r, min(r + 128, hi), 0) for g, (lo, hi) in enumerate(groups) for r in range(lo, hi, 128)]
    before = [sum(t[0] < g for t in tiles) for g in range(len(groups) + 1)]
    words = [len(tiles), len(groups)] + (first or before)
    words += [0] * (-len(words) % 4) + [v for t in tiles for v in t]
    return torch.tensor(words, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("groups,first,rows,N,K", [
    ([(0, 256)], None, 40, 32, 64),                      # its second tile starts past the rows
    ([(0, 100), (200, 300)], None, 150, 96, 320),        # a group past the rows
    ([(0, 100), (150, 300)], None, 150, 200, 64),        # a group that starts where the rows end
    ([(0, 5120)], None, 4990, 1000, 2048),               # the same by pairs of SMs
    ([(0, 5119), (5119, 5120)], None, 5000, 1000, 2048),
    ([(0, 100), (100, 300)], [0, 2, 1], 300, 64, 64),    # counts that fall
    ([(0, 100), (100, 300)], [1, 1, 3], 300, 64, 64),
    ([(0, 100), (100, 300)], [0, 1, 2], 300, 64, 64)])   # a tile of no group
def test_a_schedule_of_other_rows_is_reported(gpu_lib, groups, first, rows, N, K):
    """A tile schedule that has as many groups and tiles as the call may have, but of other rows, computes nothing; the next
    call is whole."""
    moe = gpu_lib
    G = len(groups)
    c, s, _ = weight(moe, G, N, K, "mx", 3)
    packed = moe.moe_fp4_pack_weight(c, s, K, "mx")
    x = data((rows, K), "bf16", 4)
    out = torch.full((rows, N), 5.0, dtype=torch.bfloat16, device="cuda")
    sched = tile_sched(groups, first)
    moe.moe_fp4_linear(x, None, packed, N, "mx", G=G, tile_sched=sched, out=out)
    torch.cuda.synchronize()
    assert moe.moe_check_device_error() == moe.MOE_ERR_INVALID_ARG
    assert (out == 5).all()
    own = [(min(lo, rows), min(hi, rows)) for lo, hi in groups]
    y = moe.moe_fp4_linear(x, None, packed, N, "mx", G=G, tile_sched=tile_sched(own))
    off = torch.tensor([lo for lo, _ in own] + [own[-1][1]], dtype=torch.int32, device="cuda")
    z = moe.moe_fp4_linear(x, off, packed, N, "mx")
    ok(moe)
    for lo, hi in own:
        assert torch.equal(y[lo:hi], z[lo:hi])


@pytest.mark.parametrize("rows", [300, 3000])
def test_buffers_rewritten_between_calls(gpu_lib, rows):
    """Offsets, row indices, multipliers, rows and schedule rewritten in place between calls that follow at once: each call
    sees its own (the kernels start ahead of those before them, and no call may see the last one's)."""
    moe = gpu_lib
    G, N, K = 6, 320, 512
    c, s, _ = weight(moe, G, N, K, "nv", 3)
    packed = moe.moe_fp4_pack_weight(c, s, K, "nv")
    g = torch.Generator().manual_seed(rows)
    sets = []
    for i in range(6):
        cuts = torch.sort(torch.randint(0, rows + 1, (G - 1,), generator=g)).values
        off = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.full((1,), rows)]).int().cuda()
        sets.append((data((rows, K), "bf16", i), off, torch.rand(G, generator=g).cuda() + 0.5,
                     torch.randperm(rows, generator=g).int().cuda()))
    want = [moe.moe_fp4_linear(x, off, packed, N, "nv", alpha=al, src=src) for x, off, al, src in sets]
    torch.cuda.synchronize()
    x, off, al, src = (t.clone() for t in sets[0])
    ws = torch.empty(moe.moe_fp4_linear_workspace_size(G, K, rows, "nv"), dtype=torch.uint8, device="cuda")
    got = []
    for k in range(90):
        for t, new in zip((x, off, al, src), sets[k % 6]):
            t.copy_(new)
        got.append(moe.moe_fp4_linear(x, off, packed, N, "nv", alpha=al, src=src, ws=ws))
    ok(moe)
    for k, y in enumerate(got):
        assert torch.equal(y, want[k % 6]), k


# --------------------------------------------------------------------------------------------------- FFN


def check_ffn(moe, counts, h, F, fmt, dtype, out_dtype=None, scaled=False, T=None, seed=1):
    out_dtype = out_dtype or dtype
    E, rows = len(counts), int(sum(counts))
    rng = np.random.default_rng(seed)
    x = data((T or rows, h), dtype, seed)
    src = None if T is None else torch.from_numpy(rng.integers(-1, T, rows).astype(np.int32)).cuda()
    mats = [weight(moe, E, n, k, fmt, seed + 10 + i) for i, (n, k) in enumerate(((F, h), (F, h), (h, F)))]
    packed = moe.moe_fp4_pack_expert_weights(*((m[0], m[1]) for m in mats), h, F, fmt)
    al = [torch.from_numpy(rng.uniform(0.25, 1.5, E).astype(np.float32)).cuda() if scaled else None for _ in range(3)]
    gs, ags = (torch.tensor([v], device="cuda") if scaled else None for v in (4.0, 32.0))
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = moe.moe_fp4_expert_ffn(x, torch.from_numpy(off).cuda(), packed, F, fmt, src=src, alpha_gate=al[0], alpha_up=al[1],
                               alpha_down=al[2], gscale=gs, act_gscale=ags, out_dtype=DT[out_dtype])
    ok(moe)
    xx = f64(x) if src is None else np.where(src.cpu().numpy()[:, None] >= 0, f64(x)[src.cpu().numpy().clip(0)], 0.0)
    a = Q.dequantize(*Q.quantize(xx * (4.0 if scaled else 1.0), fmt), fmt)
    tight = []
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        A = [1.0 if t is None else float(t[e]) for t in al]
        g, u = (a[lo:hi] @ mats[i][2][e].T * A[i] for i in (0, 1))
        eg, eu = (Q.product_bound(a[lo:hi] * A[i], mats[i][2][e], (g, u)[i], 2.0**-24) for i in (0, 1))
        act, err = Q.swiglu_bound(g, eg, u, eu)
        m = 32.0 if scaled else 1.0
        q, dq = Q.requantized(act * m, err * m, fmt)
        want = q @ mats[2][2][e].T * A[2]
        bound = Q.product_bound(q * A[2], mats[2][2][e], want, HALF_STEP[out_dtype])
        bound = bound + (1 + HALF_STEP[out_dtype]) * (dq * A[2]) @ np.abs(mats[2][2][e]).T
        got = f64(y[lo:hi])
        assert (np.abs(got - want) <= bound).all(), (e, np.abs(got - want).max(), bound.max())
        tight.append((bound / (np.abs(want).mean() + 1e-30)).ravel() if want.any() else np.zeros(0))
    # (of the test itself: over all experts the ties are few, and the bound stays near the output's own rounding)
    assert np.median(np.concatenate(tight)) < max(0.02, 4 * HALF_STEP[out_dtype])


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("counts,h,F,T", [
    ([1], 64, 64, None), ([0, 3, 1], 128, 96, 2), ([130, 1, 0, 40], 256, 200, None), ([64, 64], 520, 33, 40),
    ([1] * 24, 512, 448, 3), ([257], 320, 1024, 100)])
def test_expert_ffn(gpu_lib, fmt, counts, h, F, T):
    check_ffn(gpu_lib, counts, h, F, fmt, "bf16", T=T)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("K", [1024, 1100, 1350])
def test_linear_of_rows_used_many_times(gpu_lib, fmt, K):
    """Rows that src names several times are quantised once and copied: the same values, pads and a group of one row."""
    g = torch.Generator().manual_seed(K)
    src = torch.randint(-1, 600, (4500,), generator=g, dtype=torch.int32).cuda()
    check_linear(gpu_lib, [1, 0, 3000, 1499], 96, K, fmt, "bf16", src=src, x_rows=600, gscale=torch.tensor([4.0], device="cuda"))


@pytest.mark.parametrize("fmt", ["nv", "mx"])
def test_expert_ffn_of_many_tiles(gpu_lib, fmt):
    check_ffn(gpu_lib, [1000, 1620], 128, 2080, fmt, "bf16", T=900)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("dtype,out_dtype", [("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_expert_ffn_types_and_multipliers(gpu_lib, fmt, dtype, out_dtype):
    check_ffn(gpu_lib, [17, 0, 150], 192, 160, fmt, dtype, out_dtype, scaled=True, T=60)


@pytest.mark.parametrize("fmt", ["nv", "mx"])
@pytest.mark.parametrize("F", [64, 40])
def test_expert_ffn_far_gates(gpu_lib, fmt, F):
    """Gates g far from 0 and infinite, and the activations one by one: an expert a magnitude of g, made by its alpha, a row a
    sign; u of many magnitudes; the down weights give each activation's 4-bit value back, times a number that the format
    holds. silu(inf) u is infinite and ends at the largest code, silu(-inf) is NaN as in the formula, and what is left of
    silu(g) at a very negative g is as small as it is: an MX scale follows it down to 2^-127.

    Bound of act: 2^-18 of it, and fp32's last places below the normal range: exp(-|g|) and its product with g within 2^-149
    each, the former times |g|, all times |u|, and act's own. Codes as the definition gives for an act within its bound."""
    moe = gpu_lib
    mags = [0.0, 1.0, 20.0, 47.9, 48.1, 63.0, 63.99, 64.01, 70.0, 75.0, 80.0, 86.0, 87.5, 89.0, 95.0, 110.0, 1e4, 1e10, 1e25, 1e35, 3e38, np.inf]
    E, h = len(mags), 64
    x = torch.zeros((2 * E, h), dtype=torch.float64)
    x[0::2, 0], x[1::2, 0], x[:, 32] = 6.0, -6.0, 6.0
    wg, wu, wd = torch.zeros(E, F, h), torch.zeros(E, F, h), torch.zeros(E, h, F)
    wg[:, :, 0] = torch.where(torch.arange(F) % 7 == 0, 0.0, 6.0)
    wu[:, :, 32] = 6.0 * 2.0 ** (torch.arange(F) % 12 - 6) * (1 - 2 * (torch.arange(F) % 2))
    back = np.array([6.0 if fmt == "nv" else 6.0 * (2.0**-40 if m > 1e9 else 2.0**40 if m > 60 else 1.0) for m in mags])
    wd[:, torch.arange(F), torch.arange(F)] = torch.from_numpy(back).float()[:, None]
    mats = []
    for w in (wg, wu, wd):
        c, s = moe.moe_fp4_quantize(w.reshape(-1, w.shape[2]).cuda(), fmt)
        held = Q.dequantize(Q.unpack_codes(c.cpu().numpy(), w.shape[2]), s.cpu().numpy(), fmt)
        np.testing.assert_array_equal(held, w.double().reshape(-1, w.shape[2]).numpy())
        mats.append((c.view(*w.shape[:2], -1), s.view(*w.shape[:2], -1)))
    packed = moe.moe_fp4_pack_expert_weights(*mats, h, F, fmt)
    alpha = np.array([np.float32(3e38 if np.isinf(m) else m / 36) for m in mags], np.float32)
    off = torch.arange(0, 2 * E + 1, 2, dtype=torch.int32, device="cuda")
    y = moe.moe_fp4_expert_ffn(x.bfloat16().cuda(), off, packed, F, fmt, alpha_gate=torch.from_numpy(alpha).cuda(),
                               out_dtype=torch.float32)
    ok(moe)
    got = f64(y)
    for r in range(2 * E):
        e = r // 2
        with np.errstate(over="ignore"):
            g = np.float64(np.float32(float(x[r, 0]) * wg[e, :, 0].double().numpy() * np.float64(alpha[e])))
        u = 6.0 * wu[e, :, 32].double().numpy()
        if (g == -np.inf).any():
            assert np.isnan(got[r]).all()
            continue
        n = np.minimum(g, 0.0)
        act = np.where(g < 0, n * np.exp(n) / (1 + np.exp(n)), g / (1 + np.exp(-np.maximum(g, 0.0)))) * u
        act = np.where(np.abs(act) > np.finfo(np.float32).max, np.copysign(np.inf, act), act)
        fin = np.where(np.isfinite(act), act, 0.0)
        err = 2.0**-18 * np.abs(fin) + np.where(np.isfinite(g), (2 * np.minimum(np.abs(g), 110.0) + 1) * np.abs(u) + 1, 0) * 2.0**-149
        q, dq = Q.requantized(act[None], err[None], fmt)
        assert (np.abs(got[r, :F] - q[0] * back[e]) <= dq[0] * back[e]).all(), (mags[e], r, got[r, :F] / back[e], q[0])
        assert (got[r, F:] == 0).all()


def test_expert_ffn_is_deterministic_and_captures(gpu_lib):
    """The same bits on every call, on another stream and from a captured graph."""
    moe = gpu_lib
    E, h, F, rows = 8, 256, 256, 600
    mats = [weight(moe, E, n, k, "nv", 20 + i)[:2] for i, (n, k) in enumerate(((F, h), (F, h), (h, F)))]
    packed = moe.moe_fp4_pack_expert_weights(*mats, h, F, "nv")
    x = data((rows, h), "bf16", 6)
    off = torch.arange(0, rows + 1, rows // E, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_fp4_expert_ffn_workspace_size(E, h, F, rows, "nv"), dtype=torch.uint8, device="cuda")
    y0 = moe.moe_fp4_expert_ffn(x, off, packed, F, "nv", ws=ws).clone()
    ws.random_(0, 256)                                   # nothing in the workspace outlives a call
    y1 = moe.moe_fp4_expert_ffn(x, off, packed, F, "nv", ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = torch.empty_like(y0)
    moe.moe_fp4_expert_ffn(x, off, packed, F, "nv", ws=ws, out=y2, stream=side)
    torch.cuda.synchronize()
    y3 = torch.empty_like(y0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_fp4_expert_ffn(x, off, packed, F, "nv", ws=ws, out=y3)
    graph.replay()
    graph.replay()
    ok(moe)
    assert torch.equal(y0, y1) and torch.equal(y0, y2) and torch.equal(y0, y3)


def test_codes_of_another_shape_are_refused(gpu_lib):
    """A weight's codes [G, N, pitch] are no rows to bring back, and experts of another F or h are no experts of these."""
    moe = gpu_lib
    E, h, F = 2, 64, 96
    mats = [weight(moe, E, n, k, "nv", 50 + i)[:2] for i, (n, k) in enumerate(((F, h), (F, h), (h, F)))]
    with pytest.raises(moe.MoEError):
        moe.moe_fp4_dequantize(*mats[0], h, "nv")
    assert moe.moe_fp4_dequantize(*(t.flatten(0, 1) for t in mats[0]), h, "nv").shape == (E * F, h)
    for bad_h, bad_F in ((h, 64), (32, F), (F, h)):
        with pytest.raises(moe.MoEError):
            moe.moe_fp4_pack_expert_weights(*mats, bad_h, bad_F, "nv")
    ok(moe)


def test_what_a_call_allocates_is_its_streams(gpu_lib, monkeypatch):
    """Outputs and workspaces that the calls allocate come from the pool of the stream that they launch on (a workspace of the
    current stream's would be handed out again while the kernels use it); results as on the current stream."""
    moe = gpu_lib
    E, h, F, rows = 3, 128, 96, 70
    mats = [weight(moe, E, n, k, "nv", 40 + i)[:2] for i, (n, k) in enumerate(((F, h), (F, h), (h, F)))]
    x = data((rows, h), "bf16", 6)
    off = torch.tensor([0, 10, 10, rows], dtype=torch.int32, device="cuda")
    real, seen = torch.empty, []

    def empty(*a, **k):
        seen.append(torch.cuda.current_stream())
        return real(*a, **k)

    def calls(stream):
        codes, scales = moe.moe_fp4_quantize(x, "nv", stream=stream)
        back = moe.moe_fp4_dequantize(codes, scales, h, "nv", stream=stream)
        linear = moe.moe_fp4_linear(x, off, moe.moe_fp4_pack_weight(*mats[0], h, "nv", stream=stream), F, "nv", stream=stream)
        packed = moe.moe_fp4_pack_expert_weights(*mats, h, F, "nv", stream=stream)
        return codes, scales, back, linear, packed, moe.moe_fp4_expert_ffn(x, off, packed, F, "nv", stream=stream)

    want = [t.clone() for t in calls(None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    monkeypatch.setattr(torch, "empty", empty)
    got = calls(side)
    monkeypatch.undo()
    ok(moe)
    assert len(seen) == 9 and all(s == side for s in seen)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------------------- layer


@pytest.mark.parametrize("experts,name,over", [
    ("nvfp4", "page3_cf1.25", dict(T=700, h=256, F=192)),            # capacity, drops and pad rows
    ("mxfp4", "deepseek_v3", dict(T=300, h=256, F=128, E=32, k=4)),  # shared expert, groups of few rows
    ("nvfp4", "page3_expert_choice", dict(T=512, h=256, F=128)),
    ("mxfp4", "mixtral_sinkhorn", dict(T=512, h=256, F=192, bias="none"))])
def test_layer_with_experts_in_4_bits(gpu_lib, experts, name, over):
    """MoELayer(experts=...) against the float64 layer on the quantised weights and rows: normwise 2e-2, as the bf16 layer's
    outputs; and the same bits from a captured graph."""
    import moe_inputs
    from oracle import moe_oracle as O
    from tests import cases
    from top_routing_dispatch_moe_gb300.layer import MoELayer
    cfg = moe_inputs.get_config(name, **over)
    inp = cases.ec_inputs(cfg) if cfg.routing == "expert_choice" else cases.router_inputs(cfg)
    dev = torch.device("cuda")
    up = lambda a: cases.to_device(a, cfg, dev)   # noqa: E731
    ws = [up(w) for w in moe_inputs.all_expert_weights(cfg)]
    sh = [up(np.ascontiguousarray(w[0])[None]) for w in moe_inputs.all_expert_weights(cfg, shared=True)] if cfg.n_shared else None
    gs, ags = torch.tensor([64.0], device=dev), torch.tensor([256.0], device=dev)
    fmt = experts[:2]
    if fmt == "mx":
        gs = ags = None
    layer = MoELayer(T=cfg.T, h=cfg.h, E=cfg.E, k=cfg.k, F=cfg.F, gating=cfg.gating, cf=cfg.cf, R=cfg.R, alpha=cfg.alpha,
                     w_r=up(inp["w_r"]), bias=torch.from_numpy(inp["bias"]).to(dev) if inp["bias"] is not None else None,
                     w_gate=ws[0], w_up=ws[1], w_down=ws[2], shared=sh, device=dev, routing=cfg.routing, experts=experts,
                     fp4_gscale=gs, fp4_act_gscale=ags)
    x = up(inp["x"])
    y = layer.forward(x).clone()
    ok(gpu_lib)

    def quantised(w):                                    # [n, k] -> the values it is held as
        m = 2.0 ** np.floor(np.log2(448.0 * 6.0 / np.abs(w).max())) if fmt == "nv" else 1.0
        return Q.dequantize(*Q.quantize(w * m, fmt), fmt) / m

    def through(v, m):
        m = float(m) if m is not None else 1.0
        return Q.dequantize(*Q.quantize(v * m, fmt), fmt) / m

    def ffn(rows, w):
        g, u = (through(rows, gs) @ quantised(t).T for t in w[:2])
        return through(g / (1 + np.exp(-g)) * u, ags) @ quantised(w[2]).T

    x64 = f64(x)
    w64 = [f64(w) for w in ws]
    if cfg.routing == "expert_choice":
        tokens = layer.ec["tokens"].cpu().numpy()
        gates = layer.ec["gates"].double().cpu().numpy()
        want = np.zeros_like(x64)
        for e in range(cfg.E):
            want[tokens[e]] += gates[e][:, None] * ffn(x64[tokens[e]], [w[e] for w in w64])
    else:
        want = np.zeros_like(x64) if sh is None else ffn(x64, [f64(w[0]) for w in sh])
        ids, gates = layer.r_out["topk_ids"].cpu().numpy(), layer.r_out["gates"].double().cpu().numpy()
        kept = layer.d_out["drop_mask"].cpu().numpy() == 0
        np.testing.assert_array_equal(ids, inp["route"]["ids"])
        for e in range(cfg.E):
            t, j = np.nonzero((ids == e) & kept)
            if len(t):
                want[t] += gates[t, j][:, None] * ffn(x64[t], [w[e] for w in w64])
    assert cases.rel_l2(f64(y), want) <= 2e-2
    graph = layer.capture_forward(x)
    layer.y.zero_()
    graph.replay()
    ok(gpu_lib)
    assert torch.equal(layer.y, y)
    x.mul_(0.5)                                          # other rows, other routes: the graph reads x where it is
    y = layer.forward(x).clone()
    layer.y.zero_()
    graph.replay()
    ok(gpu_lib)
    assert torch.equal(layer.y, y)
    with pytest.raises(NotImplementedError):
        layer.native_desc()
    with pytest.raises(RuntimeError):
        layer.backward(x, y)


def test_a_layers_multipliers_are_its_own(gpu_lib):
    """The tensors given for fp4_gscale and fp4_act_gscale may change after construction: the layer computes as it was made, call
    by call and from a graph."""
    from top_routing_dispatch_moe_gb300.layer import MoELayer
    T, h, E, F = 64, 128, 4, 96
    gs, ags = torch.tensor([64.0], device="cuda"), torch.tensor([256.0], device="cuda")
    layer = MoELayer(T=T, h=h, E=E, k=2, F=F, gating="softmax_renorm", cf=0.0, R=1, alpha=0.0,
                     w_r=data((h, E), "bf16", 1, 0.1), bias=None,
                     w_gate=data((E, F, h), "bf16", 2, 0.1), w_up=data((E, F, h), "bf16", 3, 0.1), w_down=data((E, h, F), "bf16", 4, 0.1),
                     experts="nvfp4", fp4_gscale=gs, fp4_act_gscale=ags)
    x = data((T, h), "bf16", 5)
    want = layer.forward(x).clone()
    graph = layer.capture_forward(x)
    gs.mul_(4)
    ags.mul_(0.5)
    assert torch.equal(layer.forward(x), want)
    layer.y.zero_()
    graph.replay()
    ok(gpu_lib)
    assert torch.equal(layer.y, want)
