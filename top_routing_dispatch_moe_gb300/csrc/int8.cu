// Rows to 8-bit integers under one scale a row and back, and the packing of 8-bit weights.
//
// Both directions are bound by memory: x is read once and one byte a value written (two as fp16 operand), or the other way
// round. A row is held in registers by one to eight warps between its largest magnitude and its codes; rows past 16384
// columns are read twice.
#include <algorithm>
#include "int8.cuh"

namespace moe {
namespace int8 {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int SEG = 32 * UNIT;       // columns a warp takes at a time
constexpr int HELD = 4;              // such pieces that a warp holds

// How a row lies: its 16-column units on 16 bytes in x and in the codes (WHOLE), both after `skip` columns of a contiguous matrix's row
// before (FLAT: the unit that holds the row's start, and its last, are the neighbours' too), or on no boundary (ANY).
enum Lie { WHOLE, FLAT, ANY };

// Piece `c` of a row: WHOLE, FLAT: this lane's 16 consecutive columns; ANY: every 32nd column from the lane's own, so that loads and stores
// of a warp stay together.
template <typename T, Lie LIE>
__device__ __forceinline__ Raw16<T> load_piece(const T* row, int c, int K, int skip, bool again) {
    const int lane = threadIdx.x & 31, k0 = c * SEG + lane * UNIT - skip;
    if constexpr (LIE == WHOLE) return load_unit<T, true>(row, k0, K, again);
    Raw16<T> r;
    T* e = reinterpret_cast<T*>(r.q);
    if constexpr (LIE == FLAT) {
        if (k0 >= 0 && k0 + UNIT <= K) return load_unit<T, true>(row, k0, K, again);
#pragma unroll
        for (int j = 0; j < UNIT; ++j) e[j] = k0 + j >= 0 && k0 + j < K ? row[k0 + j] : T(0.f);
    } else {
#pragma unroll
        for (int j = 0; j < UNIT; ++j) {
            const int k = c * SEG + j * 32 + lane;
            e[j] = k < K ? row[k] : T(0.f);
        }
    }
    return r;
}
template <typename T, int FORM, Lie LIE>
__device__ __forceinline__ void store_piece(const Raw16<T>& raw, void* codes, size_t base, int c, int width, int skip, const Steps& st) {
    const int lane = threadIdx.x & 31;
    const T* e = reinterpret_cast<const T*>(raw.q);
    float v[UNIT];
#pragma unroll
    for (int i = 0; i < UNIT; ++i) v[i] = as_f32(e[i]);
    codes_of<T, UNIT>(v, st);
    if constexpr (LIE != ANY) {
        const int k = c * SEG + lane * UNIT - skip;
        if (k >= width) return;
        if constexpr (FORM == FORM_F16) {
            uint4 w[2];
            __half2* h = reinterpret_cast<__half2*>(w);
#pragma unroll
            for (int i = 0; i < UNIT / 2; ++i) h[i] = halves2(v + 2 * i);
            st32(static_cast<__half*>(codes) + base + k, w);
        } else if (LIE == WHOLE || (k >= 0 && k + UNIT <= width)) {
            *reinterpret_cast<uint4*>(static_cast<int8_t*>(codes) + base + k) =
                make_uint4(bytes4(v), bytes4(v + 4), bytes4(v + 8), bytes4(v + 12));
        } else {
#pragma unroll
            for (int j = 0; j < UNIT; ++j)
                if (k + j >= 0 && k + j < width) static_cast<uint8_t*>(codes)[base + k + j] = (uint8_t)__float_as_uint(v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < UNIT; ++j) {
            const int k = c * SEG + j * 32 + lane;
            if (k >= width) continue;
            if constexpr (FORM == FORM_F16) static_cast<__half*>(codes)[base + k] = __float2half_rn(v[j] - MAGIC);
            else static_cast<uint8_t*>(codes)[base + k] = (uint8_t)__float_as_uint(v[j]);
        }
    }
}

// WPR warps to a row.
template <typename T, int FORM, int WPR, Lie LIE>
__global__ void __launch_bounds__(THREADS)
quantize_kernel(const T* x, long long ldx, int x_rows, const int32_t* src, int rows, int K, int width, void* codes, float* scales,
                unsigned* err) {
    __shared__ float s_amax[WARPS];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % WPR;
    const int row = blockIdx.x * (WARPS / WPR) + warp / WPR;
    int from = row < rows ? row : -1;
    if (from >= 0 && src) {
        from = src[row];
        if (from >= x_rows || from < -1) {
            if (lane == 0) latch_device_error(err, kDevErrBadIndex, 0x310u);
            from = -1;
        }
    }
    const T* xr = x + (long long)max(from, 0) * ldx;
    const int k_in = from >= 0 ? K : 0, skip = LIE == FLAT ? (row & 15) * (K & 15) & 15 : 0,
              pieces = (width + skip + SEG - 1) / SEG;
    const bool held = pieces <= HELD * WPR, again = src != nullptr;
    Raw16<T> raw[HELD];
    float amax = 0.f;
    if (held) {
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (i * WPR + w < pieces) raw[i] = load_piece<T, LIE>(xr, i * WPR + w, k_in, skip, again);
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (i * WPR + w < pieces) amax = max_nan(amax, unit_amax(raw[i]));
    } else {
        for (int c = w; c < pieces; c += WPR) amax = max_nan(amax, unit_amax(load_piece<T, LIE>(xr, c, k_in, skip, again)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if constexpr (WPR > 1) {
        if (lane == 0) s_amax[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WPR; ++i) amax = max_nan(amax, s_amax[warp - w + i]);
    }
    if (row >= rows) return;
    Steps st;
    const float scale = scale_of<T>(amax, st);
    if (w == 0 && lane == 0) scales[row] = scale;
    const size_t base = (size_t)row * width;
    if (held) {
#pragma unroll
        for (int i = 0; i < HELD; ++i)
            if (i * WPR + w < pieces) store_piece<T, FORM, LIE>(raw[i], codes, base, i * WPR + w, width, skip, st);
    } else {
        for (int c = w; c < pieces; c += WPR)
            store_piece<T, FORM, LIE>(load_piece<T, LIE>(xr, c, k_in, skip, again), codes, base, c, width, skip, st);
    }
}

// Rows of up to 256 columns: 1, 2, 4, 8 or 16 lanes (1 << lanes_log) to a row. (65536 x 96 bf16 4.5 us,
// x 256 8.4; by a warp a row 17.6 and 20.)
template <typename T, int FORM>
__global__ void __launch_bounds__(THREADS)
quantize_short_kernel(const T* x, long long ldx, int x_rows, const int32_t* src, int rows, int K, int width, int lanes_log, void* codes,
                      float* scales, unsigned* err) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, in_row = lane & ((1 << lanes_log) - 1), skip = (lane - in_row) * UNIT;
    const int row = (int)(blockIdx.x * (THREADS >> lanes_log) + (threadIdx.x >> lanes_log));
    int from = row < rows ? row : -1;
    if (from >= 0 && src) {
        from = src[row];
        if (from >= x_rows || from < -1) {
            if (in_row == 0) latch_device_error(err, kDevErrBadIndex, 0x310u);
            from = -1;
        }
    }
    const Raw16<T> raw = load_piece<T, WHOLE>(x + (long long)max(from, 0) * ldx, 0, from >= 0 ? K : 0, skip, src != nullptr);
    float amax = unit_amax(raw);
    for (int o = 1 << lanes_log >> 1; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (row >= rows) return;
    Steps st;
    const float scale = scale_of<T>(amax, st);
    if (in_row == 0) scales[row] = scale;
    store_piece<T, FORM, WHOLE>(raw, codes, (size_t)row * width, 0, width, skip, st);
}

// BLOCKS: a scale for 128 columns (a checkpoint) instead of one for a row.
template <typename T, bool VEC, bool BLOCKS>
__global__ void __launch_bounds__(THREADS)
dequantize_kernel(const int8_t* codes, const float* scales, int rows, int K, T* out, long long ldo) {
    pdl_wait();
    pdl_trigger();
    constexpr int U = VEC ? 4 : 1;       // pieces whose codes a lane has under way
    const int lane = threadIdx.x & 31, nseg = (K + SEG - 1) / SEG;
    auto scale = [&](int row, int k) { return scales[BLOCKS ? (size_t)row * ((K + CKPT - 1) / CKPT) + k / CKPT : row]; };
    Walk at((long long)blockIdx.x * WARPS + (threadIdx.x >> 5), (long long)gridDim.x * WARPS, (long long)rows * nseg, nseg);
    while (at.left > 0) {
        if constexpr (VEC) {
            uint4 q[U];
            float s[U];
            T* to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = at.seg * SEG + lane * UNIT;
                to[u] = nullptr;
                if (at.left > 0 && k < K) {
                    q[u] = __ldcs(reinterpret_cast<const uint4*>(codes + (size_t)at.row * K + k));
                    s[u] = scale(at.row, k);
                    to[u] = out + at.row * ldo + k;
                }
                if (at.left > 0) at.next();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!to[u]) continue;
                float v[UNIT];
                values4(q[u].x, s[u], v);
                values4(q[u].y, s[u], v + 4);
                values4(q[u].z, s[u], v + 8);
                values4(q[u].w, s[u], v + 12);
                alignas(16) T o[UNIT];
#pragma unroll
                for (int i = 0; i < UNIT; ++i) o[i] = rounded<T>(v[i]);
                const uint4* ov = reinterpret_cast<const uint4*>(o);
                if ((reinterpret_cast<uintptr_t>(to[u]) & 31u) == 0) {
#pragma unroll
                    for (int i = 0; i < (int)sizeof(T); i += 2) st32(reinterpret_cast<uint4*>(to[u]) + i, ov + i);
                } else {
#pragma unroll
                    for (int i = 0; i < (int)sizeof(T); ++i) reinterpret_cast<uint4*>(to[u])[i] = ov[i];
                }
            }
        } else {
            const int8_t* cr = codes + (size_t)at.row * K;
            T* orow = out + at.row * ldo;
#pragma unroll
            for (int j = 0; j < UNIT; ++j) {
                const int k = at.seg * SEG + j * 32 + lane;
                if (k < K) orow[k] = rounded<T>((float)cr[k] * scale(at.row, k));
            }
            at.next();
        }
    }
}

// Contiguous rows of any width from 16 on (a scale a row): 16 elements a lane across the rows' ends, two scales at most. For widths that are
// no whole units, and for short rows.
template <typename T>
__global__ void __launch_bounds__(THREADS)
dequantize_flat_kernel(const int8_t* codes, const float* scales, long long total, int K, T* out) {
    pdl_wait();
    pdl_trigger();
    constexpr int U = 2;                 // units whose codes a lane has under way
    const long long units = (total + UNIT - 1) / UNIT, step = (long long)gridDim.x * THREADS;
    const bool small = total < (1LL << 31);
    for (long long i = (long long)blockIdx.x * THREADS + threadIdx.x; i < units; i += U * step) {
        uint4 q[U];
        float s0[U], s1[U];
        int here[U];                     // elements of the first row
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long at = (i + u * step) * UNIT;
            here[u] = 0;
            if (at + UNIT > total) continue;
            const long long row = small ? (long long)((unsigned)at / (unsigned)K) : at / K;
            here[u] = (int)min((row + 1) * K - at, (long long)UNIT);
            q[u] = __ldcs(reinterpret_cast<const uint4*>(codes + at));
            s0[u] = scales[row];
            s1[u] = here[u] < UNIT ? scales[row + 1] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (here[u] == 0) continue;
            T* to = out + (i + u * step) * UNIT;
            float v[UNIT];
            values4(q[u].x, 1.f, v);
            values4(q[u].y, 1.f, v + 4);
            values4(q[u].z, 1.f, v + 8);
            values4(q[u].w, 1.f, v + 12);
            alignas(16) T o[UNIT];
#pragma unroll
            for (int j = 0; j < UNIT; ++j) o[j] = rounded<T>(v[j] * (j < here[u] ? s0[u] : s1[u]));
            const uint4* ov = reinterpret_cast<const uint4*>(o);
            if ((reinterpret_cast<uintptr_t>(to) & 31u) == 0) {
#pragma unroll
                for (int j = 0; j < (int)sizeof(T); j += 2) st32(reinterpret_cast<uint4*>(to) + j, ov + j);
            } else {
#pragma unroll
                for (int j = 0; j < (int)sizeof(T); ++j) reinterpret_cast<uint4*>(to)[j] = ov[j];
            }
        }
    }
    // the last elements, less than a unit (all of the last row)
    const long long at = total / UNIT * UNIT + threadIdx.x;
    if (blockIdx.x == 0 && at < total) out[at] = rounded<T>((float)codes[at] * scales[at / K]);
}

// A 16-byte chunk of the packed weight a thread. b: null, or the rows that follow those of a in turn (gate, up).
__global__ void __launch_bounds__(THREADS)
pack_kernel(const int8_t* __restrict__ a, const int8_t* __restrict__ b, int N, int K, int NB, int KST, size_t chunks, uint4* __restrict__ out) {
    for (size_t i = (size_t)blockIdx.x * THREADS + threadIdx.x; i < chunks; i += (size_t)gridDim.x * THREADS) {
        const int c = (int)(i >> 7 & 3), r = (int)(i & 127) ^ (2 * c);
        const size_t piece = i >> 9, at = piece / KST;
        const int k0 = (int)(piece - at * KST) * STAGE_K + c * UNIT, nb = (int)(at % NB);
        const size_t g = at / NB;
        const int n = nb * BLOCK_N + r, rows = b ? N / 2 : N;      // rows of each source
        const int8_t* src = (b && (n & 1)) ? b : a;
        const size_t row = g * rows + (b ? n >> 1 : n);
        alignas(16) uint8_t v[UNIT];
#pragma unroll
        for (int j = 0; j < UNIT; ++j) v[j] = n < N && k0 + j < K ? (uint8_t)(src[row * K + k0 + j] + 128) : (uint8_t)128;
        out[i] = *reinterpret_cast<const uint4*>(v);
    }
}

static int launch_pack(const void* a, const void* b, int G, int N, int K, void* out, cudaStream_t s) {
    const WeightLayout L = weight_layout(G, N, K);
    const size_t chunks = L.total / 16;
    const int grid = (int)std::min<size_t>((chunks + THREADS - 1) / THREADS, (size_t)num_sms() * 16);
    pack_kernel<<<grid, THREADS, 0, s>>>(static_cast<const int8_t*>(a), static_cast<const int8_t*>(b), N, K, L.NB, L.KST, chunks,
                                         static_cast<uint4*>(out));
    return check_launch("int8 pack_kernel");
}

template <typename T, int FORM>
static cudaError_t quantize_form(const void* x, long long ldx, int x_rows, const int32_t* src, int rows, int K, void* codes, float* scales,
                                 unsigned* err, cudaStream_t s) {
    const int width = FORM == FORM_ROWS ? K : pad64(K);
    const T* xt = static_cast<const T*>(x);
    // whole 16-byte pieces of x's rows and of the codes' (the operand's rows are padded: any K)
    const bool aligned = aligned16(x) && aligned16(codes), vec = width % UNIT == 0 && aligned && ldx * (long long)sizeof(T) % 16 == 0;
    auto go = [&](auto kernel, int wpr) {
        return launch_pdl(kernel, dim3(cdiv(rows, WARPS / wpr)), dim3(THREADS), 0, s, xt, ldx, x_rows, src, rows, K, width, codes, scales, err);
    };
    // a row's warps: as many as hold it four pieces each (16384 x 3001 fp32, six pieces, by eight warps instead of two 110 us, not 60)
    const int pieces = (width + SEG - 1) / SEG;
    if (vec && width <= SEG / 2) {
        int lanes_log = 0;
        while (UNIT << lanes_log < width) ++lanes_log;
        return launch_pdl(quantize_short_kernel<T, FORM>, dim3(cdiv(rows, THREADS >> lanes_log)), dim3(THREADS), 0, s, xt, ldx, x_rows, src, rows,
                          K, width, lanes_log, codes, scales, err);
    }
    if (vec) {
        if (pieces <= HELD) return go(quantize_kernel<T, FORM, 1, WHOLE>, 1);
        if (pieces <= 2 * HELD) return go(quantize_kernel<T, FORM, 2, WHOLE>, 2);
        if (pieces <= 4 * HELD) return go(quantize_kernel<T, FORM, 4, WHOLE>, 4);
        return go(quantize_kernel<T, FORM, 8, WHOLE>, 8);
    }
    // contiguous rows of other widths, of 16-bit types (65536 x 999 fp16 69 -> 52 us, x 1500 bf16 90 -> 62; fp32, whose lanes already load
    // whole sectors, 74 -> 88)
    if constexpr (FORM == FORM_ROWS && sizeof(T) == 2)
        if (aligned && !src && ldx == K && K >= 2 * UNIT) {
            const int most = (K + UNIT - 1 + SEG - 1) / SEG;
            if (most <= HELD) return go(quantize_kernel<T, FORM, 1, FLAT>, 1);
            if (most <= 2 * HELD) return go(quantize_kernel<T, FORM, 2, FLAT>, 2);
            if (most <= 4 * HELD) return go(quantize_kernel<T, FORM, 4, FLAT>, 4);
            return go(quantize_kernel<T, FORM, 8, FLAT>, 8);
        }
    if (pieces <= HELD) return go(quantize_kernel<T, FORM, 1, ANY>, 1);
    if (pieces <= 2 * HELD) return go(quantize_kernel<T, FORM, 2, ANY>, 2);
    if (pieces <= 4 * HELD) return go(quantize_kernel<T, FORM, 4, ANY>, 4);
    return go(quantize_kernel<T, FORM, 8, ANY>, 8);
}

int launch_quantize(const void* x, long long ldx, int x_rows, const int32_t* src, int rows, int K, int dtype, int form, void* codes,
                    float* scales, unsigned* err, cudaStream_t s) {
    if (rows == 0) return MOE_OK;
    cudaError_t e = cudaErrorInvalidValue;
#define MOE_QUANT(T)                                                                                                       \
    e = form == FORM_ROWS ? quantize_form<T, FORM_ROWS>(x, ldx, x_rows, src, rows, K, codes, scales, err, s)               \
                          : quantize_form<T, FORM_F16>(x, ldx, x_rows, src, rows, K, codes, scales, err, s)
    if (dtype == MOE_F32) MOE_QUANT(float);
    else if (dtype == MOE_BF16) MOE_QUANT(__nv_bfloat16);
    else MOE_QUANT(__half);
#undef MOE_QUANT
    return check_launch(e, "int8 quantize_kernel");
}

template <typename T, bool VEC>
static cudaError_t dequantize_form(const void* codes, const float* scales, int rows, int K, void* out, long long ldo, bool blocks, cudaStream_t s) {
    const long long items = (long long)rows * cdiv(K, SEG);
    const int grid = (int)std::min<long long>((items + WARPS - 1) / WARPS, 8LL * num_sms());
    auto go = [&](auto kernel) {
        return launch_pdl(kernel, dim3(grid), dim3(THREADS), 0, s, static_cast<const int8_t*>(codes), scales, rows, K, static_cast<T*>(out), ldo);
    };
    return blocks ? go(dequantize_kernel<T, VEC, true>) : go(dequantize_kernel<T, VEC, false>);
}

// (4099 x 999 fp16 5.4 -> 3.1 us, 65536 x 999 fp16 69 -> 33, fp32 73 -> 54: before, a lane took every 32nd column; 65536 x 96 bf16 9.0 -> 4.1:
// before, a warp took a row.)
template <typename T>
static cudaError_t dequantize_flat(const void* codes, const float* scales, int rows, int K, void* out, cudaStream_t s) {
    const long long total = (long long)rows * K, units = (total + UNIT - 1) / UNIT;
    const int grid = (int)std::min<long long>((units + 2 * THREADS - 1) / (2 * THREADS), 8LL * num_sms());
    return launch_pdl(dequantize_flat_kernel<T>, dim3(grid), dim3(THREADS), 0, s, static_cast<const int8_t*>(codes), scales, total, K,
                      static_cast<T*>(out));
}

int launch_dequantize(const void* codes, const float* scales, int rows, int K, int dtype, void* out, long long ldo, bool blocks, cudaStream_t s) {
    const bool flat = !blocks && (K % UNIT != 0 || K <= SEG / 2) && K >= UNIT && ldo == K && aligned16(codes) && aligned16(out);
    const bool vec = K % UNIT == 0 && aligned16(codes) && aligned16(out) && ldo * (dtype == MOE_F32 ? 4 : 2) % 16 == 0;
    cudaError_t e = cudaErrorInvalidValue;
#define MOE_DEQUANT(T)                                                                     \
    e = flat  ? dequantize_flat<T>(codes, scales, rows, K, out, s)                         \
        : vec ? dequantize_form<T, true>(codes, scales, rows, K, out, ldo, blocks, s)      \
              : dequantize_form<T, false>(codes, scales, rows, K, out, ldo, blocks, s)
    if (dtype == MOE_F32) MOE_DEQUANT(float);
    else if (dtype == MOE_BF16) MOE_DEQUANT(__nv_bfloat16);
    else MOE_DEQUANT(__half);
#undef MOE_DEQUANT
    return check_launch(e, "int8 dequantize_kernel");
}

static bool known(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }
static bool type_aligned(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (dtype == MOE_F32 ? 4 : 2) == 0; }

}  // namespace int8
}  // namespace moe

using namespace moe;

extern "C" int moe_int8_quantize(const void* x, long long ldx, int x_rows, const int32_t* src, int rows, int K, int dtype, void* codes,
                                 float* scales, void* stream) {
    const char* fn = "moe_int8_quantize";
    MOE_REQUIRE(int8::known(dtype), MOE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    MOE_REQUIRE(rows >= 0 && rows <= MOE_INT8_MAX_ROWS && K >= 1 && K <= MOE_INT8_MAX_K && ldx >= K && x_rows >= (src ? 0 : rows),
                MOE_ERR_INVALID_ARG, "%s: rows=%d x_rows=%d K=%d ldx=%lld", fn, rows, x_rows, K, ldx);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE((x || x_rows == 0) && codes && scales, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    MOE_REQUIRE(int8::type_aligned(x, dtype) && int8::type_aligned(scales, MOE_F32) && int8::type_aligned(src, MOE_F32), MOE_ERR_INVALID_ARG,
                "%s: misaligned pointer", fn);
    unsigned* err = device_error_word();
    MOE_REQUIRE(err, MOE_ERR_CUDA, "%s: device error word unavailable", fn);
    return int8::launch_quantize(x, ldx, x_rows, src, rows, K, dtype, int8::FORM_ROWS, codes, scales, err, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_int8_dequantize(const void* codes, const float* scales, int rows, int K, int dtype, void* out, long long ldo,
                                   void* stream) {
    const char* fn = "moe_int8_dequantize";
    MOE_REQUIRE(int8::known(dtype), MOE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    MOE_REQUIRE(rows >= 0 && rows <= MOE_INT8_MAX_ROWS && K >= 1 && K <= MOE_INT8_MAX_K && ldo >= K, MOE_ERR_INVALID_ARG,
                "%s: rows=%d K=%d ldo=%lld", fn, rows, K, ldo);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(codes && scales && out, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    MOE_REQUIRE(int8::type_aligned(out, dtype) && int8::type_aligned(scales, MOE_F32), MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return int8::launch_dequantize(codes, scales, rows, K, dtype, out, ldo, false, static_cast<cudaStream_t>(stream));
}

static bool int8_sizes(int G, int N, int K) {
    return G >= 1 && G <= 1024 && N >= 1 && N <= MOE_INT8_MAX_K && K >= 1 && K <= MOE_INT8_MAX_K;
}

extern "C" size_t moe_int8_packed_weight_bytes(int G, int N, int K) { return int8_sizes(G, N, K) ? int8::weight_layout(G, N, K).total : 0; }

extern "C" int moe_int8_pack_weight(const void* codes, int G, int N, int K, void* packed, void* stream) {
    MOE_REQUIRE(int8_sizes(G, N, K), MOE_ERR_INVALID_ARG, "moe_int8_pack_weight: G=%d N=%d K=%d", G, N, K);
    MOE_REQUIRE(codes && packed && aligned16(packed), MOE_ERR_INVALID_ARG, "moe_int8_pack_weight: null or misaligned pointer");
    return int8::launch_pack(codes, nullptr, G, N, K, packed, static_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_int8_packed_expert_weights_bytes(int E, int h, int F) {
    return int8_sizes(E, h, F) && F <= MOE_INT8_MAX_K / 2 ? int8::expert_layout(E, h, F).total : 0;
}

extern "C" int moe_int8_pack_expert_weights(const void* gate, const void* up, const void* down, int E, int h, int F, void* packed,
                                            void* stream) {
    const char* fn = "moe_int8_pack_expert_weights";
    MOE_REQUIRE(int8_sizes(E, h, F) && F <= MOE_INT8_MAX_K / 2, MOE_ERR_INVALID_ARG, "%s: E=%d h=%d F=%d", fn, E, h, F);
    MOE_REQUIRE(gate && up && down && packed && aligned16(packed), MOE_ERR_INVALID_ARG, "%s: null or misaligned pointer", fn);
    const int8::ExpertLayout L = int8::expert_layout(E, h, F);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int rc = int8::launch_pack(gate, up, E, 2 * F, h, packed, s)) return rc;
    return int8::launch_pack(down, nullptr, E, h, F, static_cast<char*>(packed) + L.down_off, s);
}
