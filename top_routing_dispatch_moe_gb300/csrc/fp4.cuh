// Block-scaled 4-bit floating point (e2m1): formats, layouts and the arithmetic shared by the quantisation
// kernels and the product's epilogue.
//
// A value is code * scale of its block. e2m1 codes (sign, 2 exponent bits, 1 mantissa bit) stand for 0, 0.5, 1, 1.5,
// 2, 3, 4, 6; two codes to a byte, the even column in the low half.
//   MOE_FP4_NV: blocks of 16 columns, scale s = e4m3(amax / 6), held below 448 (rounded to nearest even);
//   MOE_FP4_MX: blocks of 32 columns, scale s = 2^(floor(log2 amax) - 2), stored as the exponent + 127.
#pragma once

#include <cuda_fp16.h>
#include "common.cuh"
#include "quant_io.cuh"

namespace moe {
namespace fp4 {

constexpr int SEG_K = 256;           // columns of a shared-memory stage of the product: 128 bytes of codes a row

struct Nv { static constexpr int ID = MOE_FP4_NV, BLK = 16; };
struct Mx { static constexpr int ID = MOE_FP4_MX, BLK = 32; };

// Bytes of block scales of 128 rows x SEG_K columns, in the tile layout: 512-byte pieces of 128 rows x 4 blocks,
// block b of row r of a piece at byte (r % 32) * 16 + (r / 32) * 4 + b: the order in which a piece lands in tensor
// memory as the scale operand of the block-scaled tcgen05.mma (lane r % 32, column r / 32, byte b).
template <class F> constexpr int SF_PIECES = SEG_K / F::BLK / 4;
template <class F> constexpr int SF_BYTES = SF_PIECES<F> * 512;
__host__ __device__ constexpr int sf_bytes(int fmt) { return fmt == MOE_FP4_NV ? 2048 : 1024; }
__host__ __device__ constexpr int block_of(int fmt) { return fmt == MOE_FP4_NV ? 16 : 32; }

inline int pad64(int k) { return (k + 63) / 64 * 64; }
inline int stages_of(int k) { return (k + SEG_K - 1) / SEG_K; }

// A packed weight [G][N][K]: codes [G][stage][N / 64 padded to pairs][64 rows x 128 bytes, the 16-byte chunk c of row r
// at chunk c ^ (r % 8): a K-major operand tile with 128-byte swizzling], zero past N and K; then, from the next
// 256-byte boundary, scales [G][stage][N / 128][SF_BYTES] in the tile layout. A stage's codes of any run of 64-row
// blocks are contiguous, and so are its scales: the product fetches each with one bulk copy.
struct WeightLayout {
    int NB64, NB128, KST;
    size_t sf_off, total;
};
inline WeightLayout weight_layout(int G, int N, int K, int fmt) {
    WeightLayout L;
    L.NB128 = (N + 127) / 128;
    L.NB64 = 2 * L.NB128;
    L.KST = stages_of(K);
    L.sf_off = (size_t)G * L.KST * L.NB64 * 8192;
    L.total = L.sf_off + (size_t)G * L.KST * L.NB128 * sf_bytes(fmt);
    return L;
}

// The expert FFN's packed weight: the gate/up matrix (N = 2 pad64(F): 32 gate rows, then the 32 up rows of the same f,
// and so on; K = h) and the down matrix (N = h, K = F) from the next 256-byte boundary.
struct ExpertLayout { WeightLayout gu, down; size_t down_off, total; };
inline ExpertLayout expert_layout(int E, int h, int F, int fmt) {
    ExpertLayout L;
    L.gu = weight_layout(E, 2 * pad64(F), h, fmt);
    L.down = weight_layout(E, h, F, fmt);
    L.down_off = align_up(L.gu.total, 256);
    L.total = L.down_off + L.down.total;
    return L;
}

// A quantised row operand of the product: codes [rows][pad64(K) / 2] and scales [tile of the schedule][stage][SF_BYTES].
inline size_t operand_codes_bytes(long long rows, int K) { return align_up((size_t)rows * (pad64(K) / 2), 1024); }
inline size_t operand_sf_bytes(long long rows, int G, int K, int fmt) {
    return align_up(sched_max_tiles(rows, G) * stages_of(K) * sf_bytes(fmt), 1024);
}

#ifdef __CUDACC__
// Eight values -> eight codes, to nearest, ties to even, held at +-6.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
    uint32_t h2;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "r"(byte));
    return __low2float(*reinterpret_cast<const __half2*>(&h2));
}
__device__ __forceinline__ uint32_t e4m3_byte(float v) {           // v >= 0 or NaN, held at 448
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %2, %1;\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(r) : "f"(v), "f"(0.f));
    return r & 0xFFu;
}

// The scale byte of a block whose largest magnitude is `amax` (NaN if one of its values is), the scale itself and its
// reciprocal (0 where the scale is 0 or NaN).
template <class F>
__device__ __forceinline__ uint32_t block_scale(float amax, float& s, float& r) {
    if constexpr (F::ID == MOE_FP4_NV) {
        // amax / 6, rounded (the correction of quotient2; past 1e30 the scale is at its ceiling either way)
        const float q = amax * (1.f / 6.f), d = fmaf(fmaf(-q, 6.f, amax), 1.f / 6.f, q);
        const uint32_t b = e4m3_byte(amax < 1e30f ? d : q);
        s = e4m3_value(b);
        r = s > 0.f ? __frcp_rn(s) : 0.f;
        return b;
    } else {
        if (amax != amax) { s = amax; r = 0.f; return 255u; }
        const int f = max((int)(__float_as_uint(amax) >> 23) - 2, 0);   // (inf: 253, its block ends at +-6 * 2^126)
        s = f ? __uint_as_float((uint32_t)f << 23) : __uint_as_float(1u << 22);
        r = f < 254 ? __uint_as_float((uint32_t)(254 - f) << 23) : __uint_as_float(1u << 22);
        return (uint32_t)f;
    }
}

// The rounded quotients v / s of two values, given the rounded reciprocal r of s: q = v r is off by less than two units in
// its last place, and q + (v - q s) r is the rounded quotient (Markstein's correction: v - q s is exact in one fused step,
// and r has no error beyond its own rounding), as long as neither product leaves the normal range.
__device__ __forceinline__ void quotient2(float* v, float s, float r) {
    float q[2], e[2];
    mul2(q, v, r);
    fma2(e, q, -s, v);
    fma2(v, e, r, q);
}
// The same of two quotients v / d, r within a unit in the last place of 1 / d (the result is then within one rounding of the
// quotient, and all but always the rounded quotient).
__device__ __forceinline__ void quotient2v(float* v, const float* d, const float* r) {
    float q[2], e[2];
    mul2v(q, v, r);
    const float n[2] = {-q[0], -q[1]};
    fma2v(e, n, d, v);
    fma2v(v, e, r, q);
}

// N values of one block -> codes, as the correctly rounded quotient v / s rounded to e2m1, so that a quotient half way
// between two codes is one here too. MX: s is a power of two and v * r exact. NV: quotient2. Past 1e30 its products could
// overflow: such a block is one whose scale is at its ceiling, and its values are cut to 1e30 first (they end at +-6 either
// way). (Where v is so small that v - q s is no longer exact, the code is 0 either way.)
template <class F, int N = F::BLK>
__device__ __forceinline__ void block_codes(float* v, float amax, float s, float r, uint32_t* w) {
    if constexpr (F::ID == MOE_FP4_NV) {
        if (amax > 1e30f) {
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = fminf(fmaxf(v[i], -1e30f), 1e30f);
        }
#pragma unroll
        for (int i = 0; i < N; i += 2) quotient2(v + i, s, r);
    } else {
        const float zero[2] = {0.f, 0.f};        // (-0, as a missing column times a negative multiplier, becomes 0)
#pragma unroll
        for (int i = 0; i < N; i += 2) fma2(v + i, v + i, r, zero);
    }
    const bool bad = amax != amax;
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        const uint32_t c = e2m1x8(v + 8 * i);
        w[i] = bad ? 0u : c;
    }
}

template <class F>
__device__ __forceinline__ float scale_value(uint32_t b) {
    if constexpr (F::ID == MOE_FP4_NV) return e4m3_value(b);
    return b == 255u ? __uint_as_float(0x7FC00000u) : b ? __uint_as_float(b << 23) : __uint_as_float(1u << 22);
}

// Tile counts of the groups [offsets[g], offsets[g + 1]) summed up into first[0 .. G] (G <= 1024) by a block of NT threads (and the
// groups' first and last rows into beg and end);
// 0 everywhere, and true, if an offset falls or leaves [0, rows]. (Read from L2: a product does so before it has waited for
// the kernel before it, when an L1 line of an earlier call's offsets may still be there.)
template <int NT>
__device__ __forceinline__ bool scan_groups(const int32_t* offsets, int G, int rows, int* first, int* beg = nullptr,
                                            int* end = nullptr) {
    constexpr int PER = (1024 + NT - 1) / NT;
    __shared__ int s_warp[NT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g0 = threadIdx.x * PER;
    int n[PER], sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        n[i] = 0;
        if (g0 + i < G) {
            const int lo = __ldcg(offsets + g0 + i), hi = __ldcg(offsets + g0 + i + 1);
            if (beg) { beg[g0 + i] = lo; end[g0 + i] = hi; }
            if (lo < 0 || hi < lo || hi > rows) bad = true;
            else n[i] = (int)(((long long)hi - lo + MOE_TILE_M - 1) / MOE_TILE_M);
        }
        sum += n[i];
    }
    bad = __syncthreads_or(bad);
    int v = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) s_warp[warp] = v;
    __syncthreads();
    int at = v - sum;
    for (int i = 0; i < warp; ++i) at += s_warp[i];
    if (threadIdx.x == 0) first[0] = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        at += n[i];
        if (g0 + i < G) first[g0 + i + 1] = bad ? 0 : at;
    }
    __syncthreads();
    return bad;
}

// Tile t of the groups: {group, first row, end, 0}.
__device__ __forceinline__ int4 group_tile(const int32_t* offsets, const int* first, int G, int t) {
    int lo = 0, hi = G;
    while (lo < hi) {                    // last group with first[g] <= t
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= t) lo = mid; else hi = mid - 1;
    }
    const int row0 = offsets[lo] + (t - first[lo]) * MOE_TILE_M;
    return make_int4(lo, row0, min(row0 + MOE_TILE_M, offsets[lo + 1]), 0);
}
#endif

// The rows of the groups, quantised into the product's operand: of `offsets`, or (offsets null) of the schedule that `sched`
// holds. rows_ws: null, or room for x's rows quantised once (gathered_bytes), from which the rows that src names are then
// copied, by the schedule of `offsets` written to `sched`.
int launch_quantize_operand(const void* x, long long ldx, int x_rows, const int32_t* src, const int32_t* offsets, int32_t* sched,
                            int G, int rows, int K, int dtype, int fmt, const float* gscale, void* codes, void* sf,
                            void* rows_ws, unsigned* err, cudaStream_t s);
inline size_t gathered_bytes(int x_rows, int K, int fmt) {
    return align_up((size_t)x_rows * ((K + 31) / 32 * 16), 1024) + align_up((size_t)x_rows * ((K + block_of(fmt) - 1) / block_of(fmt)), 1024);
}
// Whether rows are quantised once and copied: where each row of x is used twice or more on average and the work is worth a
// second launch. (131072 rows of 16384 x 2048 in bf16: 150 us quantised in place.)
inline bool quantize_once(bool gathered, int x_rows, int rows, int K) {
    return gathered && rows >= 2LL * x_rows && (long long)rows * K >= (1LL << 22);
}

}  // namespace fp4
}  // namespace moe
