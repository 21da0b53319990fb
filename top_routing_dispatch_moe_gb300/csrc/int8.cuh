// 8-bit integers under fp32 scales: format, layouts and the arithmetic shared by the quantisation kernels.
//
// A row (or a block of 128 columns of an activation checkpoint) has the scale amax / 127, and each value the code nearest to
// x * 127 / amax, ties to even: -127 .. 127. A row whose amax is below 2^-96 counts as zero (scale and codes 0; 127 / amax
// stays in fp32's range); one that holds an infinity or a NaN has the scale NaN and codes 0, so that its products are NaN.
#pragma once

#include "common.cuh"
#include "quant_io.cuh"

namespace moe {
namespace int8 {

constexpr int STAGE_K = 64;          // columns of a packed weight piece
constexpr int BLOCK_N = 128;         // output channels of a packed weight piece
constexpr int PIECE = BLOCK_N * STAGE_K;
constexpr int CKPT = 128;            // columns under one scale of a checkpoint

inline int pad64(int k) { return (k + 63) / 64 * 64; }

// A packed weight [G][N][K]: pieces [G][N / 128][K / 64] of 8 KB, the 16-byte chunk c (columns 16 c ..) of channel r of a piece at
// (c * 128 + (r ^ 2 c)) * 16: eight lanes with a chunk of eight channels each, or with four chunks of two, read different banks. Bytes
// are code + 128 (the byte under 0x64 is the fp16 number 1024 + byte), 128 past N and K.
struct WeightLayout { int NB, KST; size_t total; };
inline WeightLayout weight_layout(int G, int N, int K) {
    WeightLayout L;
    L.NB = (N + BLOCK_N - 1) / BLOCK_N;
    L.KST = pad64(K) / STAGE_K;
    L.total = (size_t)G * L.NB * L.KST * PIECE;
    return L;
}
// The expert FFN's packed weight: gate and up rows in turn (N = 2 F: channel 2 f the gate's row f, 2 f + 1 the up's), K = h; then
// down (N = h, K = F).
struct ExpertLayout { WeightLayout gu, down; size_t down_off, total; };
inline ExpertLayout expert_layout(int E, int h, int F) {
    ExpertLayout L;
    L.gu = weight_layout(E, 2 * F, h);
    L.down = weight_layout(E, h, F);
    L.down_off = L.gu.total;
    L.total = L.gu.total + L.down.total;
    return L;
}

#ifdef __CUDACC__
constexpr float TINY = 1.262177448e-29f;             // 2^-96

// The way of values whose largest magnitude is amax to their codes, x * 127 / amax; live: the codes are not all 0.
// 16-bit types: inv + low is 127 / amax to 2^-28 of it or better. fp32: inv the rounded 127 / amax, and x * c / a with c = 127 (both times
// 2^-32 where 127 x could leave fp32's range).
struct Steps { float c, a, inv, low; bool live; };
// The scale of such values.
template <typename T>
__device__ __forceinline__ float scale_of(float amax, Steps& st) {
    const bool finite = amax < INFINITY;             // (NaN: not)
    st.live = finite && amax >= TINY;
    if constexpr (sizeof(T) == 2) {
        const float a = st.live ? amax : 1.f, r = __frcp_rn(a);
        st.inv = 127.f * r;
        st.low = fmaf(-st.inv, a, 127.f) * r;
    } else {
        const float f = amax > 1e30f ? 2.3283064365386963e-10f : 1.f;
        st.c = 127.f * f;
        st.a = st.live ? amax * f : 1.f;
        st.inv = st.live ? __fdiv_rn(127.f, amax) : 0.f;
    }
    const float q = amax * (1.f / 127.f), scale = fmaf(fmaf(-q, 127.f, amax), 1.f / 127.f, q);      // amax / 127, rounded
    return st.live ? scale : finite ? 0.f : __uint_as_float(0x7FC00000u);
}

// 1.5 * 2^23: its sum with |q| < 2^22 is q rounded to a whole number, ties to even, whose two's complement are the sum's low bits.
constexpr float MAGIC = 12582912.f;

// MAGIC + the code of an fp32 value whose product with inv lies so near the border between two codes that its roundings may have crossed
// it: the side that x c - border a says, x c in two parts and each step exact.
static __device__ __noinline__ float code_at_border(float x, float q, const Steps& st) {
    const float n = rintf(q), border = q >= n ? n + 0.5f : n - 0.5f, lo = border - 0.5f;
    const float p = x * st.c, pe = fmaf(-x, st.c, p), rest = fmaf(-border, st.a, p) - pe;
    const bool up = rest > 0.f || (rest == 0.f && ((int)lo & 1));
    return MAGIC + (up ? lo + 1.f : lo);
}

// N values (even) of one row, of type T -> MAGIC + their codes, two values an instruction.
// 16 bits: x inv + x low, the second rounded by itself, is the quotient to 2^-27 of it before its one rounding. Half way between two codes
// is a number of eight bits, so a tie is met to the bit, and no other quotient of numbers of 11 bits comes within 2^-20 of itself to a border.
// (With a test for quotients near a border instead, two thirds of all blocks of bf16 values had a tie, and 16384 x 28672 of them
// took 690 us; with the quotient corrected by its exact remainder, two more steps a value, those kept
// and through the SwiGLU backward took 617 us, then 606; 592 since four blocks share an SM.)
// fp32: x inv is off by less than 127 * 2^-23; only a product that close to a border, which among sums and products few are, is looked at again.
template <typename T, int N>
__device__ __forceinline__ void codes_of(float* v, const Steps& st) {
    if (!st.live) {                                  // (zeros, or an infinity or a NaN among them)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = MAGIC;
        return;
    }
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float q[2];
            mul2(q, v + i, st.low);
            fma2(q, v + i, st.inv, q);
            add2(v + i, q, MAGIC);
        }
    } else {
        float t[N], far = 0.f;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            float q[2], d[2];
            mul2(q, v + i, st.inv);
            add2(t + i, q, MAGIC);
            add2(d, t + i, -MAGIC);
            sub2(d, q, d);
            far = max3_abs(far, d[0], d[1]);
        }
        if (far > 0.49998f) {                        // (rolled, through local memory: it hardly runs)
            float x[N], y[N];
#pragma unroll
            for (int i = 0; i < N; ++i) { x[i] = v[i]; y[i] = t[i]; }
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                const float q = x[i] * st.inv;
                if (fabsf(q - (y[i] - MAGIC)) > 0.49998f) y[i] = code_at_border(x[i], q, st);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) t[i] = y[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = t[i];
    }
}
// Four codes as codes_of leaves them -> bytes; two -> fp16 numbers.
__device__ __forceinline__ uint32_t bytes4(const float* v) {
    return __byte_perm(__byte_perm(__float_as_uint(v[0]), __float_as_uint(v[1]), 0x0040),
                       __byte_perm(__float_as_uint(v[2]), __float_as_uint(v[3]), 0x0040), 0x5410);
}
__device__ __forceinline__ __half2 halves2(const float* v) {
    float n[2];
    add2(n, v, -MAGIC);
    return __floats2half2_rn(n[0], n[1]);
}
// Four bytes of codes -> fp32 numbers times s: a byte with its sign bit turned, under 0x4B0000, is the number 2^23 + 128 + code.
__device__ __forceinline__ void values4(uint32_t w, float s, float* v) {
    w ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440 + i));
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        add2(v + i, v + i, -8388736.f);
        mul2(v + i, v + i, s);
    }
}
#endif

// Form of quantised rows: codes [rows][K] as they are kept; the product's operand [rows][pad64(K)], codes as fp16 numbers, 0 past K.
enum Form : int { FORM_ROWS = 0, FORM_F16 = 1 };
// Rows of x (or those that src names, -1: a row of zeros) -> codes and scales, a programmatic dependent of the kernel before.
int launch_quantize(const void* x, long long ldx, int x_rows, const int32_t* src, int rows, int K, int dtype, int form, void* codes,
                    float* scales, unsigned* err, cudaStream_t s);
// Codes [rows][K] -> values; blocks: under the scales of a checkpoint.
int launch_dequantize(const void* codes, const float* scales, int rows, int K, int dtype, void* out, long long ldo, bool blocks, cudaStream_t s);

}  // namespace int8
}  // namespace moe
