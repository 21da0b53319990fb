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
// (c * 128 + r) * 16, so that a warp whose lanes hold 32 channels reads 512 contiguous bytes. Bytes are code + 128 (the byte under
// 0x64 is the fp16 number 1024 + byte), 128 past N and K.
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

// The scale of values whose largest magnitude is amax, and what they are multiplied with on the way to their codes.
__device__ __forceinline__ float scale_of(float amax, float& inv) {
    const bool finite = amax < INFINITY, live = finite && amax >= TINY;      // (NaN: neither)
    inv = live ? __fdiv_rn(127.f, amax) : 0.f;
    return live ? __fdiv_rn(amax, 127.f) : finite ? 0.f : __uint_as_float(0x7FC00000u);
}

// The code of a value whose product with inv lies so near a border between two codes that its rounding may have crossed it:
// |x| * 127 against border * amax, both exact in 64 bits.
static __device__ __noinline__ float code_at_border(float x, float q, float amax) {
    const float a = fabsf(q), n = rintf(a), lo = a >= n ? n : n - 1.f;
    const double v = (double)fabsf(x) * 127.0, b = ((double)lo + 0.5) * (double)amax;
    const bool up = v > b || (v == b && ((int)lo & 1));
    return copysignf(up ? lo + 1.f : lo, x);
}

// 1.5 * 2^23: its sum with |q| < 2^22 is q rounded to a whole number, ties to even, whose two's complement are the sum's low bits.
constexpr float MAGIC = 12582912.f;

// N values (even) of one row -> MAGIC + their codes. x * inv is off by less than 127 * 2^-23 (both roundings): only a product that
// close to a border is looked at again. Two at a time: the divisions that the definition names would cost four times as much.
template <int N>
__device__ __forceinline__ void codes_of(float* v, float inv, float amax) {
    float t[N], far = 0.f;
    if (inv == 0.f) {                                // (a row of zeros, or one that holds an infinity or a NaN)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        float q[2], d[2];
        mul2(q, v + i, inv);
        add2(t + i, q, MAGIC);
        add2(d, t + i, -MAGIC);
        sub2(d, q, d);
        far = max3_abs(far, d[0], d[1]);
    }
    if (far > 0.49998f) {                            // (rolled, through local memory: it hardly runs)
        float x[N], y[N];
#pragma unroll
        for (int i = 0; i < N; ++i) { x[i] = v[i]; y[i] = t[i]; }
#pragma unroll 1
        for (int i = 0; i < N; ++i) {
            const float q = x[i] * inv;
            if (fabsf(q - (y[i] - MAGIC)) > 0.49998f) y[i] = code_at_border(x[i], q, amax) + MAGIC;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = y[i];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = t[i];
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

// Form of quantised rows: codes [rows][K] as they are kept; the product's operands [rows][pad64(K)], codes as fp16 numbers or as
// bytes, 0 past K.
enum Form : int { FORM_ROWS = 0, FORM_F16 = 1, FORM_BYTES = 2 };
// Rows of x (or those that src names, -1: a row of zeros) -> codes and scales, a programmatic dependent of the kernel before.
int launch_quantize(const void* x, long long ldx, int x_rows, const int32_t* src, int rows, int K, int dtype, int form, void* codes,
                    float* scales, unsigned* err, cudaStream_t s);

}  // namespace int8
}  // namespace moe
