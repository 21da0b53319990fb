// Rows of values on their way into and out of a quantised form: types, 16-element units, largest magnitudes, packed fp32
// arithmetic.
#pragma once

#include <cuda_fp16.h>
#include "common.cuh"

namespace moe {

#ifdef __CUDACC__
constexpr int UNIT = 16;             // columns per lane

// NaN if either is: a NaN has to reach its block's scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ void mul2(float* d, const float* a, float b) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1]) : "f"(a[0]), "f"(a[1]), "f"(b));
}
__device__ __forceinline__ void mul2v(float* d, const float* a, const float* b) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1]) : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
__device__ __forceinline__ void add2(float* d, const float* a, float b) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1]) : "f"(a[0]), "f"(a[1]), "f"(b));
}
__device__ __forceinline__ void sub2(float* d, const float* a, const float* b) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tsub.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1]) : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
// The largest of three magnitudes; a NaN counts as none.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void fma2(float* d, const float* a, float b, const float* c) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %6};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1]) : "f"(a[0]), "f"(a[1]), "f"(b), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void fma2v(float* d, const float* a, const float* b, const float* c) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1]) : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T rounded(float v);
template <> __device__ __forceinline__ float rounded<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half rounded<__half>(float v) { return __float2half_rn(v); }

// 16 elements as they lie in memory.
template <typename T> struct alignas(16) Raw16 { uint4 q[sizeof(T)]; };

// 32 bytes at an address on 32, for the 64 bytes of an fp32 unit: one request for a whole sector, where requests of 16 bytes
// 64 apart touch each sector twice (12288 x 4096 fp32 there and back 97 -> 81 us; 16-bit types measured no faster).
__device__ __forceinline__ void ld32(uint4* d, const void* p) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(d[0].x), "=r"(d[0].y), "=r"(d[0].z), "=r"(d[0].w), "=r"(d[1].x), "=r"(d[1].y), "=r"(d[1].z), "=r"(d[1].w)
                 : "l"(p));
}
__device__ __forceinline__ void st32(void* p, const uint4* d) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(p), "r"(d[0].x), "r"(d[0].y), "r"(d[0].z), "r"(d[0].w), "r"(d[1].x), "r"(d[1].y), "r"(d[1].z), "r"(d[1].w)
                 : "memory");
}

// Columns [k0, k0 + 16) of a row as stored, zero past K. VEC: the row starts on 16 bytes. The caller's lanes of one warp
// hold consecutive units of the same row in the other case too, where the elements are fetched one by one.
// again: other rows of the call are the same one, which is to stay in L2 (16384 x 2048 bf16 read eight times over: 121 -> 107 us).
template <typename T, bool VEC>
__device__ __forceinline__ Raw16<T> load_unit(const T* row, int k0, int K, bool again = false) {
    Raw16<T> r;
    if (VEC && k0 + UNIT <= K) {
        if (again) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) r.q[i] = reinterpret_cast<const uint4*>(row + k0)[i];
            return r;
        }
        if (sizeof(T) == 4 && (reinterpret_cast<uintptr_t>(row) & 31u) == 0) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); i += 2) ld32(r.q + i, reinterpret_cast<const uint4*>(row + k0) + i);
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T); ++i) r.q[i] = __ldcs(reinterpret_cast<const uint4*>(row + k0) + i);
        }
        return r;
    }
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) r.q[i] = make_uint4(0u, 0u, 0u, 0u);
    if (k0 < K) {
        T* e = reinterpret_cast<T*>(r.q);
#pragma unroll
        for (int i = 0; i < UNIT; ++i)
            if (k0 + i < K) e[i] = row[k0 + i];
    }
    return r;
}

// The largest magnitude of a unit, NaN if an element is one; 16-bit types two at a time.
__device__ __forceinline__ float unit_amax(const Raw16<float>& raw) {
    const float* e = reinterpret_cast<const float*>(raw.q);
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < UNIT; ++i) m = max_nan(m, fabsf(e[i]));
    return m;
}
__device__ __forceinline__ float unit_amax(const Raw16<__nv_bfloat16>& raw) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw.q);
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < UNIT / 2; ++i) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    return max_nan(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xFFFF0000u)));
}
__device__ __forceinline__ float unit_amax(const Raw16<__half>& raw) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(raw.q);
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < UNIT / 2; ++i) asm("max.NaN.xorsign.abs.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return max_nan(fabsf(f.x), fabsf(f.y));
}

// Items of the row-major kernels, `step` apart, as (row group, segment) without a division each.
struct Walk {
    int row, seg, drow, dseg, nseg;
    long long left;                      // items still to come, this one included, in steps
    __device__ __forceinline__ Walk(long long first, long long step, long long items, int nseg_) : nseg(nseg_) {
        if (((items | (first + step)) >> 30) == 0) {     // (a 64-bit division takes some hundred instructions)
            const unsigned f = (unsigned)first, st = (unsigned)step, n = (unsigned)nseg;
            left = first < items ? ((unsigned)items - f + st - 1) / st : 0;
            row = (int)(f / n);
            seg = (int)(f - (unsigned)row * n);
            drow = (int)(st / n);
            dseg = (int)(st - (unsigned)drow * n);
            return;
        }
        left = first < items ? (items - first + step - 1) / step : 0;
        row = (int)(first / nseg);
        seg = (int)(first - (long long)row * nseg);
        drow = (int)(step / nseg);
        dseg = (int)(step - (long long)drow * nseg);
    }
    __device__ __forceinline__ void next() {
        --left;
        row += drow;
        seg += dseg;
        if (seg >= nseg) { seg -= nseg; ++row; }
    }
};
#endif

}  // namespace moe
