// Quantisation to block-scaled e2m1 and back, with the tile schedule of ragged groups, and the packing of 4-bit weights.
//
// Quantisation and its inverse are bound by memory: x is read once and 0.5 + 1 / BLK bytes a value are written (or the
// other way round). A lane owns 16 consecutive columns (two 16-byte loads of bf16, one 8-byte store of codes), so an NV
// block lives in one lane and an MX block in a pair of lanes; a warp covers 512 columns of a row, or several rows where
// rows are narrower.
#include <algorithm>
#include "fp4.cuh"
#include "quant_io.cuh"

namespace moe {
namespace fp4 {

constexpr int QTHREADS = 256;
constexpr int QWARPS = QTHREADS / 32;
constexpr int SEG = 32 * UNIT;       // columns per warp

// (The kernels that run as programmatic dependents read what the kernel before them may have written by plain loads through
// pointers without __restrict__, which the compiler does not move ahead of the wait.)

// Units whose loads a lane keeps in flight: with four blocks of 256 threads an SM has 64 KB under way.
template <typename T> constexpr int IN_FLIGHT = 4 / (int)sizeof(T);
// The codes (2 words) and the scale byte of this lane's unit; an MX block spans lanes 2i and 2i + 1. (max |x g| is
// max |x| times |g|: rounding keeps the order.)
template <class F, typename T>
__device__ __forceinline__ uint2 quantize_unit(const Raw16<T>& raw, bool scaled, float g, uint32_t& byte) {
    float amax = unit_amax(raw);
    if constexpr (F::ID == MOE_FP4_MX) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    if (scaled) amax = fabsf(amax * g);
    const T* e = reinterpret_cast<const T*>(raw.q);
    float v[UNIT], s, r;
#pragma unroll
    for (int i = 0; i < UNIT; ++i) v[i] = as_f32(e[i]);
    if (scaled) {
#pragma unroll
        for (int i = 0; i < UNIT; i += 2) mul2(v + i, v + i, g);
    }
    byte = block_scale<F>(amax, s, r);
    uint32_t w[2];
    block_codes<F, UNIT>(v, amax, s, r, w);
    return make_uint2(w[0], w[1]);
}

// The schedule of the groups, by one block.
__device__ __noinline__ void write_schedule(const int32_t* offsets, int G, int rows, int32_t* sched, unsigned* err) {
    __shared__ int first[1025];
    const bool bad = scan_groups<QTHREADS>(offsets, G, rows, first);
    if (threadIdx.x == 0) {
        sched[0] = first[G];
        sched[1] = G;
        if (bad) latch_device_error(err, kDevErrBadIndex, 0x202u);
    }
    for (int i = threadIdx.x; i <= G; i += QTHREADS) sched[kSchedHeader + i] = first[i];
    for (int t = threadIdx.x; t < first[G]; t += QTHREADS)
        reinterpret_cast<int4*>(sched + sched_tiles_offset(G))[t] = group_tile(offsets, first, G, t);
}

// Row-major form: codes [rows][pitch], scales [rows][nb]. An item is one row segment of lpr units, 32 / lpr rows to a
// warp (lpr: a power of two, the units of a row where there are fewer than 32).
template <class F, typename T, bool VEC>
__global__ void __launch_bounds__(QTHREADS, 4)
quantize_rows_kernel(const T* x, long long ldx, int x_rows, const int32_t* src, int rows, int K,
                     int lpr, const float* gscale, uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                     const int32_t* offsets, int32_t* sched, int G, int group_rows, unsigned* err) {
    constexpr int U = IN_FLIGHT<T>;
    pdl_wait();
    pdl_trigger();
    if (offsets && blockIdx.x == gridDim.x - 1) write_schedule(offsets, G, group_rows, sched, err);
    __shared__ __align__(16) T s_in[VEC ? 1 : QWARPS][VEC ? 1 : SEG + 8 * 32];
    const int lane = threadIdx.x & 31;
    const int units = (K + 31) / 32 * 2;
    const int nseg = (units + lpr - 1) / lpr, rpw = 32 / lpr, sub = lane / lpr;
    const int nb = (K + F::BLK - 1) / F::BLK;
    const size_t pitch = (size_t)units * 8;
    const float g = gscale ? *gscale : 1.f;
    const int col = lane - sub * lpr;
    Walk at((long long)blockIdx.x * QWARPS + (threadIdx.x >> 5), (long long)gridDim.x * QWARPS,
            (long long)((rows + rpw - 1) / rpw) * nseg, nseg);
    while (at.left > 0) {
        Raw16<T> raw[U];
        int row[U], unit[U];
        const int n = (int)min(at.left, (long long)U);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            row[i] = i < n ? at.row * rpw + sub : rows;
            unit[i] = at.seg * lpr + col;
            const bool live = row[i] < rows && unit[i] < units;
            int from = row[i];
            if (live && src) {
                from = src[row[i]];
                if (from >= x_rows || from < -1) { latch_device_error(err, kDevErrBadIndex, 0x200u); from = -1; }
            }
            if (!VEC && lpr == 32) {             // one row segment a warp, a column a lane: taken apart below
                from = live ? from : -1;
                from = __shfl_sync(0xffffffffu, from, 0);
                const int base = at.seg * SEG;
                const T* row0 = x + (long long)max(from, 0) * ldx + base;
                T* e = reinterpret_cast<T*>(raw[i].q);
#pragma unroll
                for (int j = 0; j < UNIT; ++j) {
                    const int c = j * 32 + lane;
                    e[j] = from >= 0 && base + c < K ? row0[c] : T(0.f);
                }
            } else {
                raw[i] = load_unit<T, VEC>(x + (long long)(live ? max(from, 0) : 0) * ldx, unit[i] * UNIT, live && from >= 0 ? K : 0);
            }
            at.next();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i >= n) break;
            if (!VEC && lpr == 32) {             // (8 elements between the lanes' units, for the banks)
                T* box = s_in[threadIdx.x >> 5];
                T* e = reinterpret_cast<T*>(raw[i].q);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < UNIT; ++j) box[j * 32 + lane + ((j * 32 + lane) >> 4) * 8] = e[j];
                __syncwarp();
#pragma unroll
                for (int j = 0; j < (int)sizeof(T); ++j)
                    raw[i].q[j] = *reinterpret_cast<const uint4*>(box + lane * (UNIT + 8) + j * (16 / (int)sizeof(T)));
            }
            uint32_t byte;
            const uint2 w = quantize_unit<F>(raw[i], gscale != nullptr, g, byte);
            if (row[i] < rows && unit[i] < units) {
                *reinterpret_cast<uint2*>(codes + row[i] * pitch + (size_t)unit[i] * 8) = w;
                const int b = unit[i] * UNIT / F::BLK;
                if (unit[i] * UNIT % F::BLK == 0 && b < nb) scales[(size_t)row[i] * nb + b] = (uint8_t)byte;
            }
        }
    }
}

// Operand form: the rows of the tiles, codes [rows][pad64(K) / 2], scales in the tile layout. The tiles are those of `sched`,
// or with `offsets` those of the groups, found by every block for itself (a launch fewer than a kernel of its own), as the
// products do. A block takes one item at a time, 512 columns of a tile's rows or, where there are few full tiles, of a
// quarter of them (parts = 2: the rows r with r % 32 in its range of 8, whole 16-byte granules of the scale pieces): its
// warps take the rows in turn, the scale bytes meet in shared memory (pieces 528 bytes apart, so that the pieces of one row
// fall into different banks) and leave as whole granules.
template <class F, typename T, bool VEC>
__global__ void __launch_bounds__(QTHREADS, 4)
quantize_operand_kernel(const T* x, long long ldx, int x_rows, const int32_t* src,
                        const int32_t* offsets, const int32_t* sched, int G, int rows, int max_tiles, int parts, int K,
                        const float* gscale, uint8_t* __restrict__ codes, uint8_t* __restrict__ sf, unsigned* err) {
    constexpr int U = IN_FLIGHT<T>, PIECES = 2 * SF_PIECES<F>, STRIDE = 528;
    __shared__ __align__(16) uint8_t s_sf[PIECES * STRIDE];
    __shared__ int s_first[1025];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int units = (K + 63) / 64 * 4, kst = (K + SEG_K - 1) / SEG_K;
    const int nseg = (kst + 1) / 2;
    const size_t pitch = (size_t)units * 8;
    pdl_wait();                          // (a programmatic dependent of the kernel that wrote x or the schedule)
    pdl_trigger();
    const float g = gscale ? *gscale : 1.f;
    const int4* tiles = reinterpret_cast<const int4*>(sched + sched_tiles_offset(G));
    auto tile_of = [&](int t) -> int4 {
        if (offsets) return group_tile(offsets, s_first, G, t);
        const int4 e = tiles[t];
        return make_int4(e.x, min(e.y, rows), min(e.z, rows), 0);
    };
    int ntiles;
    if (offsets) {
        const bool bad = scan_groups<QTHREADS>(offsets, G, rows, s_first);
        ntiles = s_first[G];
        if (bad && blockIdx.x == 0 && threadIdx.x == 0) latch_device_error(err, kDevErrBadIndex, 0x202u);
    } else {
        const bool fits = sched[1] == G && sched[0] <= max_tiles;        // (else: another call's schedule)
        ntiles = fits ? sched[0] : 0;
        if (!fits && blockIdx.x == 0 && threadIdx.x == 0) latch_device_error(err, kDevErrBadIndex, 0x203u);
    }
    const int shift = 5 - parts, per = 1 << shift, ip = nseg << parts;      // granules of four rows in a part; items of a tile
    for (long long it = blockIdx.x; it < (long long)ntiles * ip; it += gridDim.x) {
        const int t = (int)(it / ip), at = (int)(it - (long long)t * ip), seg = at >> parts, part = at & ((1 << parts) - 1);
        const int4 ent = tile_of(t);
        const int n = ent.z - ent.y, unit = seg * 32 + lane;
        for (int i = threadIdx.x; i < PIECES * STRIDE / 16; i += QTHREADS)
            reinterpret_cast<uint4*>(s_sf)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        for (int i0 = warp; i0 < (parts ? 4 * per : n); i0 += U * QWARPS) {
            Raw16<T> raw[U];
            int r[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int j = i0 + i * QWARPS;               // row j of the part: granule j % per, quarter j / per
                r[i] = j < 4 * per ? (j >> shift) * 32 + part * per + (j & (per - 1)) : n;
                int from = r[i] < n ? ent.y + r[i] : -1;
                if (from >= 0 && src) {
                    from = src[from];
                    if (from >= x_rows || from < -1) { latch_device_error(err, kDevErrBadIndex, 0x201u); from = -1; }
                }
                raw[i] = load_unit<T, VEC>(x + (long long)max(from, 0) * ldx, unit * UNIT, from >= 0 ? K : 0);
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                if (r[i] >= n) continue;
                uint32_t byte;
                const uint2 w = quantize_unit<F>(raw[i], gscale != nullptr, g, byte);
                if (unit < units) *reinterpret_cast<uint2*>(codes + (size_t)(ent.y + r[i]) * pitch + (size_t)unit * 8) = w;
                const int b = lane * UNIT / F::BLK;
                if (lane * UNIT % F::BLK == 0)
                    s_sf[(b >> 2) * STRIDE + (r[i] & 31) * 16 + (r[i] >> 5) * 4 + (b & 3)] = (uint8_t)byte;
            }
        }
        __syncthreads();
        const int np = min(2, kst - 2 * seg) * SF_PIECES<F>;      // pieces of the stages that exist
        uint4* dst = reinterpret_cast<uint4*>(sf + ((size_t)t * kst + 2 * seg) * SF_BYTES<F>);
        for (int i = threadIdx.x; i < np << shift; i += QTHREADS) {
            const int q = i >> shift, gr = part * per + (i & (per - 1));
            dst[q * 32 + gr] = *reinterpret_cast<const uint4*>(s_sf + q * STRIDE + gr * 16);
        }
        __syncthreads();
    }
}

// Operand form from rows that are quantised already (row-major, codes [x_rows][q_pitch], scales [x_rows][nb]): a token's rows
// in several groups are quantised once and copied. An item is 512 columns of a tile's rows; 16 lanes copy a row's 256 bytes
// of codes, and a thread gathers a granule of scales, four rows' words.
template <class F>
__global__ void __launch_bounds__(QTHREADS)
gather_operand_kernel(const uint8_t* q_codes, const uint8_t* q_scales, int x_rows,
                      const int32_t* src, const int32_t* sched, int G, int rows, int max_tiles, int K,
                      uint8_t* __restrict__ codes, uint8_t* __restrict__ sf, unsigned* err) {
    constexpr int U = 8, PIECES = 2 * SF_PIECES<F>;
    __shared__ int s_from[MOE_TILE_M];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kst = (K + SEG_K - 1) / SEG_K, nseg = (kst + 1) / 2, nb = (K + F::BLK - 1) / F::BLK;
    const int pitch = (K + 63) / 64 * 32, q_pitch = (K + 31) / 32 * 16;
    pdl_wait();
    pdl_trigger();
    const bool fits = sched[1] == G && sched[0] <= max_tiles;            // (else: another call's schedule)
    const int ntiles = fits ? sched[0] : 0;
    if (!fits && blockIdx.x == 0 && threadIdx.x == 0) latch_device_error(err, kDevErrBadIndex, 0x203u);
    const int4* tiles = reinterpret_cast<const int4*>(sched + sched_tiles_offset(G));
    for (long long it = blockIdx.x; it < (long long)ntiles * nseg; it += gridDim.x) {
        const int t = (int)(it / nseg), seg = (int)(it - (long long)t * nseg);
        const int4 ent = tiles[t];
        const int n = min(ent.z, rows) - ent.y;
        __syncthreads();
        if (threadIdx.x < MOE_TILE_M) {
            int from = -1;
            if ((int)threadIdx.x < n) {
                from = src[ent.y + threadIdx.x];
                if (from >= x_rows || from < -1) { latch_device_error(err, kDevErrBadIndex, 0x201u); from = -1; }
            }
            s_from[threadIdx.x] = from;
        }
        __syncthreads();
        // codes: 16 lanes to a row's 256 bytes
        const int c = seg * 256 + (lane & 15) * 16;
        for (int r0 = warp * 2 + (lane >> 4); r0 < n; r0 += U * 2 * QWARPS) {
            uint4 v[U];
            int from[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {            // (loads without a branch: they stay in flight together)
                from[i] = s_from[min(r0 + i * 2 * QWARPS, MOE_TILE_M - 1)];
                v[i] = *reinterpret_cast<const uint4*>(q_codes + (size_t)max(from[i], 0) * q_pitch + min(c, q_pitch - 16));
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int r = r0 + i * 2 * QWARPS;
                if (from[i] < 0 || c >= q_pitch) v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < n && c < pitch) *reinterpret_cast<uint4*>(codes + (size_t)(ent.y + r) * pitch + c) = v[i];
            }
        }
        // scales: a thread writes a granule (16 bytes: four rows' words) of a piece
        const int np = min(2, kst - 2 * seg) * SF_PIECES<F>;
        uint4* dst = reinterpret_cast<uint4*>(sf + ((size_t)t * kst + 2 * seg) * SF_BYTES<F>);
        for (int i = threadIdx.x; i < np * 32; i += QTHREADS) {
            const int q = i >> 5, b0 = (seg * PIECES + q) * 4;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int from = s_from[(i & 31) + 32 * j];
                w[j] = 0u;
                if (from >= 0) {
                    const uint8_t* row = q_scales + (size_t)from * nb + b0;
                    if ((nb & 3) == 0) {
                        if (b0 < nb) w[j] = *reinterpret_cast<const uint32_t*>(row);
                    } else {
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            if (b0 + b < nb) w[j] |= (uint32_t)row[b] << (8 * b);
                    }
                }
            }
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Sixteen codes under one scale -> values, exact in fp32 (2 and 4 significant bits; NV in fp16 too, two at a time), divided
// by g where there is one: the rounded quotient (quotient2), or the division itself where scale or g come near the ends of
// the range.
template <class F>
__device__ __forceinline__ void unit_values(uint2 c, uint32_t sb, bool scaled, float g, float r, float* v) {
    const uint32_t w[2] = {c.x, c.y};
    const float s = scale_value<F>(sb);
    const __half2 sh = __float2half2_rn(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t h2;
        asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h2) : "r"(w[j >> 2] >> (8 * (j & 3))));
        __half2 h = *reinterpret_cast<const __half2*>(&h2);
        if constexpr (F::ID == MOE_FP4_NV) h = __hmul2(h, sh);
        const float2 f = __half22float2(h);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
        if constexpr (F::ID == MOE_FP4_MX) mul2(v + 2 * j, v + 2 * j, s);
    }
    if (!scaled) return;
    const float m = fabsf(s), a = fabsf(g);
    if (((m < 1e15f && m > 1e-15f) || m == 0.f) && a < 1e15f && a > 1e-15f) {
#pragma unroll
        for (int j = 0; j < UNIT; j += 2) quotient2(v + j, g, r);
    } else {
#pragma unroll
        for (int j = 0; j < UNIT; ++j) v[j] = __fdiv_rn(v[j], g);
    }
}

template <class F, typename T, bool VEC>
__global__ void __launch_bounds__(QTHREADS, 4)
dequantize_rows_kernel(const uint8_t* codes, const uint8_t* scales, int rows, int K, int lpr, const float* gscale, T* out,
                       long long ldo) {
    constexpr int U = 2;
    pdl_wait();
    pdl_trigger();
    __shared__ __align__(16) T s_out[VEC ? 1 : QWARPS][VEC ? 1 : SEG + 8 * 32];
    const int lane = threadIdx.x & 31;
    const int units = (K + 31) / 32 * 2;
    const int nseg = (units + lpr - 1) / lpr, rpw = 32 / lpr, sub = lane / lpr, col = lane - sub * lpr;
    const int nb = (K + F::BLK - 1) / F::BLK;
    const size_t pitch = (size_t)units * 8;
    const float g = gscale ? *gscale : 1.f, r = __frcp_rn(g);
    Walk at((long long)blockIdx.x * QWARPS + (threadIdx.x >> 5), (long long)gridDim.x * QWARPS,
            (long long)((rows + rpw - 1) / rpw) * nseg, nseg);
    while (at.left > 0) {
        uint2 c[U];
        uint32_t sb[U];
        int row[U], unit[U];
        const int n = (int)min(at.left, (long long)U);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            row[i] = i < n ? at.row * rpw + sub : rows;
            unit[i] = at.seg * lpr + col;
            c[i] = make_uint2(0u, 0u);
            sb[i] = 0u;
            if (row[i] < rows && unit[i] < units) {
                c[i] = __ldcs(reinterpret_cast<const uint2*>(codes + row[i] * pitch + (size_t)unit[i] * 8));
                const int b = unit[i] * UNIT / F::BLK;
                if (b < nb) sb[i] = scales[(size_t)row[i] * nb + b];
            }
            at.next();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i >= n) break;
            float v[UNIT];
            unit_values<F>(c[i], sb[i], gscale != nullptr, g, r, v);
            Raw16<T> o;
            T* e = reinterpret_cast<T*>(o.q);
#pragma unroll
            for (int j = 0; j < UNIT; ++j) e[j] = rounded<T>(v[j]);
            const int k0 = unit[i] * UNIT;
            const bool live = row[i] < rows && k0 < K;
            T* dst = out + (long long)row[i] * ldo + k0;
            if (VEC) {
                if (live && k0 + UNIT <= K) {
                    if (sizeof(T) == 4 && (reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
#pragma unroll
                        for (int q = 0; q < (int)sizeof(T); q += 2) st32(reinterpret_cast<uint4*>(dst) + q, o.q + q);
                    } else {
#pragma unroll
                        for (int q = 0; q < (int)sizeof(T); ++q) __stcs(reinterpret_cast<uint4*>(dst) + q, o.q[q]);
                    }
                } else if (live) {
#pragma unroll
                    for (int q = 0; q < UNIT; ++q)
                        if (k0 + q < K) dst[q] = e[q];
                }
            } else if (lpr == 32) {              // one row segment a warp: through shared memory, a column a lane
                T* box = s_out[threadIdx.x >> 5];
                __syncwarp();
#pragma unroll
                for (int q = 0; q < (int)sizeof(T); ++q)     // (8 elements between the lanes' units, for the banks)
                    *reinterpret_cast<uint4*>(box + lane * (UNIT + 8) + q * (16 / (int)sizeof(T))) = o.q[q];
                __syncwarp();
                const int base = (unit[i] - lane) * UNIT;
                T* drow = out + (long long)row[i] * ldo + base;
                if (row[i] < rows) {
#pragma unroll
                    for (int j = 0; j < UNIT; ++j) {
                        const int q = j * 32 + lane;
                        if (base + q < K) drow[q] = box[q + (q >> 4) * 8];
                    }
                }
            } else if (live) {
#pragma unroll
                for (int q = 0; q < UNIT; ++q)
                    if (k0 + q < K) dst[q] = e[q];
            }
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// weight packing (once per weight)
// ---------------------------------------------------------------------------------------------------
// Row p of the packed matrix: row p of `c0`, or with c1 (gate and up) 32 rows of c0, the same 32 of c1, and so on.
struct PackSrc { const uint8_t *c0, *c1; };
__device__ __forceinline__ const uint8_t* pack_row(const PackSrc& s, int g, int p, int N, size_t bytes_per_row) {
    int n = p;
    const uint8_t* m = s.c0;
    if (s.c1) {
        n = (p >> 6) * 32 + (p & 31);
        m = (p & 32) ? s.c1 : s.c0;
    }
    return n < N ? m + ((size_t)g * N + n) * bytes_per_row : nullptr;
}

// One 16-byte chunk of codes (32 columns) a thread, codes past K cleared.
__global__ void __launch_bounds__(256)
pack_codes_kernel(PackSrc src, int N, int K, WeightLayout L, long long chunks, uint8_t* __restrict__ dst) {
    const size_t pitch = (size_t)(K + 31) / 32 * 16;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < chunks; i += (long long)gridDim.x * blockDim.x) {
        const int c = (int)(i & 7), r = (int)(i >> 3 & 63);
        long long q = i >> 9;                    // (group, stage, 64-row block)
        const int nb = (int)(q % L.NB64);
        q /= L.NB64;
        const int st = (int)(q % L.KST), g = (int)(q / L.KST);
        const int k0 = st * SEG_K + c * 32;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        const uint8_t* row = k0 < K ? pack_row(src, g, nb * 64 + r, N, pitch) : nullptr;
        if (row) {
            v = *reinterpret_cast<const uint4*>(row + k0 / 2);
            uint32_t* w = &v.x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int left = K - (k0 + 8 * j);
                if (left < 8) w[j] &= left <= 0 ? 0u : (1u << (4 * left)) - 1u;
            }
        }
        *reinterpret_cast<uint4*>(dst + (i >> 9) * 8192 + r * 128 + ((c ^ (r & 7)) << 4)) = v;
    }
}

// One scale byte a thread.
__global__ void __launch_bounds__(256)
pack_scales_kernel(PackSrc src, int N, int K, int blk, int sfb, WeightLayout L, long long bytes, uint8_t* __restrict__ dst) {
    const int nblk = (K + blk - 1) / blk;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < bytes; i += (long long)gridDim.x * blockDim.x) {
        const int at = (int)(i % sfb);
        long long q = i / sfb;                   // (group, stage, 128-row block)
        const int nb = (int)(q % L.NB128);
        q /= L.NB128;
        const int st = (int)(q % L.KST), g = (int)(q / L.KST);
        const int r = (at >> 4 & 31) + (at >> 2 & 3) * 32, b = (at >> 9) * 4 + (at & 3) + st * (SEG_K / blk);
        const uint8_t* row = b < nblk ? pack_row(src, g, nb * 128 + r, N, nblk) : nullptr;
        dst[i] = row ? row[b] : 0;
    }
}

static int pack(PackSrc codes, PackSrc scales, int G, int N, int n_packed, int K, int fmt, void* packed, cudaStream_t s) {
    const WeightLayout L = weight_layout(G, n_packed, K, fmt);
    uint8_t* p = static_cast<uint8_t*>(packed);
    const long long chunks = (long long)L.sf_off / 16, bytes = (long long)(L.total - L.sf_off);
    pack_codes_kernel<<<(int)std::min<long long>(cdiv(chunks, 256), 16384), 256, 0, s>>>(codes, N, K, L, chunks, p);
    if (int rc = check_launch("pack_codes_kernel")) return rc;
    pack_scales_kernel<<<(int)std::min<long long>(cdiv(bytes, 256), 16384), 256, 0, s>>>(scales, N, K, block_of(fmt),
                                                                                      sf_bytes(fmt), L, bytes, p + L.sf_off);
    return check_launch("pack_scales_kernel");
}

// ---------------------------------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------------------------------
static int el_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
static bool dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }
static bool vec_ok(const void* p, long long ld, int dtype) { return aligned16(p) && ld * el_bytes(dtype) % 16 == 0; }

// Calls fn<Format, T, VEC>(...) for the run-time format, type and alignment.
template <typename Fn>
static int by_kind(int fmt, int dtype, bool vec, Fn fn) {
    auto typed = [&](auto f) -> int {
        auto go = [&](auto t) -> int { return vec ? fn(f, t, std::true_type{}) : fn(f, t, std::false_type{}); };
        if (dtype == MOE_F32) return go(float{});
        if (dtype == MOE_BF16) return go(__nv_bfloat16{});
        return go(__half{});
    };
    return fmt == MOE_FP4_NV ? typed(Nv{}) : typed(Mx{});
}

static int lanes_per_row(int K) {
    const int units = (K + 31) / 32 * 2;
    int l = 2;
    while (l < 32 && l < units) l *= 2;
    return l;
}
static int row_grid(int rows, int K, int lpr) {
    const long long items = (long long)cdiv(rows, 32 / lpr) * cdiv((K + 31) / 32 * 2, lpr);
    return (int)std::max<long long>(1, std::min<long long>(cdiv(items, QWARPS), (long long)num_sms() * 4));
}

int launch_quantize_operand(const void* x, long long ldx, int x_rows, const int32_t* src, const int32_t* offsets, int32_t* sched,
                            int G, int rows, int K, int dtype, int fmt, const float* gscale, void* codes, void* sf,
                            void* rows_ws, unsigned* err, cudaStream_t s) {
    if (rows_ws) {
        // once per row of x, then a copy per use
        uint8_t *qc = static_cast<uint8_t*>(rows_ws), *qs = qc + align_up((size_t)x_rows * ((K + 31) / 32 * 16), 1024);
        const int lpr = lanes_per_row(K), grid = row_grid(x_rows, K, lpr);
        if (int rc = by_kind(fmt, dtype, vec_ok(x, ldx, dtype), [&](auto f, auto t, auto v) {
                using T = decltype(t);
                return check_launch(launch_pdl(quantize_rows_kernel<decltype(f), T, decltype(v)::value>, dim3(grid), dim3(QTHREADS), 0, s,
                                               static_cast<const T*>(x), ldx, x_rows, nullptr, x_rows, K, lpr, gscale, qc, qs,
                                               offsets, sched, G, rows, err),
                                    "quantize_rows_kernel");
            }))
            return rc;
        const int g2 = (int)std::min<long long>((long long)sched_max_tiles(rows, std::min(G, rows)) * cdiv(stages_of(K), 2),
                                                (long long)num_sms() * 8);
        auto gather = [&](auto f) {
            return check_launch(launch_pdl(gather_operand_kernel<decltype(f)>, dim3(g2), dim3(QTHREADS), 0, s, qc, qs, x_rows, src,
                                           sched, G, rows, (int)sched_max_tiles(rows, G), K, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(sf), err),
                                "gather_operand_kernel");
        };
        return fmt == MOE_FP4_NV ? gather(Nv{}) : gather(Mx{});
    }
    const long long items = (long long)sched_max_tiles(rows, std::min(G, rows)) * cdiv(stages_of(K), 2);
    const int parts = items < 4LL * num_sms() && rows > 32LL * std::min(G, rows) ? 2 : 0;
    const int grid = (int)std::min<long long>(items << parts, (long long)num_sms() * 4);
    return by_kind(fmt, dtype, vec_ok(x, ldx, dtype), [&](auto f, auto t, auto v) {
        using F = decltype(f);
        using T = decltype(t);
        return check_launch(launch_pdl(quantize_operand_kernel<F, T, decltype(v)::value>, dim3(grid), dim3(QTHREADS), 0, s,
                                       static_cast<const T*>(x), ldx, x_rows, src, offsets, sched, G, rows,
                                       (int)sched_max_tiles(rows, G), parts, K, gscale, static_cast<uint8_t*>(codes),
                                       static_cast<uint8_t*>(sf), err),
                            "quantize_operand_kernel");
    });
}

}  // namespace fp4
}  // namespace moe

using namespace moe;
using namespace moe::fp4;

static bool fmt_ok(int fmt) { return fmt == MOE_FP4_NV || fmt == MOE_FP4_MX; }

extern "C" size_t moe_fp4_codes_pitch(int K) { return K < 1 ? 0 : (size_t)(((long long)K + 31) / 32) * 16; }
extern "C" size_t moe_fp4_scales_pitch(int K, int fmt) {
    return K < 1 || !fmt_ok(fmt) ? 0 : (size_t)((K + block_of(fmt) - 1) / block_of(fmt));
}

extern "C" int moe_fp4_quantize(const void* x, long long ldx, int x_rows, const int32_t* src, int rows, int K, int dtype,
                                int fmt, const float* gscale, void* codes, void* scales, void* stream) {
    MOE_REQUIRE(dtype_ok(dtype), MOE_ERR_UNSUPPORTED, "moe_fp4_quantize: dtype %d", dtype);
    MOE_REQUIRE(fmt_ok(fmt), MOE_ERR_UNSUPPORTED, "moe_fp4_quantize: format %d", fmt);
    MOE_REQUIRE(rows >= 0 && x_rows >= 0 && K >= 1 && K <= MOE_FP4_MAX_K && ldx >= K, MOE_ERR_INVALID_ARG,
                "moe_fp4_quantize: rows=%d x_rows=%d K=%d ldx=%lld", rows, x_rows, K, ldx);
    MOE_REQUIRE(src || x_rows >= rows, MOE_ERR_INVALID_ARG, "moe_fp4_quantize: x has %d rows, %d wanted", x_rows, rows);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE((x || x_rows == 0) && codes && scales, MOE_ERR_INVALID_ARG, "moe_fp4_quantize: null pointer");
    MOE_REQUIRE(aligned16(codes) && reinterpret_cast<uintptr_t>(x) % el_bytes(dtype) == 0, MOE_ERR_INVALID_ARG,
                "moe_fp4_quantize: codes must be 16-byte aligned, x aligned to its type");
    const int lpr = lanes_per_row(K), grid = row_grid(rows, K, lpr);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_kind(fmt, dtype, vec_ok(x, ldx, dtype), [&](auto f, auto t, auto v) {
        using T = decltype(t);
        return check_launch(launch_pdl(quantize_rows_kernel<decltype(f), T, decltype(v)::value>, dim3(grid), dim3(QTHREADS), 0, s,
                                       static_cast<const T*>(x), ldx, x_rows, src, rows, K, lpr, gscale,
                                       static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), nullptr, nullptr, 0, 0,
                                       device_error_word()),
                            "quantize_rows_kernel");
    });
}

extern "C" int moe_fp4_dequantize(const void* codes, const void* scales, int rows, int K, int fmt, const float* gscale,
                                  int dtype, void* out, long long ldo, void* stream) {
    MOE_REQUIRE(dtype_ok(dtype), MOE_ERR_UNSUPPORTED, "moe_fp4_dequantize: dtype %d", dtype);
    MOE_REQUIRE(fmt_ok(fmt), MOE_ERR_UNSUPPORTED, "moe_fp4_dequantize: format %d", fmt);
    MOE_REQUIRE(rows >= 0 && K >= 1 && K <= MOE_FP4_MAX_K && ldo >= K, MOE_ERR_INVALID_ARG,
                "moe_fp4_dequantize: rows=%d K=%d ldo=%lld", rows, K, ldo);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(codes && scales && out, MOE_ERR_INVALID_ARG, "moe_fp4_dequantize: null pointer");
    MOE_REQUIRE(aligned16(codes) && reinterpret_cast<uintptr_t>(out) % el_bytes(dtype) == 0, MOE_ERR_INVALID_ARG,
                "moe_fp4_dequantize: codes must be 16-byte aligned, out aligned to its type");
    const int lpr = lanes_per_row(K), grid = row_grid(rows, K, lpr);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    return by_kind(fmt, dtype, vec_ok(out, ldo, dtype), [&](auto f, auto t, auto v) {
        using T = decltype(t);
        return check_launch(launch_pdl(dequantize_rows_kernel<decltype(f), T, decltype(v)::value>, dim3(grid), dim3(QTHREADS), 0, s,
                                       static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), rows, K, lpr,
                                       gscale, static_cast<T*>(out), ldo),
                            "dequantize_rows_kernel");
    });
}

// G * N * K in packed bytes stays far below what a 64-bit size holds; the kernels' row indices are 32-bit.
static int check_weight(const char* who, int G, int N, int K, int fmt) {
    MOE_REQUIRE(fmt_ok(fmt), MOE_ERR_UNSUPPORTED, "%s: format %d", who, fmt);
    MOE_REQUIRE(G >= 1 && G <= 1024 && N >= 1 && N <= MOE_FP4_MAX_K && K >= 1 && K <= MOE_FP4_MAX_K, MOE_ERR_INVALID_ARG,
                "%s: groups=%d N=%d K=%d", who, G, N, K);
    return MOE_OK;
}

extern "C" size_t moe_fp4_packed_weight_bytes(int G, int N, int K, int fmt) {
    return check_weight("moe_fp4_packed_weight_bytes", G, N, K, fmt) ? 0 : weight_layout(G, N, K, fmt).total;
}

extern "C" int moe_fp4_pack_weight(const void* codes, const void* scales, int G, int N, int K, int fmt, void* packed,
                                   void* stream) {
    if (int rc = check_weight("moe_fp4_pack_weight", G, N, K, fmt)) return rc;
    MOE_REQUIRE(codes && scales && packed && aligned16(codes) && aligned16(packed), MOE_ERR_INVALID_ARG,
                "moe_fp4_pack_weight: pointers must be non-null, codes and packed 16-byte aligned");
    return pack(PackSrc{static_cast<const uint8_t*>(codes), nullptr}, PackSrc{static_cast<const uint8_t*>(scales), nullptr},
                G, N, N, K, fmt, packed, static_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_fp4_packed_expert_weights_bytes(int E, int h, int F, int fmt) {
    if (check_weight("moe_fp4_packed_expert_weights_bytes", E, h, F, fmt)) return 0;
    return expert_layout(E, h, F, fmt).total;
}

extern "C" int moe_fp4_pack_expert_weights(const void* gate_codes, const void* gate_scales, const void* up_codes,
                                           const void* up_scales, const void* down_codes, const void* down_scales, int E,
                                           int h, int F, int fmt, void* packed, void* stream) {
    if (int rc = check_weight("moe_fp4_pack_expert_weights", E, h, F, fmt)) return rc;
    MOE_REQUIRE(gate_codes && gate_scales && up_codes && up_scales && down_codes && down_scales && packed,
                MOE_ERR_INVALID_ARG, "moe_fp4_pack_expert_weights: null pointer");
    MOE_REQUIRE(aligned16(gate_codes) && aligned16(up_codes) && aligned16(down_codes) && aligned16(packed),
                MOE_ERR_INVALID_ARG, "moe_fp4_pack_expert_weights: codes and packed must be 16-byte aligned");
    const ExpertLayout L = expert_layout(E, h, F, fmt);
    auto u8 = [](const void* p) { return static_cast<const uint8_t*>(p); };
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int rc = pack(PackSrc{u8(gate_codes), u8(up_codes)}, PackSrc{u8(gate_scales), u8(up_scales)}, E, F, 2 * pad64(F), h,
                      fmt, packed, s))
        return rc;
    return pack(PackSrc{u8(down_codes), nullptr}, PackSrc{u8(down_scales), nullptr}, E, h, h, F, fmt,
                static_cast<uint8_t*>(packed) + L.down_off, s);
}
