// Activation checkpoints in 8 bits: what a forward keeps for its backward, a byte a value and an fp32 scale for 128 columns, and the
// SwiGLU backward straight from it.
//
// All bound by memory: a value is read once (2 bytes in bf16) and its code written (1 byte), and in the backward the codes of g and u
// are read (2 bytes a feature) with the act gradient (2) where d_g, d_u and act are written (6); act is computed again there, so
// that it need not be kept.
#include <algorithm>
#include "ffn.cuh"
#include "int8.cuh"

namespace moe {
namespace int8 {

constexpr int C_THREADS = 256, C_WARPS = C_THREADS / 32;
// Blocks of an SM, as many as are resident, with half the loads under way in a lane that three would have room for, each passing
// over its share: 16384 x 28672 bf16 kept in 227 us and through the backward in 361 (6.3 and 6.5 TB/s), where three blocks, and eight an SM launched,
// took 233 and 368.
constexpr int RESIDENT = 4;

// Tiles of a schedule; none (reported) of one of other experts, or of more tiles than the call's rows can have.
__device__ __forceinline__ int tiles_of(const int32_t* sched, int E, int rows, unsigned* err) {
    const bool fits = sched[1] == E && sched[0] <= (rows + MOE_TILE_M - 1) / MOE_TILE_M + E;
    if (!fits && blockIdx.x == 0 && threadIdx.x == 0) latch_device_error(err, kDevErrBadIndex, 0x330u);
    return fits ? sched[0] : 0;
}

// The rows of a call, or of its schedule's tiles, as items of one segment each, `step` apart; row -1: no row of the call.
struct Rows {
    Walk at;
    const int4* tiles;
    int rows;
    __device__ __forceinline__ Rows(const int32_t* sched, int E, int rows_, int nseg, unsigned* err)
        : at((long long)blockIdx.x * C_WARPS + (threadIdx.x >> 5), (long long)gridDim.x * C_WARPS,
             (sched ? (long long)tiles_of(sched, E, rows_, err) * MOE_TILE_M : rows_) * nseg, nseg),
          tiles(sched ? reinterpret_cast<const int4*>(sched + sched_tiles_offset(E)) : nullptr), rows(rows_) {}
    __device__ __forceinline__ int row() const {
        if (!tiles) return at.row;
        const int4 t = tiles[at.row / MOE_TILE_M];
        const int r = t.y + at.row % MOE_TILE_M;
        return r >= 0 && r < min(t.z, rows) ? r : -1;
    }
};

// A warp takes 512 columns of a row at a time: 16 columns a lane, eight lanes to a block, two such items of 16-bit types under way, or
// (!VEC) four blocks one after the other, a lane every 32nd column.
template <typename T, bool VEC>
__global__ void __launch_bounds__(C_THREADS, RESIDENT)
checkpoint_save_kernel(const T* x, long long ldx, int rows, int C, const int32_t* sched, int E, int8_t* codes, float* scales, unsigned* err) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, nb = (C + CKPT - 1) / CKPT;
    Rows it(sched, E, rows, (C + 511) / 512, err);
    while (it.at.left > 0) {
        if constexpr (VEC) {
            constexpr int U = 4 / (int)sizeof(T);
            Raw16<T> raw[U];
            int row[U], k[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                row[u] = it.at.left > 0 ? it.row() : -1;
                k[u] = it.at.seg * 512 + lane * UNIT;
                raw[u] = load_unit<T, true>(x + max(row[u], 0) * ldx, k[u], row[u] >= 0 ? C : 0);
                if (it.at.left > 0) it.at.next();
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (row[u] < 0) continue;
                Steps st;
                float amax = unit_amax(raw[u]);
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const float s = scale_of<T>(amax, st);
                const T* e = reinterpret_cast<const T*>(raw[u].q);
                float v[UNIT];
#pragma unroll
                for (int i = 0; i < UNIT; ++i) v[i] = as_f32(e[i]);
                codes_of<T, UNIT>(v, st);
                if (k[u] < C) {
                    __stcs(reinterpret_cast<uint4*>(codes + (size_t)row[u] * C + k[u]), make_uint4(bytes4(v), bytes4(v + 4), bytes4(v + 8), bytes4(v + 12)));
                    if ((lane & 7) == 0) scales[(size_t)row[u] * nb + k[u] / CKPT] = s;
                }
            }
        } else {
            const int row = it.row(), seg = it.at.seg;
            it.at.next();
            if (row < 0) continue;
            const T* xr = x + row * ldx;
            int8_t* cr = codes + (size_t)row * C;
#pragma unroll 1
            for (int b = 0; b < 4; ++b) {
                const int k0 = seg * 512 + b * CKPT;
                if (k0 >= C) break;
                Steps st;
                float v[4], amax = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = k0 + j * 32 + lane < C ? as_f32(xr[k0 + j * 32 + lane]) : 0.f;
                    amax = max_nan(amax, fabsf(v[j]));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const float s = scale_of<T>(amax, st);
                codes_of<T, 4>(v, st);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (k0 + j * 32 + lane < C) cr[k0 + j * 32 + lane] = (int8_t)__float_as_uint(v[j]);
                if (lane == 0) scales[(size_t)row * nb + k0 / CKPT] = s;
            }
        }
    }
}

// Block b of a row of gu: 128 codes of g, then the 128 of u of the same features, each under its own scale. A lane takes eight
// features, sixteen lanes a block:
//   s = 1 / (1 + exp(-g)), act = g s u, d_g = da u s (1 + g (1 - s)), d_u = da g s     (da 0 past F)
// (The exponential and the quotient are the quick ones: s is off by 2^-21 of itself near g = 0 and by 2^-16 at g = -80, a 2^-7th of bf16's
// half step.)
__global__ void __launch_bounds__(C_THREADS, RESIDENT)
checkpoint_swiglu_backward_kernel(const int8_t* codes, const float* scales, const __nv_bfloat16* d_act, const int32_t* sched, int E, int rows,
                                  int F, int Fp, __nv_bfloat16* d_gu, __nv_bfloat16* act, unsigned* err) {
    pdl_wait();
    pdl_trigger();
    constexpr int U = 1;                      // items whose loads a lane has under way
    const int lane = threadIdx.x & 31;
    Rows it(sched, E, rows, (Fp + 255) / 256, err);
    while (it.at.left > 0) {
        uint2 cg[U], cu[U];
        float2 sc[U];
        Vec16<__nv_bfloat16> da[U];
        size_t at[U], to[U];
        bool live[U], in[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int row = it.at.left > 0 ? it.row() : -1, f = it.at.seg * 256 + lane * 8;
            live[i] = row >= 0 && f < Fp;
            in[i] = row >= 0 && f < F;
            at[i] = (size_t)max(row, 0) * 2 * Fp + (size_t)(f >> 7) * 256 + (f & 127);
            to[i] = (size_t)max(row, 0) * F + f;
            da[i].v = make_uint4(0u, 0u, 0u, 0u);
            if (live[i]) {
                cg[i] = __ldcs(reinterpret_cast<const uint2*>(codes + at[i]));
                cu[i] = __ldcs(reinterpret_cast<const uint2*>(codes + at[i] + 128));
                sc[i] = *reinterpret_cast<const float2*>(scales + (size_t)row * (2 * Fp / CKPT) + (f >> 7) * 2);
            }
            if (in[i]) da[i].v = __ldcs(reinterpret_cast<const uint4*>(d_act + to[i]));
            if (it.at.left > 0) it.at.next();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (!live[i]) continue;
            float g[8], u[8];
            values4(cg[i].x, sc[i].x, g);
            values4(cg[i].y, sc[i].x, g + 4);
            values4(cu[i].x, sc[i].y, u);
            values4(cu[i].y, sc[i].y, u + 4);
            Vec16<__nv_bfloat16> og, ou, oa;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float a = da[i].get(j), s = __fdividef(1.f, 1.f + __expf(-g[j])), gs = g[j] * s;
                og.set(j, a * u[j] * (s + gs * (1.f - s)));
                ou.set(j, a * gs);
                oa.set(j, gs * u[j]);
            }
            st16(d_gu + at[i], og);
            st16(d_gu + at[i] + 128, ou);
            if (in[i]) st16(act + to[i], oa);
        }
    }
}

static int ckpt_grid(long long items) { return (int)std::max<long long>(1, std::min<long long>((items + C_WARPS - 1) / C_WARPS, (long long)RESIDENT * num_sms())); }

static int backward_launch(const void* codes, const float* scales, const void* d_act, const int32_t* sched, int E, int rows, int F, void* d_gu,
                           void* act, cudaStream_t s) {
    const int Fp = (F + 127) / 128 * 128;
    unsigned* err = device_error_word();
    MOE_REQUIRE(err, MOE_ERR_CUDA, "moe_checkpoint8: device error word unavailable");
    const cudaError_t e = launch_pdl(checkpoint_swiglu_backward_kernel, dim3(ckpt_grid((long long)rows * ((Fp + 255) / 256))), dim3(C_THREADS), 0, s,
                                     static_cast<const int8_t*>(codes), scales, static_cast<const __nv_bfloat16*>(d_act), sched, E, rows, F, Fp,
                                     static_cast<__nv_bfloat16*>(d_gu), static_cast<__nv_bfloat16*>(act), err);
    return check_launch(e, "checkpoint_swiglu_backward_kernel");
}

}  // namespace int8
}  // namespace moe

using namespace moe;

static int ckpt_check(const char* fn, int rows, int C, int dtype) {
    MOE_REQUIRE(dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16, MOE_ERR_UNSUPPORTED, "%s: dtype %d", fn, dtype);
    MOE_REQUIRE(rows >= 0 && rows <= MOE_INT8_MAX_ROWS && C >= 1 && C <= MOE_INT8_MAX_K, MOE_ERR_INVALID_ARG, "%s: rows=%d C=%d", fn, rows, C);
    return MOE_OK;
}
static bool on_type(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (dtype == MOE_F32 ? 4 : 2) == 0; }

extern "C" int moe_checkpoint8_save(const void* x, long long ldx, int rows, int C, int dtype, const int32_t* tile_sched, int E, void* codes,
                                    float* scales, void* stream) {
    const char* fn = "moe_checkpoint8_save";
    if (int rc = ckpt_check(fn, rows, C, dtype)) return rc;
    MOE_REQUIRE(ldx >= C && (!tile_sched || (E >= 1 && E <= 1024)), MOE_ERR_INVALID_ARG, "%s: ldx=%lld E=%d", fn, ldx, E);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(x && codes && scales, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    MOE_REQUIRE(on_type(x, dtype) && on_type(scales, MOE_F32) && aligned16(tile_sched), MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    const int el = dtype == MOE_F32 ? 4 : 2;
    const bool vec = C % UNIT == 0 && aligned16(x) && ldx * el % 16 == 0 && aligned16(codes);
    unsigned* err = device_error_word();
    MOE_REQUIRE(err, MOE_ERR_CUDA, "%s: device error word unavailable", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int grid = int8::ckpt_grid((long long)rows * ((C + 511) / 512));
    auto go = [&](auto kernel, auto* p) {
        return launch_pdl(kernel, dim3(grid), dim3(int8::C_THREADS), 0, s, p, ldx, rows, C, tile_sched, E, static_cast<int8_t*>(codes), scales, err);
    };
    cudaError_t e;
    if (dtype == MOE_F32) {
        auto* p = static_cast<const float*>(x);
        e = vec ? go(int8::checkpoint_save_kernel<float, true>, p) : go(int8::checkpoint_save_kernel<float, false>, p);
    } else if (dtype == MOE_BF16) {
        auto* p = static_cast<const __nv_bfloat16*>(x);
        e = vec ? go(int8::checkpoint_save_kernel<__nv_bfloat16, true>, p) : go(int8::checkpoint_save_kernel<__nv_bfloat16, false>, p);
    } else {
        auto* p = static_cast<const __half*>(x);
        e = vec ? go(int8::checkpoint_save_kernel<__half, true>, p) : go(int8::checkpoint_save_kernel<__half, false>, p);
    }
    return check_launch(e, "checkpoint_save_kernel");
}

extern "C" int moe_checkpoint8_load(const void* codes, const float* scales, int rows, int C, int dtype, void* out, long long ldo, void* stream) {
    const char* fn = "moe_checkpoint8_load";
    if (int rc = ckpt_check(fn, rows, C, dtype)) return rc;
    MOE_REQUIRE(ldo >= C, MOE_ERR_INVALID_ARG, "%s: ldo=%lld", fn, ldo);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(codes && scales && out, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    MOE_REQUIRE(on_type(out, dtype) && on_type(scales, MOE_F32), MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    return int8::launch_dequantize(codes, scales, rows, C, dtype, out, ldo, true, static_cast<cudaStream_t>(stream));
}

static int ckpt_backward_check(const char* fn, const void* codes, const float* scales, const void* d_act, const int32_t* sched, int E, int F,
                               int rows, const void* d_gu, const void* act) {
    MOE_REQUIRE(rows >= 0 && rows <= MOE_INT8_MAX_ROWS && F >= 8 && F % 8 == 0 && F <= MOE_INT8_MAX_K / 2 && (!sched || (E >= 1 && E <= 1024)),
                MOE_ERR_INVALID_ARG, "%s: rows=%d F=%d E=%d (need F%%8==0)", fn, rows, F, E);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(codes && scales && d_act && d_gu && act, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    MOE_REQUIRE(aligned16(codes) && aligned16(scales) && aligned16(d_act) && aligned16(sched) && aligned16(d_gu) && aligned16(act),
                MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
    return MOE_OK;
}

extern "C" int moe_checkpoint8_swiglu_backward(const void* codes, const float* scales, const void* d_act, const int32_t* tile_sched, int E, int F,
                                               int rows, void* d_gu, void* act, void* stream) {
    const char* fn = "moe_checkpoint8_swiglu_backward";
    if (int rc = ckpt_backward_check(fn, codes, scales, d_act, tile_sched, E, F, rows, d_gu, act)) return rc;
    if (rows == 0) return MOE_OK;
    return int8::backward_launch(codes, scales, d_act, tile_sched, E, rows, F, d_gu, act, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_expert_up_gate_backward_checkpoint8(const void* codes, const float* scales, const void* d_act, const int32_t* tile_sched,
                                                       const void* packed_bwd, int E, int h, int F, int rows, void* d_gu, void* act, void* d_buf,
                                                       void* stream) {
    const char* fn = "moe_expert_up_gate_backward_checkpoint8";
    MOE_REQUIRE(E >= 1 && E <= 1024 && h > 0 && h % 8 == 0, MOE_ERR_INVALID_ARG, "%s: E=%d h=%d", fn, E, h);
    if (int rc = ckpt_backward_check(fn, codes, scales, d_act, tile_sched, E, F, rows, d_gu, act)) return rc;
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(tile_sched && packed_bwd && d_buf, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    MOE_REQUIRE(aligned16(packed_bwd) && aligned16(d_buf), MOE_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (int rc = int8::backward_launch(codes, scales, d_act, tile_sched, E, rows, F, d_gu, act, s)) return rc;
    return ffn_tc_dbuf(d_gu, tile_sched, packed_bwd, E, h, F, rows, d_buf, s);
}
