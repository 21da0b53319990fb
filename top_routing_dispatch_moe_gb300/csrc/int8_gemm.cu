// Grouped products of 8-bit integers with a scale for each row and each output channel, and the SwiGLU expert FFN made of two.
//
//   y[r, n] = (sum_k A[r, k] W[g, n, k]) * a_scale[r] * w_scale[g, n]     for the rows r of group g
#include <algorithm>
#include "int8.cuh"

namespace moe {
namespace int8 {

constexpr int MAX_G = 1024;

enum Epi : int { EPI_OUT = 0, EPI_SWIGLU = 1 };

struct Params {
    const int32_t* offsets;      // the groups' rows, or null: the tiles of `sched`
    const int32_t* sched;
    int G, rows, max_tiles;      // (groups and tiles: what a schedule has to agree with)
    const uint8_t* w;            // packed weight
    int NB, KST;                 // its 128-channel blocks and 64-column stages
    const void* a;               // operand codes [rows][64 KST]
    const float* a_scales;       // [rows]
    const float *w_scales, *w_scales_up;   // [G][N]; EPI_SWIGLU: of the gate and of the up channels [G][N / 2]
    int N;                       // output channels (EPI_SWIGLU: 2 F)
    long long ld;                // row stride of the output
    int out_dtype;
    void* out;                   // EPI_SWIGLU: act [rows][N / 2] fp32
    unsigned* err;
    long long wait_limit;
};

// The groups in shared memory: first[g] tiles of `tile` rows before group g (first[G]: all of them; 0 where offsets or schedule are
// no good), its rows [beg[g], end[g]). Read from L2: the offsets and the schedule are older than the kernel before this one, so
// they are read without waiting for it, when an L1 line of an earlier call's may still be there.
struct Groups { int *first, *beg, *end; };
constexpr int GROUPS_INTS = 3 * MAX_G + 1;
__device__ __forceinline__ Groups groups_at(int* smem) { return Groups{smem, smem + MAX_G + 1, smem + 2 * MAX_G + 1}; }

template <int NT>
__device__ __forceinline__ void find_groups(const Params& p, int tile, const Groups& gs) {
    constexpr int PER = (MAX_G + NT - 1) / NT;
    __shared__ int s_warp[NT / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g0 = threadIdx.x * PER;
    const bool by_tiles = p.offsets == nullptr;
    const int ntiles = by_tiles ? __ldcg(p.sched) : 0;
    const bool fits = !by_tiles || (__ldcg(p.sched + 1) == p.G && ntiles <= p.max_tiles);
    const int32_t* prefix = p.sched + kSchedHeader;
    const int4* tiles = reinterpret_cast<const int4*>(p.sched + sched_tiles_offset(p.G));
    int n[PER], sum = 0;
    bool bad = !fits;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = g0 + i;
        n[i] = 0;
        if (g < p.G && fits) {
            int lo, hi;
            if (by_tiles) {
                // the schedule's tiles are those of the group's rows, within the call
                const int t0 = __ldcg(prefix + g), t1 = __ldcg(prefix + g + 1);
                const bool some = 0 <= t0 && t0 < t1 && t1 <= ntiles;
                lo = some ? min(__ldcg(tiles + t0).y, p.rows) : 0;
                hi = some ? min(__ldcg(tiles + t1 - 1).z, p.rows) : 0;
                bad |= (some ? lo < 0 || (max(hi - lo, 0) + MOE_TILE_M - 1) / MOE_TILE_M != t1 - t0 : t0 != t1) || (g == 0 && t0 != 0) ||
                       (g == p.G - 1 && t1 != ntiles);
            } else {
                lo = __ldcg(p.offsets + g);
                hi = __ldcg(p.offsets + g + 1);
                bad |= lo < 0 || hi < lo || hi > p.rows;
            }
            gs.beg[g] = lo;
            gs.end[g] = hi;
            n[i] = hi > lo ? (hi - lo + tile - 1) / tile : 0;
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
    if (threadIdx.x == 0) gs.first[0] = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        at += n[i];
        if (g0 + i < p.G) gs.first[g0 + i + 1] = bad ? 0 : at;
    }
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) latch_device_error(p.err, kDevErrBadIndex, 0x320u);
    __syncthreads();
}
// The last group g from `g` on with before[g] * per <= w: steps that double (items rise), then halving.
__device__ __forceinline__ int group_of(const int* before, int G, int per, long long w, int g) {
    int hi = g + 1;
#pragma unroll 1
    for (int step = 1; hi < G && (long long)before[hi] * per <= w; step *= 2) {
        g = hi;
        hi = min(hi + step, G);
    }
#pragma unroll 1
    while (hi - g > 1) {
        const int mid = (g + hi) >> 1;
        if ((long long)before[mid] * per <= w) g = mid; else hi = mid;
    }
    return g;
}

__device__ __forceinline__ void store_value(const Params& p, long long at, float v) {
    if (p.out_dtype == MOE_F32) static_cast<float*>(p.out)[at] = v;
    else if (p.out_dtype == MOE_BF16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p.out)[at] = __float2half_rn(v);
}
// silu(g) u in fp32, each step rounded as the formula has it.
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + expf(-g)) * u; }

// ---------------------------------------------------------------------------------------------------
// few rows: integer dot products on the CUDA cores
// ---------------------------------------------------------------------------------------------------
// Where groups have few rows the weights' bytes decide. A block takes 32 channels (a lane each) of a group and up to 8 of its rows;
// its warps take the 64-column stages in turn, 16 bytes of weight a lane and load, the rows' codes the same for all lanes, and meet in
// shared memory: exact integer sums, whatever the order. Groups with more rows are passed over several times, the weights then coming
// from L2.
constexpr int FEW_THREADS = 256, FEW_WARPS = FEW_THREADS / 32, FEW_ROWS = 8, FEW_N = 32;

template <int NT>
__device__ __forceinline__ void few_dots(const uint8_t* w, const uint8_t* const (&a)[NT], int kst, int (&acc)[NT]) {
    const int warp = threadIdx.x >> 5;
    uint4 v[4];
    auto fetch = [&](int kb) {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = __ldcs(reinterpret_cast<const uint4*>(w + (size_t)kb * PIECE + c * (BLOCK_N * 16)));
    };
    if (warp < kst) fetch(warp);
#pragma unroll 1
    for (int kb = warp; kb < kst; kb += FEW_WARPS) {
        uint4 x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = make_uint4(v[c].x ^ 0x80808080u, v[c].y ^ 0x80808080u, v[c].z ^ 0x80808080u, v[c].w ^ 0x80808080u);
        if (kb + FEW_WARPS < kst) fetch(kb + FEW_WARPS);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint4 q = *reinterpret_cast<const uint4*>(a[t] + kb * STAGE_K + c * 16);
                acc[t] = __dp4a((int)x[c].x, (int)q.x, acc[t]);
                acc[t] = __dp4a((int)x[c].y, (int)q.y, acc[t]);
                acc[t] = __dp4a((int)x[c].z, (int)q.z, acc[t]);
                acc[t] = __dp4a((int)x[c].w, (int)q.w, acc[t]);
            }
        }
    }
}

template <int EPI>
__global__ void __launch_bounds__(FEW_THREADS, 2) few_rows_kernel(const Params p) {
    __shared__ int s_groups[GROUPS_INTS];
    __shared__ int s_sum[FEW_WARPS][FEW_ROWS][32];
    const Groups gs = groups_at(s_groups);
    find_groups<FEW_THREADS>(p, FEW_ROWS, gs);
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nch = (p.N + FEW_N - 1) / FEW_N, width = p.KST * STAGE_K;
    const long long items = (long long)gs.first[p.G] * nch;
    int g = 0;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        g = group_of(gs.first, p.G, nch, it, g);
        const int passes = gs.first[g + 1] - gs.first[g];
        const int local = (int)(it - (long long)gs.first[g] * nch), ch = local / passes, row0 = gs.beg[g] + (local - ch * passes) * FEW_ROWS;
        const int nt = min(FEW_ROWS, gs.end[g] - row0), n = ch * FEW_N + lane;
        const uint8_t* w = p.w + ((size_t)g * p.NB + (ch >> 2)) * p.KST * PIECE + ((ch & 3) * 32 + lane) * 16;
        const uint8_t* a0 = static_cast<const uint8_t*>(p.a) + (size_t)row0 * width;
        auto run = [&](auto rows) {
            constexpr int NT = decltype(rows)::value;
            const uint8_t* a[NT];
            int acc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                a[t] = a0 + (size_t)min(t, nt - 1) * width;
                acc[t] = 0;
            }
            few_dots<NT>(w, a, p.KST, acc);
#pragma unroll
            for (int t = 0; t < NT; ++t) s_sum[warp][t][lane] = acc[t];
        };
        if (nt <= 1) run(std::integral_constant<int, 1>());
        else if (nt <= 2) run(std::integral_constant<int, 2>());
        else if (nt <= 4) run(std::integral_constant<int, 4>());
        else run(std::integral_constant<int, 8>());
        __syncthreads();
        if (warp < nt) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < FEW_WARPS; ++i) sum += s_sum[i][warp][lane];
            const int row = row0 + warp;
            const float v = (float)sum * p.a_scales[row];
            if constexpr (EPI == EPI_OUT) {
                if (n < p.N) store_value(p, row * p.ld + n, v * p.w_scales[(size_t)g * p.N + n]);
            } else {
                const int F = p.N / 2, f = n >> 1;
                const float s = n < p.N ? ((n & 1) ? p.w_scales_up : p.w_scales)[(size_t)g * F + f] : 0.f;
                const float x = v * s, u = __shfl_down_sync(0xffffffffu, x, 1);
                if (!(n & 1) && n < p.N) static_cast<float*>(p.out)[(size_t)row * F + f] = swiglu(x, u);
            }
        }
        __syncthreads();
    }
}

static int launch_product(const Params& p, int epi, cudaStream_t s) {
    auto go = [&](auto kernel) {
        int per_sm = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, FEW_THREADS, 0) != cudaSuccess || per_sm < 1) per_sm = 1;
        const long long most = ((long long)cdiv(p.rows, FEW_ROWS) + std::min(p.G, p.rows)) * cdiv(p.N, FEW_N);
        return launch_pdl(kernel, dim3((unsigned)std::min<long long>(most, (long long)per_sm * num_sms())), dim3(FEW_THREADS), 0, s, p);
    };
    return check_launch(epi == EPI_OUT ? go(few_rows_kernel<EPI_OUT>) : go(few_rows_kernel<EPI_SWIGLU>), "int8 few_rows_kernel");
}

// A row operand in the workspace: codes (room for fp16), then the rows' scales.
static size_t operand_bytes(long long rows, int K) { return align_up((size_t)rows * pad64(K) * 2, 256) + align_up((size_t)rows * 4, 256); }
static float* scales_at(void* operand, long long rows, int K) {
    return reinterpret_cast<float*>(static_cast<char*>(operand) + align_up((size_t)rows * pad64(K) * 2, 256));
}

static bool sizes_ok(int G, int N, int K, int rows) {
    return G >= 1 && G <= MAX_G && N >= 1 && N <= MOE_INT8_MAX_K && K >= 1 && K <= MOE_INT8_MAX_K && rows >= 0 && rows <= MOE_INT8_MAX_ROWS;
}
static bool on(const void* p, unsigned a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

static int check_call(const char* fn, const void* x, long long ldx, int x_rows, const int32_t* src, const int32_t* offsets,
                      const int32_t* sched, const void* packed, int rows, int K, int N, int dtype, const void* out, long long ldo,
                      int out_dtype, const void* ws, size_t ws_bytes, size_t need) {
    const auto known = [](int d) { return d == MOE_F32 || d == MOE_BF16 || d == MOE_F16; };
    MOE_REQUIRE(known(dtype) && known(out_dtype), MOE_ERR_UNSUPPORTED, "%s: dtype %d, out_dtype %d", fn, dtype, out_dtype);
    MOE_REQUIRE(x_rows >= (src ? 0 : rows) && ldx >= K && ldo >= N, MOE_ERR_INVALID_ARG, "%s: x_rows=%d rows=%d ldx=%lld ldo=%lld", fn, x_rows,
                rows, ldx, ldo);
    MOE_REQUIRE((offsets != nullptr) != (sched != nullptr), MOE_ERR_INVALID_ARG, "%s: one of offsets and tile_sched", fn);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE((x || x_rows == 0) && packed && out, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    MOE_REQUIRE(on(x, dtype == MOE_F32 ? 4 : 2) && on(out, out_dtype == MOE_F32 ? 4 : 2) && on(packed, 16) && on(src, 4) && on(offsets, 4) &&
                    on(sched, 16),
                MOE_ERR_INVALID_ARG, "%s: misaligned pointer", fn);
    MOE_REQUIRE(ws && on(ws, 256) && ws_bytes >= need, MOE_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes (256-byte aligned)", fn, ws_bytes, need);
    return MOE_OK;
}

}  // namespace int8
}  // namespace moe

using namespace moe;

extern "C" size_t moe_int8_linear_workspace_size(int G, int N, int K, int rows) {
    return int8::sizes_ok(G, N, K, rows) ? std::max<size_t>(int8::operand_bytes(rows, K), 256) : 0;
}

extern "C" int moe_int8_linear(const void* x, long long ldx, int x_rows, const int32_t* src, const int32_t* offsets,
                               const int32_t* tile_sched, const void* packed, const float* w_scales, int G, int N, int K, int rows,
                               int dtype, void* out, long long ldo, int out_dtype, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "moe_int8_linear";
    MOE_REQUIRE(int8::sizes_ok(G, N, K, rows), MOE_ERR_INVALID_ARG, "%s: G=%d N=%d K=%d rows=%d", fn, G, N, K, rows);
    if (int rc = int8::check_call(fn, x, ldx, x_rows, src, offsets, tile_sched, packed, rows, K, N, dtype, out, ldo, out_dtype, ws, ws_bytes,
                                  moe_int8_linear_workspace_size(G, N, K, rows)))
        return rc;
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(w_scales && int8::on(w_scales, 4), MOE_ERR_INVALID_ARG, "%s: null or misaligned scales", fn);
    unsigned* err = device_error_word();
    MOE_REQUIRE(err, MOE_ERR_CUDA, "%s: device error word unavailable", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int8::WeightLayout L = int8::weight_layout(G, N, K);
    int8::Params p{};
    p.offsets = offsets; p.sched = tile_sched; p.G = G; p.rows = rows; p.max_tiles = (int)sched_max_tiles(rows, G);
    p.w = static_cast<const uint8_t*>(packed); p.NB = L.NB; p.KST = L.KST;
    p.a = ws; p.a_scales = int8::scales_at(ws, rows, K);
    p.w_scales = w_scales; p.N = N; p.ld = ldo; p.out_dtype = out_dtype; p.out = out;
    p.err = err; p.wait_limit = wait_limit();
    if (int rc = int8::launch_quantize(x, ldx, x_rows, src, rows, K, dtype, int8::FORM_BYTES, ws, int8::scales_at(ws, rows, K), err, s)) return rc;
    return int8::launch_product(p, int8::EPI_OUT, s);
}

// The FFN's workspace: x's operand, act [rows][F] in fp32, act's operand.
namespace moe {
namespace int8 {
struct FfnWs { char* x; float* act; char* a; size_t bytes; };
static FfnWs ffn_ws(void* ws, int h, int F, long long rows) {
    FfnWs w{};
    char* base = static_cast<char*>(ws);
    w.x = base;
    size_t off = operand_bytes(rows, h);
    w.act = reinterpret_cast<float*>(base + off);
    off = align_up(off + (size_t)rows * F * 4, 256);
    w.a = base + off;
    w.bytes = off + operand_bytes(rows, F);
    return w;
}
}  // namespace int8
}  // namespace moe

extern "C" size_t moe_int8_expert_ffn_workspace_size(int E, int h, int F, int rows) {
    if (!int8::sizes_ok(E, F, h, rows) || F > MOE_INT8_MAX_K / 2) return 0;
    return std::max<size_t>(int8::ffn_ws(nullptr, h, F, rows).bytes, 256);
}

extern "C" int moe_int8_expert_ffn(const void* x, long long ldx, int x_rows, const int32_t* src, const int32_t* offsets,
                                   const int32_t* tile_sched, const void* packed, const float* gate_scales, const float* up_scales,
                                   const float* down_scales, int E, int h, int F, int rows, int dtype, void* out, long long ldo,
                                   int out_dtype, void* ws, size_t ws_bytes, void* stream) {
    const char* fn = "moe_int8_expert_ffn";
    MOE_REQUIRE(int8::sizes_ok(E, F, h, rows) && F <= MOE_INT8_MAX_K / 2, MOE_ERR_INVALID_ARG, "%s: E=%d h=%d F=%d rows=%d", fn, E, h, F, rows);
    if (int rc = int8::check_call(fn, x, ldx, x_rows, src, offsets, tile_sched, packed, rows, h, h, dtype, out, ldo, out_dtype, ws, ws_bytes,
                                  moe_int8_expert_ffn_workspace_size(E, h, F, rows)))
        return rc;
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE(gate_scales && up_scales && down_scales && int8::on(gate_scales, 4) && int8::on(up_scales, 4) && int8::on(down_scales, 4),
                MOE_ERR_INVALID_ARG, "%s: null or misaligned scales", fn);
    unsigned* err = device_error_word();
    MOE_REQUIRE(err, MOE_ERR_CUDA, "%s: device error word unavailable", fn);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int8::ExpertLayout L = int8::expert_layout(E, h, F);
    const int8::FfnWs w = int8::ffn_ws(ws, h, F, rows);
    int8::Params p{};
    p.offsets = offsets; p.sched = tile_sched; p.G = E; p.rows = rows; p.max_tiles = (int)sched_max_tiles(rows, E);
    p.w = static_cast<const uint8_t*>(packed); p.NB = L.gu.NB; p.KST = L.gu.KST;
    p.a = w.x; p.a_scales = int8::scales_at(w.x, rows, h);
    p.w_scales = gate_scales; p.w_scales_up = up_scales; p.N = 2 * F; p.out_dtype = MOE_F32; p.out = w.act;
    p.err = err; p.wait_limit = wait_limit();
    if (int rc = int8::launch_quantize(x, ldx, x_rows, src, rows, h, dtype, int8::FORM_BYTES, w.x, int8::scales_at(w.x, rows, h), err, s)) return rc;
    if (int rc = int8::launch_product(p, int8::EPI_SWIGLU, s)) return rc;
    if (int rc = int8::launch_quantize(w.act, F, rows, nullptr, rows, F, MOE_F32, int8::FORM_BYTES, w.a, int8::scales_at(w.a, rows, F), err, s))
        return rc;
    p.w += L.down_off; p.NB = L.down.NB; p.KST = L.down.KST;
    p.a = w.a; p.a_scales = int8::scales_at(w.a, rows, F);
    p.w_scales = down_scales; p.w_scales_up = nullptr; p.N = h; p.ld = ldo; p.out_dtype = out_dtype; p.out = out;
    return int8::launch_product(p, int8::EPI_OUT, s);
}
