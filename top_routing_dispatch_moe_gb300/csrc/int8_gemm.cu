// Grouped products of 8-bit integers with a scale for each row and each output channel, and the SwiGLU expert FFN made of two.
//
//   y[r, n] = (sum_k A[r, k] W[g, n, k]) * a_scale[r] * w_scale[g, n]     for the rows r of group g
#include <algorithm>
#include "int8.cuh"
#include "tc_elect.cuh"
#include "tc_map.cuh"

namespace moe {
namespace int8 {
using namespace moe::tc;

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
    void* out;                   // EPI_SWIGLU: act [rows][N / 2] fp32, its rows ld apart as well
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
// few rows: weights through shared memory to mma.sync
// ---------------------------------------------------------------------------------------------------
// Where groups have few rows the weights' bytes decide, and the way through tensor memory is the limit: each tcgen05.mma of 16 columns
// reads its 4 KB of converted weights at the rate that 256 rows need, 128 cycles, however few rows there are (16 bytes of weights a cycle
// and SM, 5.1 TB/s in all: 128 groups of 4 rows by 1536 x 2048 in 83 us). Here a lane takes 16 bytes of a channel from shared memory, makes
// them fp16 as above and has them as a fragment of mma.sync.m16n8k16 (16 channels x 8 rows; the order of the columns within a piece is the
// same for both operands). (Loaded straight into registers, two pieces ahead, the weights came at 3.3 TB/s: too few under way.)
//
// A persistent CTA per SM: one warp brings stages of 128 columns, 16 KB of weights of 128 channels and up to 16 rows' codes, eight of them under
// way; four groups of four warps, 32 channels to a warp, take them in turn (where every warp took a part of every stage, the waits and arrivals on
// the stages' barriers cost more than the work). Their sums meet in shared memory in a fixed order. Groups with
// more rows are passed over several times, the weights then coming from L2.
//
// SPLIT: where that leaves most SMs without a tile, a cluster of two to eight CTAs takes one, each a share of its columns (a tile of
// 6528 columns is 51 stages by one SM); the CTAs' sums meet through distributed shared memory, in their order, each finishing some of the rows.
constexpr int FEW_ROWS = 16, FEW_STAGES = 8, FEW_GROUPS = 4, FEW_WARPS = 4 * FEW_GROUPS, FEW_THREADS = 32 * (1 + FEW_WARPS);
constexpr int FEW_PITCH = 33;                    // words of a row's 32 channels in shared memory
constexpr int FEW_X_BYTES = FEW_ROWS * STAGE_K * 2, FEW_STAGE = 2 * (PIECE + FEW_X_BYTES);
constexpr int FEW_SUM = 4 * FEW_ROWS * FEW_PITCH, FEW_SUM_BYTES = FEW_GROUPS * FEW_SUM * 4;
constexpr int FEW_SMEM = 1024 + FEW_STAGES * FEW_STAGE + FEW_SUM_BYTES + 256 + GROUPS_INTS * 4 + 16;
static_assert(FEW_SMEM <= 227 * 1024, "shared memory per CTA");
// A stage of the ring is one group's in every round: a warp that waits for a round of it has seen the round before, and the barrier's
// parity, all that a wait asks for, cannot be that of two rounds ago.
static_assert(FEW_STAGES % FEW_GROUPS == 0, "stages of a group");

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four packed bytes -> two pairs of fp16 numbers: a byte under 0x64 is 1024 + byte, byte = code + 128.
__device__ __forceinline__ void halves4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const __half2 off = __float2half2_rn(-1152.f);
    const uint32_t l = __byte_perm(w, 0x64646464u, 0x4140), h = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&l), off), b = __hadd2(*reinterpret_cast<const __half2*>(&h), off);
    lo = *reinterpret_cast<const uint32_t*>(&a);
    hi = *reinterpret_cast<const uint32_t*>(&b);
}
// A barrier of the groups' warps, and whether any of their threads says so.
__device__ __forceinline__ bool few_any(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((uint32_t)v), "n"(32 * FEW_WARPS) : "memory");
    return r != 0;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

struct FewRing {
    uint32_t sW, sX, bar0;
    volatile int* abort_flag;
    int stage;
    uint32_t phase;
    __device__ __forceinline__ uint32_t full(int s) const { return bar0 + 8u * s; }
    __device__ __forceinline__ uint32_t empty(int s) const { return bar0 + 8u * (FEW_STAGES + s); }
};

// One tile by one warp: the sums of its 32 channels x 8 NT rows over its group's stages of kb0 .. kb1 - 1, into `sum` [group][8 NT][FEW_PITCH] beside those of
// the other groups, all of which are there on return. False: a wait ran out in some warp.
template <int NT>
__device__ __forceinline__ bool few_tile(const Params& p, FewRing& ring, int quarter, int group, float* sum, int kb0, int kb1) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.f;
    // chunk t of channel r is at row r ^ 2 t of the chunk (of eight lanes, two channels and four chunks, no two on a bank); r = 32 quarter + g + 8 i
    const uint32_t wat = (uint32_t)(t * BLOCK_N + ((quarter * 32 + g) ^ (2 * t))) * 16, xat = (uint32_t)(g * 128);
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
        const int st = ring.stage;
        const uint32_t ph = ring.phase;
        if (++ring.stage == FEW_STAGES) { ring.stage = 0; ring.phase ^= 1u; }
        if (st % FEW_GROUPS != group || !ok) continue;
        ok = wait_warp(ring.full(st), ph, p.wait_limit, ring.abort_flag, p.err, 0x382u);
        if (!ok) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (2 * kb + h >= p.KST) break;
            uint32_t w[4][4], x[NT][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) ld_shared_v4(ring.sW + (st * 2 + h) * PIECE + wat + i * 128, w[i]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint32_t at = ring.sX + (st * 2 + h) * FEW_X_BYTES + xat + n * 1024;
                ld_shared_v4(at + ((uint32_t)((2 * t) ^ g) << 4), x[n]);
                ld_shared_v4(at + ((uint32_t)((2 * t + 1) ^ g) << 4), x[n] + 4);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t f[4];
                    halves4(w[2 * m][s], f[0], f[2]);
                    halves4(w[2 * m + 1][s], f[1], f[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) mma_f16(acc[m][n], f, x[n][2 * s], x[n][2 * s + 1]);
                }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.empty(st));
    }
    auto at = [&](int m, int n, int i) { return (8 * n + 2 * t + (i & 1)) * FEW_PITCH + 16 * m + g + 8 * (i >> 1); };
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[group * FEW_SUM + at(m, n, i)] = acc[m][n][i];
    return !few_any(!ok);
}

template <int EPI, bool SPLIT>
__global__ void __launch_bounds__(FEW_THREADS, 1) few_rows_kernel(const __grid_constant__ CUtensorMap tm16, const Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    FewRing ring;
    ring.sX = smem_u32(smem);
    ring.sW = ring.sX + FEW_STAGES * 2 * FEW_X_BYTES;
    float* s_sum = reinterpret_cast<float*>(smem + FEW_STAGES * FEW_STAGE);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + FEW_STAGES * FEW_STAGE + FEW_SUM_BYTES);
    ring.bar0 = smem_u32(bars);
    ring.abort_flag = reinterpret_cast<volatile int*>(bars + 2 * FEW_STAGES);
    ring.stage = 0;
    ring.phase = 0;
    const Groups gs = groups_at(reinterpret_cast<int*>(bars + 32));
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < FEW_STAGES; ++s) { mbar_init(ring.full(s), 1); mbar_init(ring.empty(s), 4); }
        *ring.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&tm16);
    }
    // (a programmatic dependent of the quantisation: the groups, the set-up and the first stages of weights do not wait for it)
    find_groups<FEW_THREADS>(p, FEW_ROWS, gs);               // (its barriers also stand between the set-up and the roles)
    const int total = uniform(gs.first[p.G] * p.NB), ns = (p.KST + 1) / 2;
    // SPLIT: a cluster has one item at most, and whatever becomes of it, every thread meets the two barriers of the cluster
    const int ranks = SPLIT ? (int)cluster_size() : 1, rank = SPLIT ? (int)cluster_rank() : 0;
    const int first = (int)blockIdx.x / ranks, step = SPLIT ? total : (int)gridDim.x;
    if (SPLIT && total > (int)gridDim.x / ranks && blockIdx.x == 0 && threadIdx.x == 0)       // (a schedule whose groups overlap)
        latch_device_error(p.err, kDevErrBadIndex, 0x322u);
    const int kb0 = ns * rank / ranks, kb1 = ns * (rank + 1) / ranks;      // (ns * ranks: at most 1024 * 8)
    // Item w: group by group, 128-channel block next, row tile fastest
    auto map = [&](int w, int& g, int& nb, int& row0, int& row1) {
        g = group_of(gs.first, p.G, p.NB, w, g);
        const int nt = gs.first[g + 1] - gs.first[g], local = w - gs.first[g] * p.NB;
        nb = local / nt;
        row0 = gs.beg[g] + (local - nb * nt) * FEW_ROWS;
        row1 = min(row0 + FEW_ROWS, gs.end[g]);
    };
    if (warp == FEW_WARPS) {
        int stage = 0, g = 0;
        uint32_t phase = 0, issued = 0, last_par = 0;
        bool ok = true;
        for (int w = first; w < total && ok; w += step) {
            int nb, row0, row1;
            map(w, g, nb, row0, row1);
            nb = uniform(nb); row0 = uniform(row0);
            const uint8_t* w0 = p.w + ((size_t)uniform(g) * p.NB + nb) * p.KST * PIECE;
            auto weights = [&](int st, int kb) {
                const int n = min(2, p.KST - 2 * kb);
                expect_elected(ring.full(st), (uint32_t)(n * (PIECE + FEW_X_BYTES)));
                bulk_elected(ring.sW + st * (2 * PIECE), w0 + (size_t)kb * (2 * PIECE), n * PIECE, ring.full(st));
            };
            int early = 0;
            if (w == first) {
                for (; early < min(FEW_STAGES, kb1 - kb0); ++early) weights(early, kb0 + early);
                pdl_wait();
                pdl_trigger();
            }
            for (int kb = kb0; kb < kb1; ++kb) {
                if (kb >= kb0 + early) {
                    ok = test_warp(ring.empty(stage), phase ^ 1u) ||
                         wait_warp(ring.empty(stage), phase ^ 1u, p.wait_limit, ring.abort_flag, p.err, 0x380u);
                    if (!ok) break;
                    weights(stage, kb);
                }
                for (int q = 0; q < min(2, p.KST - 2 * kb); ++q)
                    tma_elected(ring.sX + (stage * 2 + q) * FEW_X_BYTES, &tm16, (2 * kb + q) * STAGE_K, row0, ring.full(stage));
                issued |= 1u << stage;
                last_par = (last_par & ~(1u << stage)) | (phase << stage);
                if (++stage == FEW_STAGES) { stage = 0; phase ^= 1u; }
            }
        }
        if (total <= first) {                    // (no item: the wait that every thread makes)
            pdl_wait();
            pdl_trigger();
        }
        if (lane == 0)
            for (int s = 0; s < FEW_STAGES; ++s)    // every issued copy has landed before the CTA exits
                if (issued & (1u << s)) drain_phase(ring.full(s), (last_par >> s) & 1u, p.err, 0x381u);
        __syncwarp();
        if constexpr (SPLIT) {
            cluster_sync_all();
            cluster_sync_all();
        }
        return;
    }
    pdl_wait();
    pdl_trigger();
    const int quarter = warp & 3, group = warp >> 2;
    int g = 0;
    if constexpr (SPLIT) {
        const bool some = first < total;
        int nb = 0, row0 = 0, row1 = 0;
        if (some) map(first, g, nb, row0, row1);
        const int nt = row1 - row0, n = nb * BLOCK_N + quarter * 32 + lane, F = p.N / 2, f = n >> 1;
        float* sum = s_sum + quarter * (FEW_ROWS * FEW_PITCH);
        float scale = 0.f;
        if (some && n < p.N) scale = EPI == EPI_OUT ? p.w_scales[(size_t)g * p.N + n] : ((n & 1) ? p.w_scales_up : p.w_scales)[(size_t)g * F + f];
        bool ok = false;
        if (some) ok = nt <= 8 ? few_tile<1>(p, ring, quarter, group, sum, kb0, kb1) : few_tile<2>(p, ring, quarter, group, sum, kb0, kb1);
        cluster_sync_all();                      // every CTA's sums are there
        if (ok && n - lane < p.N) {
            for (int t = rank + ranks * group; t < nt; t += ranks * FEW_GROUPS) {
                const float xs = p.a_scales[row0 + t];
                float v = 0.f;
                for (int r = 0; r < ranks; ++r) {
                    const uint32_t at = map_rank(smem_u32(sum + t * FEW_PITCH + lane), r);
#pragma unroll
                    for (int j = 0; j < FEW_GROUPS; ++j) v += ld_cluster(at + j * (FEW_SUM * 4));
                }
                v = v * xs * scale;
                if constexpr (EPI == EPI_OUT) {
                    if (n < p.N) store_value(p, (row0 + t) * p.ld + n, v);
                } else {
                    const float u = __shfl_down_sync(0xffffffffu, v, 1);
                    if (!(n & 1) && n < p.N) static_cast<float*>(p.out)[(row0 + t) * p.ld + f] = swiglu(v, u);
                }
            }
        }
        cluster_sync_all();                      // and have been read
        return;
    }
    for (int w = blockIdx.x; w < total; w += gridDim.x) {
        int nb, row0, row1;
        map(w, g, nb, row0, row1);
        const int nt = row1 - row0, n = nb * BLOCK_N + quarter * 32 + lane;
        float* sum = s_sum + quarter * (FEW_ROWS * FEW_PITCH);
        // (what the sums are multiplied with, under way while they are formed: loaded after them, it cost a tile of 768 columns a third of its
        // time)
        const int F = p.N / 2, f = n >> 1;
        float scale = 0.f, xs[FEW_ROWS / FEW_GROUPS];
        if (n < p.N) scale = EPI == EPI_OUT ? p.w_scales[(size_t)g * p.N + n] : ((n & 1) ? p.w_scales_up : p.w_scales)[(size_t)g * F + f];
#pragma unroll
        for (int i = 0; i < FEW_ROWS / FEW_GROUPS; ++i) xs[i] = p.a_scales[row0 + min(group + i * FEW_GROUPS, nt - 1)];
        const bool ok = nt <= 8 ? few_tile<1>(p, ring, quarter, group, sum, 0, ns) : few_tile<2>(p, ring, quarter, group, sum, 0, ns);
        if (!ok) break;
        if (n - lane < p.N) {                    // 32 channels of the group's share of the rows
#pragma unroll
            for (int i = 0; i < FEW_ROWS / FEW_GROUPS; ++i) {
                const int t = group + i * FEW_GROUPS, row = row0 + t;
                if (t >= nt) break;
                float v = 0.f;
#pragma unroll
                for (int j = 0; j < FEW_GROUPS; ++j) v += sum[j * FEW_SUM + t * FEW_PITCH + lane];
                v = v * xs[i] * scale;
                if constexpr (EPI == EPI_OUT) {
                    if (n < p.N) store_value(p, row * p.ld + n, v);
                } else {
                    const float u = __shfl_down_sync(0xffffffffu, v, 1);
                    if (!(n & 1) && n < p.N) static_cast<float*>(p.out)[row * p.ld + f] = swiglu(v, u);
                }
            }
        }
        if (w + (int)gridDim.x < total) few_any(false);      // the sums are read before the next tile's are written
    }
}

// ---------------------------------------------------------------------------------------------------
// many rows: fp16 tensor-core products of whole numbers, two SMs to a tile
// ---------------------------------------------------------------------------------------------------
// The chip's tensor cores have no integer kind. Whole numbers up to 2^11 are fp16 numbers, their products are exact in fp32, and so are
// sums below 2^24: the rows' codes are kept as fp16 (written so by the quantisation), the weights stay bytes in memory and become fp16
// on the chip, on their way into tensor memory, from where tcgen05.mma takes its first operand. The product is turned over for that:
// the channels are its rows (M) and a group's rows its columns (N), which also fits N to the group: 32 to 256 in steps of 32.
//
// A cluster of two CTAs computes 256 channels x up to ROWS rows with tcgen05.mma.cta_group::2: each converts its own 128 channels and
// stages half of the rows. A persistent CTA per SM with eighteen warps:
//   warp 0      producer: per stage of 128 columns 16 KB of packed weight by one bulk copy, and the CTA's half of the rows by TMA;
//   warp 1      (of the even CTA) the MMAs of a stage;
//   warps 2-9   epilogue, two to a quarter of the tensor memory lanes, 64 columns at a time in turn: a lane is a channel, a column a row
//               of the output; SwiGLU's gate and up are neighbouring lanes and exchange halves;
//   warps 10-17 converters, two to a quarter, stages in turn: a lane reads its channel's 64 bytes, puts each under 0x64 (the fp16 number
//               1024 + byte), subtracts 1152 and stores 32 columns of tensor memory, twice a stage.
// Tensor memory: two accumulators of 256 columns that share 128 (the epilogue reads the shared ones first and hands them back), and two
// stages of converted weights, 64 columns each.
//
// ROWS, the most rows of a tile: 256 where groups have many; 128 and 64 leave more of the shared memory to stages under way where
// the weights' bytes decide (64 KB of weights under way on an SM brought 3.8 TB/s, whatever the stages' size), and tensor memory to
// accumulators that share nothing and four stages of converted weights.
constexpr int EPI_WARPS = 8, CONV_WARPS = 8;
constexpr int P_THREADS = 32 * (2 + EPI_WARPS + CONV_WARPS);
constexpr int PER = 2;                                         // packed pieces (64 columns) of a stage
constexpr int A_COLS = PER * STAGE_K / 2;                      // tensor memory columns of a stage of converted weights
constexpr int TMEM_COLS = 512;
template <int ROWS>
struct Tile {
    static constexpr int STAGES = ROWS == 256 ? 4 : ROWS == 128 ? 6 : 8;
    static constexpr int X_BYTES = ROWS / 2 * STAGE_K * 2;     // the rows' 64 columns that go with a piece
    static constexpr int STAGE_BYTES = PER * (PIECE + X_BYTES);
    static constexpr int ACC2 = ROWS == 256 ? 128 : ROWS;      // the second accumulator's first column
    static constexpr int A_BUFS = ROWS == 256 ? 2 : 4, A_COL = ACC2 + ROWS;
    static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + 256 + GROUPS_INTS * 4 + 16;
    static_assert(A_COL + A_BUFS * A_COLS <= TMEM_COLS, "tensor memory columns");
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
    static_assert(8 * (2 * STAGES + A_BUFS + 3) + 8 <= 256, "barriers");
    static_assert(STAGES % 2 == 0 && A_BUFS % 2 == 0, "a stage and a buffer are the same converters' in every round");
};

// D fp32 (bits 4-5 = 1), A and B fp16 (0), K-major, N >> 3 at bits 17-22, M = 256 at bits 24-28.
__device__ __forceinline__ uint32_t idesc_pair(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((256u >> 4) << 24); }
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                 "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
                 "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]),
                 "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]) : "memory");
}

// Item w: group by group, 256-channel tile next, row tile fastest: pairs that run together share a weight tile. A group's row tiles
// are of one size, a multiple of 32 (the last may be shorter).
struct Item { int g, ch, row0, row1; };
__device__ __forceinline__ Item map_item(const Params& p, const Groups& gs, int CT, int w, int& g) {
    g = group_of(gs.first, p.G, CT, w, g);
    const int nt = gs.first[g + 1] - gs.first[g], local = w - gs.first[g] * CT, ch = local / nt, t = local - ch * nt;
    const int n = gs.end[g] - gs.beg[g], per = ((n + nt - 1) / nt + 31) & ~31;
    return Item{g, ch, gs.beg[g] + t * per, gs.beg[g] + min(n, t * per + per)};
}

// COLS columns of the accumulator at tcol, the rows row0 .. of the output (n of them, at least one); this lane's channel is `ch`. `read`
// runs once the columns are in registers.
template <int EPI, int COLS, typename Fn>
__device__ __forceinline__ void epilogue_chunk(const Params& p, int g, uint32_t tcol, int ch, int row0, int n, float scale, Fn read) {
    const int lane = threadIdx.x & 31;
    const bool mine = ch < p.N;
#pragma unroll
    for (int h = 0; h < COLS / 32; ++h) {
        float v[32];
        tmem_ld32(tcol + 32 * h, v);
        if (h == COLS / 32 - 1) read();
        const int r0 = row0 + 32 * h, nr = n - 32 * h;
        if (nr <= 0) continue;
        const float xs = lane < nr ? p.a_scales[r0 + lane] : 0.f;
        if constexpr (EPI == EPI_OUT) {
            const int el = p.out_dtype == MOE_F32 ? 4 : 2;
            uint8_t* at = static_cast<uint8_t*>(p.out) + ((size_t)r0 * p.ld + ch) * el;
            const size_t step = (size_t)p.ld * el;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float y = v[j] * __shfl_sync(0xffffffffu, xs, j) * scale;
                if (mine && j < nr) {
                    if (p.out_dtype == MOE_F32) *reinterpret_cast<float*>(at) = y;
                    else if (p.out_dtype == MOE_BF16) *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(y);
                    else *reinterpret_cast<__half*>(at) = __float2half_rn(y);
                }
                at += step;
            }
        } else {
            // even lanes hold gates, odd lanes the ups of the same features: of two rows, the even lane finishes the first
            const int odd = lane & 1;
            float* at = static_cast<float*>(p.out) + (r0 + odd) * p.ld + (ch >> 1);
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float y0 = v[j] * __shfl_sync(0xffffffffu, xs, j) * scale, y1 = v[j + 1] * __shfl_sync(0xffffffffu, xs, j + 1) * scale;
                const float got = __shfl_xor_sync(0xffffffffu, odd ? y0 : y1, 1);
                const float a = swiglu(odd ? got : y0, odd ? y1 : got);
                if (mine && j + odd < nr) *at = a;
                at += 2 * p.ld;
            }
        }
    }
}

template <int EPI, int ROWS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(P_THREADS, 1)
pair_kernel(const __grid_constant__ CUtensorMap tm128, const __grid_constant__ CUtensorMap tm16, const Params p) {
    using C = Tile<ROWS>;
    constexpr int STAGES = C::STAGES, A_BUFS = C::A_BUFS, X_BYTES = C::X_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sX = smem_u32(smem), sW = sX + STAGES * PER * X_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto afull = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    const uint32_t tfull = bar0 + 8u * (2 * STAGES + A_BUFS), tempty = tfull + 8u, mma_done = tempty + 8u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + A_BUFS + 3);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const Groups gs = groups_at(reinterpret_cast<int*>(bars + 32));

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
        for (int b = 0; b < A_BUFS; ++b) mbar_init(afull(b), 2 * 4);
        mbar_init(tfull, 1);
        mbar_init(tempty, 2 * EPI_WARPS);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&tm128);
        prefetch_tmap(&tm16);
    }
    // (a programmatic dependent of the quantisation: the groups, the set-up and the first stages of weights do not wait for it)
    find_groups<P_THREADS>(p, ROWS, gs);
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tc_fence_before();
    cluster_sync_all();                          // barriers initialised and both CTAs' tensor memory allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t peer_abort = map_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u);
    const int CT = (p.NB + 1) >> 1, NC = gridDim.x >> 1, cid = blockIdx.x >> 1, total = uniform(gs.first[p.G] * CT);
    const int NS = (p.KST + PER - 1) / PER;      // stages of a tile
    if (warp != 0) {
        pdl_wait();
        pdl_trigger();
    }

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0, issued = 0, last_par = 0;
        bool ok = true, ready = false;              // ready: the next ring stage was seen free
        int at = 0;
        for (int w = cid; w < total && ok; w += NC) {
            const Item it = map_item(p, gs, CT, w, at);
            const int half = uniform(((it.row1 - it.row0 + 31) & ~31) >> 1), row = uniform(it.row0) + (int)rank * half;
            const int nb = uniform(2 * it.ch + (int)rank);
            const bool some = nb < p.NB;             // (the odd CTA of the last tile may have no channels)
            const uint8_t* w0 = p.w + ((size_t)uniform(it.g) * p.NB + nb) * p.KST * PIECE;
            const int tx = half * STAGE_K * 2 + (some ? PIECE : 0);
            auto weights = [&](int st, int kb) {
                const int n = min(PER, p.KST - kb * PER);
                expect_elected(full(st), (uint32_t)(n * tx));
                if (some) bulk_elected(sW + st * PER * PIECE, w0 + (size_t)kb * PER * PIECE, n * PIECE, full(st));
            };
            int early = 0;                          // stages whose weights are on their way before the rows' codes are there
            if (w == cid) {
                for (; early < min(STAGES, NS); ++early) weights(early, early);
                pdl_wait();
                pdl_trigger();
            }
            for (int kb = 0; kb < NS; ++kb) {
                if (kb >= early) {
                    if (!ready) ok = wait_warp_pair(empty(stage), phase ^ 1u, p.wait_limit, abort_flag, peer_abort, p.err, 0x340u);
                    if (!ok) break;
                    weights(stage, kb);
                }
                const uint32_t f = full(stage);
                for (int q = 0; q < min(PER, p.KST - kb * PER); ++q) {
                    const uint32_t sx = sX + (stage * PER + q) * X_BYTES;
                    const int k = (kb * PER + q) * STAGE_K;
                    if (ROWS == 256 && half == 128) tma_elected(sx, &tm128, k, row, f);
                    else
                        for (int b = 0; b < half; b += 16) tma_elected(sx + b * 128, &tm16, k, row + b, f);
                }
                issued |= 1u << stage;
                last_par = (last_par & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                ready = kb + 1 >= early && test_warp(empty(stage), phase ^ 1u);
            }
        }
        if (total <= cid) {                          // (no item: the wait that every thread makes)
            pdl_wait();
            pdl_trigger();
        }
        if (lane == 0)
            for (int s = 0; s < STAGES; ++s)        // every issued copy has landed before the CTA exits
                if (issued & (1u << s)) drain_phase(full(s), (last_par >> s) & 1u, p.err, 0x341u);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            int stage = 0, b = 0, iter = 0, at = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true, ready = false;
            for (int w = cid; w < total && ok; w += NC, ++iter) {
                const Item it = map_item(p, gs, CT, w, at);
                const uint32_t id = idesc_pair(uniform((it.row1 - it.row0 + 31) & ~31)), d = tm + (iter & 1) * C::ACC2;
                for (int kb = 0; kb < NS; ++kb) {
                    if (!ready)
                        ok = (kb > 0 || wait_warp_pair(tempty, (iter & 1) ^ 1u, p.wait_limit, abort_flag, peer_abort, p.err, 0x350u)) &&
                             wait_warp_pair(afull(b), bphase, p.wait_limit, abort_flag, peer_abort, p.err, 0x351u) &&
                             (test_warp(full(stage), phase) ||
                              wait_warp_pair(full(stage), phase, p.wait_limit, abort_flag, peer_abort, p.err, 0x352u));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t s0 = stage, a = tm + C::A_COL + b * A_COLS;
                    const bool last = kb + 1 == NS, both = (kb + 1) * PER <= p.KST;
                    const uint64_t db = sw128_desc(sX + s0 * PER * X_BYTES), db1 = sw128_desc(sX + (s0 * PER + 1) * X_BYTES);
                    mma_pair(d, a, db, id, kb != 0);
                    mma_pair(d, a + 8, db + 2, id, 1u);
                    mma_pair(d, a + 16, db + 4, id, 1u);
                    mma_pair(d, a + 24, db + 6, id, 1u);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (++b == A_BUFS) { b = 0; bphase ^= 1u; }
                    const bool t0 = test_phase(full(stage), phase), t1 = test_phase(afull(b), bphase);
                    if (both) {
                        mma_pair(d, a + 32, db1, id, 1u);
                        mma_pair(d, a + 40, db1 + 2, id, 1u);
                        mma_pair(d, a + 48, db1 + 4, id, 1u);
                        mma_pair(d, a + 56, db1 + 6, id, 1u);
                    }
                    commit_pair_elected(empty(s0));
                    if (last) commit_pair_elected(tfull);
                    ready = __all_sync(0xffffffffu, t0 && t1 && !last);
                }
            }
            commit_pair_elected(mma_done);          // both CTAs learn when every MMA has finished
        }
    } else if (warp >= 2 + EPI_WARPS) {
        const int quarter = 32 * (warp & 3), turn = (warp - 2 - EPI_WARPS) >> 2;
        const uint32_t afull0 = map_rank(afull(0), 0);
        int i = 0;                                  // stages so far, this CTA's in all
        bool ok = true;
        for (int w = cid; w < total && ok; w += NC) {
            for (int kb = 0; kb < NS; ++kb, ++i) {
                if ((i & 1) != turn) continue;
                const int st = i % STAGES, b = i % A_BUFS, old = (i - A_BUFS) % STAGES;
                ok = test_warp(full(st), (i / STAGES) & 1) ||
                     wait_warp_pair(full(st), (i / STAGES) & 1, p.wait_limit, abort_flag, peer_abort, p.err, 0x360u);
                if (!ok) break;
                const int n = min(PER, p.KST - kb * PER);
#pragma unroll
                for (int h = 0; h < PER; ++h) {
                    if (h >= n) break;
                    uint32_t q[16], v[32];
                    const uint32_t src = sW + (st * PER + h) * PIECE + quarter * 16;
#pragma unroll
                    for (int c = 0; c < 4; ++c) ld_shared_v4(src + c * (BLOCK_N * 16) + (lane ^ (2 * c)) * 16, q + 4 * c);
#pragma unroll
                    for (int c = 0; c < 16; ++c) halves4(q[c], v[2 * c], v[2 * c + 1]);
                    if (h == 0 && i >= A_BUFS) {    // the buffer's last MMAs have completed
                        const uint32_t par = ((i - A_BUFS) / STAGES) & 1;
                        ok = test_warp(empty(old), par) || wait_warp_pair(empty(old), par, p.wait_limit, abort_flag, peer_abort, p.err, 0x361u);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    tmem_st32(tmem + ((uint32_t)quarter << 16) + C::A_COL + b * A_COLS + h * (STAGE_K / 2), v);
                }
                if (!ok) break;
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_pair(afull0 + 8u * b);
            }
        }
    } else {
        const int quarter = 32 * (warp & 3), half = (warp - 2) >> 2;
        const uint32_t tempty0 = map_rank(tempty, 0);
        int iter = 0, at = 0;
        for (int w = cid; w < total; w += NC, ++iter) {
            const Item it = map_item(p, gs, CT, w, at);
            const int ch = (2 * it.ch + (int)rank) * BLOCK_N + quarter + lane, F = p.N / 2;
            float scale = 0.f;
            if (ch < p.N) scale = EPI == EPI_OUT ? p.w_scales[(size_t)it.g * p.N + ch] : ((ch & 1) ? p.w_scales_up : p.w_scales)[(size_t)it.g * F + (ch >> 1)];
            if (!wait_warp_pair(tfull, iter & 1, p.wait_limit, abort_flag, peer_abort, p.err, 0x370u)) break;
            tc_fence_after();
            const uint32_t tbase = tmem + (iter & 1) * C::ACC2 + ((uint32_t)quarter << 16);
            auto hand_back = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_pair(tempty0);
            };
            const bool warp_live = ch - lane < p.N;
            const int n = it.row1 - it.row0;
            if constexpr (ROWS == 256) {
                // the chunks whose columns the next tile shares come first: the last two of an even tile, the first two of an odd
                const int first = 64 * ((iter & 1 ? 0 : 2) + half), second = first ^ 128;
                if (warp_live && first < n) epilogue_chunk<EPI, 64>(p, it.g, tbase + first, ch, it.row0 + first, n - first, scale, hand_back);
                else hand_back();
                if (warp_live && second < n)
                    epilogue_chunk<EPI, 64>(p, it.g, tbase + second, ch, it.row0 + second, n - second, scale, [] {});
            } else {
                const int first = ROWS / 2 * half;
                if (warp_live && first < n)
                    epilogue_chunk<EPI, ROWS / 2>(p, it.g, tbase + first, ch, it.row0 + first, n - first, scale, hand_back);
                else hand_back();
            }
        }
    }
    cluster_sync_all();                          // every role of both CTAs has left its loop
    if (warp == 1 && lane == 0) drain_phase(mma_done, 0, p.err, 0x353u);
    tc_fence_before();
    cluster_sync_all();                      // MMAs done, both CTAs' copies landed, all arrivals on the other CTA made
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

// Row codes [rows][width] fp16, boxes of box_rows x 64 columns with 128-byte swizzling; zero past the rows.
static int rows_map(CUtensorMap* m, const void* base, long long rows, int width, int box_rows) {
    auto fn = encode_fn();
    MOE_REQUIRE(fn, MOE_ERR_CUDA, "cuTensorMapEncodeTiled unavailable from the driver");
    cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)width * 2};
    cuuint32_t box[2] = {STAGE_K, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    MOE_REQUIRE(r == CUDA_SUCCESS, MOE_ERR_CUDA, "cuTensorMapEncodeTiled (8-bit rows) failed (%d) rows=%lld width=%d", (int)r, rows, width);
    return MOE_OK;
}

template <int EPI, int ROWS>
static int launch_pair(const Params& p, cudaStream_t s) {
    constexpr int P_SMEM = Tile<ROWS>::SMEM;
    const auto kernel = pair_kernel<EPI, ROWS>;
    static int clusters[64];                     // resident pairs, in the context they were asked for
    static unsigned long long attr_ctx[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return set_error(MOE_ERR_CUDA, "int8 product: no usable current device");
    const unsigned long long ctx = context_id();
    if (!clusters[dev] || ctx == 0 || attr_ctx[dev] != ctx) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P_SMEM);
        if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "int8 product smem attribute: %s", cudaGetErrorString(e));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (num_sms() / 2));
        cfg.blockDim = dim3(P_THREADS);
        cfg.dynamicSmemBytes = P_SMEM;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
        if (e != cudaSuccess || n <= 0) return set_error(MOE_ERR_CUDA, "int8 product: no resident cluster of two CTAs (%s)", cudaGetErrorString(e));
        clusters[dev] = std::min(n, num_sms() / 2);
        attr_ctx[dev] = context_id();
    }
    CUtensorMap m16, m128;
    const int width = p.KST * STAGE_K;
    if (int rc = rows_map(&m16, p.a, p.rows, width, 16)) return rc;
    m128 = m16;                                  // (no tile of 256 rows: the map of whole halves is not used)
    if (ROWS == 256 && p.rows >= 128)
        if (int rc = rows_map(&m128, p.a, p.rows, width, 128)) return rc;
    return check_launch(launch_pdl(kernel, dim3(2 * clusters[dev]), dim3(P_THREADS), P_SMEM, s, m128, m16, p),
                        EPI == EPI_SWIGLU ? "int8 pair_kernel<swiglu>" : "int8 pair_kernel");
}

// Rows of a tile. A stage takes its MMAs as long for 64 rows as for 256, so more rows mean fewer tiles where groups are larger than a tile;
// where they are not, fewer rows leave more weights under way. 128 groups by 1536 x 2048, us by tiles of 64 / 128 / 256 rows: 64 rows a group
// 90 / 94 / 107, 96: 153 / 105 / 116, 128: 158 / 114 / 126, 256: 304 / 197 / 174. And where the tiles are no more than the pairs that run at
// once, a call is one tile long, and the epilogue of fewer rows is shorter (1003 rows by 7 x 1001 x 1044 in fp32: 13.4 / 12.3 / 14.5).
template <int EPI>
static int launch_pairs(const Params& p, cudaStream_t s) {
    const long long avg = p.rows / p.G, used = std::min(p.G, p.rows), pairs = num_sms() / 2, blocks = (p.NB + 1) / 2;
    if (avg <= 64 || ((p.rows - used) / 64 + used) * blocks <= pairs) return launch_pair<EPI, 64>(p, s);
    if (avg <= 128 || ((p.rows - used) / 128 + used) * blocks <= pairs) return launch_pair<EPI, 128>(p, s);
    return launch_pair<EPI, 256>(p, s);
}

// Tiles of a call at most.
static long long most_tiles(const Params& p) {
    const long long used = std::min(p.G, p.rows);
    return ((p.rows - used) / FEW_ROWS + used) * p.NB;
}

template <int EPI, bool SPLIT>
static int launch_few_as(const Params& p, int ranks, cudaStream_t s) {
    const auto kernel = few_rows_kernel<EPI, SPLIT>;
    static unsigned long long attr_ctx[64];
    static int resident[64][9];                  // clusters of 2, 4 and 8 at once
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return set_error(MOE_ERR_CUDA, "int8 product: no usable current device");
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    const unsigned long long ctx = context_id();
    if (ctx == 0 || attr_ctx[dev] != ctx) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM);
        if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "int8 product smem attribute: %s", cudaGetErrorString(e));
        for (int r = 2; SPLIT && r <= 8; r *= 2) {
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = r;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(num_sms() / r * r);
            cfg.blockDim = dim3(FEW_THREADS);
            cfg.dynamicSmemBytes = FEW_SMEM;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&resident[dev][r], kernel, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                resident[dev][r] = 0;
            }
        }
        attr_ctx[dev] = context_id();
    }
    if constexpr (SPLIT) {
        while (ranks > 1 && most_tiles(p) > resident[dev][ranks]) ranks /= 2;
        if (ranks == 1) return launch_few_as<EPI, false>(p, 1, s);
    }
    CUtensorMap m16;
    if (int rc = rows_map(&m16, p.a, p.rows, p.KST * STAGE_K, 16)) return rc;
    cfg.gridDim = dim3((unsigned)(SPLIT ? most_tiles(p) * ranks : std::min<long long>(most_tiles(p), num_sms())));
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = FEW_SMEM;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    return check_launch(cudaLaunchKernelEx(&cfg, kernel, m16, p), EPI == EPI_SWIGLU ? "int8 few_rows_kernel<swiglu>" : "int8 few_rows_kernel");
}
// CTAs to a tile: as many as leave each four stages of columns, and all clusters resident at once; one where a tile's columns are no more
// than the stages under way. Rows by channels x columns, us by one CTA and split: 16 by 96 x 6528 17.6 / 8.1, 8 by 192 x 7168 16.9 / 7.1, 16 by
// 4096 x 4096 12.8 / 8.7, 8 by 2048 x 2048 7.7 / 6.2; but 8 by 1024 x 1024 5.6 / 6.2, and 60 by 512 x 4096 in more clusters than are resident
// 12.8 / 14.0.
template <int EPI>
static int launch_few(const Params& p, cudaStream_t s) {
    int ranks = 1;
    const int stages = (p.KST + 1) / 2;
    while (stages > FEW_STAGES && ranks < 8 && most_tiles(p) * 2 * ranks <= num_sms() && stages >= 2 * ranks * 4) ranks *= 2;
    return ranks > 1 ? launch_few_as<EPI, true>(p, ranks, s) : launch_few_as<EPI, false>(p, 1, s);
}

template <int EPI>
static int launch_product(const Params& p, cudaStream_t s) {
    MOE_REQUIRE(((long long)p.rows / FEW_ROWS + p.G) * p.NB < (1LL << 31), MOE_ERR_INVALID_ARG,
                "8-bit product: %d rows by %d channels are over 2^31 tiles", p.rows, p.N);
    // The few rows' kernel where a group has up to 8 on average (128 groups by 1536 x 2048, us by it / by pairs of 64 rows: 4 rows a group 67 / 73,
    // 8: 69 / 73, 16: 76 / 76, and 16 unevenly 104 / 78), and where its tiles are no more than the SMs: pairs take longer to start (16 rows by
    // 4096 x 4096: 8.7 / 16.7). The mean is all that the host knows: rows of which most go to one group pass over its weights once for 16 of them.
    const long long used = std::min(p.G, p.rows);
    return p.rows / used <= 8 || most_tiles(p) <= num_sms() ? launch_few<EPI>(p, s) : launch_pairs<EPI>(p, s);
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
    if (int rc = int8::launch_quantize(x, ldx, x_rows, src, rows, K, dtype, int8::FORM_F16, ws, int8::scales_at(ws, rows, K), err, s)) return rc;
    return int8::launch_product<int8::EPI_OUT>(p, s);
}

// The FFN's workspace: x's operand, act [rows][F] in fp32 with rows of whole 16 bytes, act's operand.
namespace moe {
namespace int8 {
struct FfnWs { char* x; float* act; int ld; char* a; size_t bytes; };
static FfnWs ffn_ws(void* ws, int h, int F, long long rows) {
    FfnWs w{};
    char* base = static_cast<char*>(ws);
    w.x = base;
    size_t off = operand_bytes(rows, h);
    w.act = reinterpret_cast<float*>(base + off);
    w.ld = (F + 3) / 4 * 4;
    off = align_up(off + (size_t)rows * w.ld * 4, 256);
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
    p.w_scales = gate_scales; p.w_scales_up = up_scales; p.N = 2 * F; p.ld = w.ld; p.out_dtype = MOE_F32; p.out = w.act;
    p.err = err; p.wait_limit = wait_limit();
    if (int rc = int8::launch_quantize(x, ldx, x_rows, src, rows, h, dtype, int8::FORM_F16, w.x, int8::scales_at(w.x, rows, h), err, s)) return rc;
    if (int rc = int8::launch_product<int8::EPI_SWIGLU>(p, s)) return rc;
    if (int rc = int8::launch_quantize(w.act, w.ld, rows, nullptr, rows, F, MOE_F32, int8::FORM_F16, w.a, int8::scales_at(w.a, rows, F), err, s))
        return rc;
    p.w += L.down_off; p.NB = L.down.NB; p.KST = L.down.KST;
    p.a = w.a; p.a_scales = int8::scales_at(w.a, rows, F);
    p.w_scales = down_scales; p.w_scales_up = nullptr; p.N = h; p.ld = ldo; p.out_dtype = out_dtype; p.out = out;
    return int8::launch_product<int8::EPI_OUT>(p, s);
}
