// Grouped products of block-scaled e2m1 operands on the 5th-generation tensor cores, and the SwiGLU expert FFN made of two.
//
//   y[r] = alpha[g] * sum_k A[r, k] W[g, n, k]     for the rows r of group g,
// A and W codes times their block scales, accumulated in fp32 in tensor memory by tcgen05.mma with block scaling
// (kind::mxf4nvf4, 16-column blocks with e4m3 scales, and kind::mxf4, 32-column blocks with powers of two; K = 64 an
// instruction).
//
// One persistent CTA per SM with fourteen warps:
//   warp 0     producer: per stage of 256 columns a 128-row tile of codes of A by TMA (boxes of 32 rows where the tile has
//              fewer rows), BN weight rows, and both operands' block scales, each one bulk copy of contiguous packed bytes;
//   warp 1     the MMAs of a stage;
//   warps 2-9  epilogue, two warps to a quarter of the tensor memory lanes, taking 64-column chunks in turn: either
//              silu(gate) * up requantised to the next product's operand, or alpha times the accumulator in the output type;
//   warps 10-13  scales: each brings a stage's scale pieces from shared memory into its quarter of the tensor memory
//              lanes (every quarter holds all of them), ahead of the MMAs.
// Two accumulators: the epilogue of one tile runs under the MMAs of the next.
//
// Every wait is bounded, as in the bf16 grouped GEMM: one that runs out latches MOE_ERR_TIMEOUT, every role leaves, the
// copies and MMAs in flight are waited for and the tensor memory is freed.
#include <cudaTypedefs.h>
#include <algorithm>
#include "fp4.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace fp4 {
using namespace moe::tc;

constexpr int BM = 128;
constexpr int A_BYTES = BM * SEG_K / 2;          // 16 KB of codes
constexpr int EPI_WARPS = 8, SF_WARPS = 4;
constexpr int THREADS = 32 * (2 + EPI_WARPS + SF_WARPS);
constexpr int TMEM_COLS = 512;
constexpr int MAX_G = 1024;
constexpr int GROUPS_BYTES = (3 * MAX_G + 1) * 4;
constexpr int BOX_BYTES = 2048;                  // an epilogue warp's staging buffer
constexpr int SF_BUFS = 3;                       // stages of scales in tensor memory
// Gates below which the epilogue's quick quotient holds: 1 + exp(-g) and its products stay far inside fp32's normal range, and
// the exponential is within 2^-18.
constexpr float FAR_GATE = 48.f;

enum Epi : int { EPI_OUT = 0, EPI_SWIGLU = 1 };

template <int BN_, int STAGES_>
struct Cfg {
    static constexpr int BN = BN_, STAGES = STAGES_;
    static constexpr int B_BYTES = BN * SEG_K / 2;
    static constexpr int SF_BLOCKS = (BN + 127) / 128;               // 128-row scale tiles a weight tile touches
    template <class F> static constexpr int SFS = (1 + SF_BLOCKS) * SF_BYTES<F>;   // scale bytes of a stage
    template <class F> static constexpr int SMEM = 1024 + EPI_WARPS * BOX_BYTES + STAGES * (A_BYTES + B_BYTES + SFS<F>) + 256 + GROUPS_BYTES;
    static constexpr int SF_COL = 2 * BN;                            // scale columns follow the two accumulators
    static constexpr int B_COLS = BN / 32;                           // scale columns of the weight rows in a piece
    template <class F> static constexpr int SF_COLS = SF_PIECES<F> * (4 + B_COLS);   // of a stage
    static_assert(SF_COL + SF_BUFS * SF_COLS<Nv> <= TMEM_COLS, "tensor memory columns");
};

struct Params {
    const int32_t* offsets;      // the groups' rows, or null: the tiles of `sched`
    const int32_t* sched;
    int G, rows, max_tiles;      // (groups and tiles: what a schedule has to agree with)
    const uint8_t *a_sf, *w, *w_sf;
    int steps, kst;              // 64-column MMA steps, 256-column stages
    int NT, NB64, NB128;         // n-tiles; 64-row and 128-row blocks of the packed weight
    int N, ldo;                  // EPI_OUT: columns and row stride of the output
    int out_dtype;
    bool vec, boxed;             // rows of the output start on 16 bytes; it is stored by TMA where a warp's rows are all valid
    void* out;
    const float *alpha, *alpha_up;   // per group, or null (1)
    const float* act_gscale;     // EPI_SWIGLU: multiplier of act before it is quantised, or null
    uint8_t *act_codes, *act_sf;
    int act_pitch, act_kst;
    unsigned* err;
    long long wait_limit;
};

// The value of lane 0, known to the compiler to be the same in the warp: branches on it and what depends on it stay uniform.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

struct Work { int g, tile, row0, row1, n; };

// The groups in shared memory: first[g] tiles before group g (first[G]: all of them; 0 where offsets or schedule are no good:
// the quantisation reports the offsets, the product the schedule), its rows [beg[g], end[g]). A role finds its items without
// touching global memory: a search there cost a decode call microseconds, and a search from scratch an epilogue 1100 cycles a
// tile. From the offsets, which are older than the kernel before this one, they are found without waiting for that kernel
// (read from L2, where its predecessors' writes are).
struct Groups { int *first, *beg, *end; };
__device__ __forceinline__ Groups groups_at(void* smem) {
    int* first = static_cast<int*>(smem);
    return Groups{first, first + MAX_G + 1, first + 2 * MAX_G + 1};
}
__device__ __forceinline__ void find_groups(const Params& p, const Groups& gs) {
    if (p.offsets) {
        scan_groups<THREADS>(p.offsets, p.G, p.rows, gs.first, gs.beg, gs.end);
        return;
    }
    // A schedule counts where its tiles are those of the groups' rows within the call: a tile that starts past the call's rows,
    // as another call's can, would have the producer ask for a negative number of rows.
    const int ntiles = __ldcg(p.sched);
    const bool fits = __ldcg(p.sched + 1) == p.G && ntiles <= p.max_tiles;
    const int32_t* prefix = p.sched + kSchedHeader;
    const int4* tiles = reinterpret_cast<const int4*>(p.sched + sched_tiles_offset(p.G));
    bool bad = !fits;
    for (int g = threadIdx.x; g < p.G; g += THREADS) {
        const int t0 = fits ? __ldcg(prefix + g) : 0, t1 = fits ? __ldcg(prefix + g + 1) : 0;
        const bool some = 0 <= t0 && t0 < t1 && t1 <= ntiles;
        const int beg = some ? min(__ldcg(tiles + t0).y, p.rows) : 0, end = some ? min(__ldcg(tiles + t1 - 1).z, p.rows) : 0;
        bad |= (some ? beg < 0 || (max(end - beg, 0) + BM - 1) / BM != t1 - t0 : t0 != t1) || (g == 0 && t0 != 0) ||
               (g == p.G - 1 && t1 != ntiles);
        gs.first[g + 1] = t1;
        gs.beg[g] = beg;
        gs.end[g] = end;
    }
    if (threadIdx.x == 0) gs.first[0] = 0;
    if (__syncthreads_or(bad)) {
        for (int g = threadIdx.x; g <= p.G; g += THREADS) gs.first[g] = 0;
        if (blockIdx.x == 0 && threadIdx.x == 0) latch_device_error(p.err, kDevErrBadIndex, 0x204u);
        __syncthreads();
    }
}
// The last group g from `g` on with before[g] * NT <= w: steps that double (a role's items rise), then halving.
__device__ __forceinline__ int group_of(const int* before, int G, int NT, int w, int g) {
    int hi = g + 1;                      // before[hi] * NT > w, or hi == G
#pragma unroll 1
    for (int step = 1; hi < G && before[hi] * NT <= w; step *= 2) {
        g = hi;
        hi = min(hi + step, G);
    }
#pragma unroll 1
    while (hi - g > 1) {
        const int mid = (g + hi) >> 1;
        if (before[mid] * NT <= w) g = mid; else hi = mid;
    }
    return g;
}
// Item w: group by group, n-tile next, m-tile fastest: CTAs that run together share a weight tile. g: the group of the role's
// item before, and of this one.
__device__ __forceinline__ Work map_work(const Params& p, const Groups& gs, int w, int& g) {
    g = group_of(gs.first, p.G, p.NT, w, g);
    const int p0 = gs.first[g], mt = gs.first[g + 1] - p0, local = w - p0 * p.NT;
    const int n = local / mt, m = local - n * mt, row0 = gs.beg[g] + m * BM;
    return Work{g, p0 + m, row0, min(row0 + BM, gs.end[g]), n};
}

// The producer's and the MMA warp's operations. The whole warp runs its loop, with conditions that are the same in all lanes
// (votes, uniform()), and one elected lane, the same each time, issues: addresses and descriptors then stay in uniform
// registers. Issued from a branch that one lane takes, a stage of four MMAs cost 690 cycles, where they take 4 x 96 (N = 192).
#define MOE_ELECTED(op) "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t@e " op "\n\t}"
__device__ __forceinline__ void expect_elected(uint32_t bar, uint32_t bytes) {
    asm volatile(MOE_ELECTED("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;") ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_elected(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(MOE_ELECTED("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];")
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_elected(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(MOE_ELECTED("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                             " [%0], [%1, {%2, %3}], [%4];")
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}
template <class F>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t accumulate) {
    if constexpr (F::ID == MOE_FP4_NV)
        asm volatile(
            "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar) : "memory");
}
// wait_phase for a whole warp, the same answer in every lane.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, long long limit, volatile int* abort_flag, unsigned* err,
                                          unsigned site) {
    for (long long i = 0; i < limit; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *abort_flag)) return false;
    }
    if ((threadIdx.x & 31) == 0) {
        *abort_flag = 1;
        latch_device_error(err, kDevErrTimeout, site);
    }
    __syncwarp();
    return false;
}
// Whether a phase has completed, without waiting. Even a wait that succeeds at once takes some 180 cycles to answer; asked
// before a stage's work and read after it, the answer about the next stage costs nothing.
__device__ __forceinline__ bool test_phase(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool test_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, test_phase(bar, parity));
}
// 16 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                 "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, uint32_t* v) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr) : "memory");
}
// Instruction descriptor of the block-scaled kinds: A and B e2m1 (bits 7-9 and 10-12 = 1), both K-major, N >> 3 at bits
// 17-22, scale type at bit 23 (0: e4m3, 1: power of two), M >> 4 at bits 24-28, K = 64 (bit 31 = 0; the chip's highest 4-bit
// rate, six times the bf16 one, is that of K = 96, which is not used: loads do not keep up with K = 64). Bits 4-5 and 29-30:
// which byte of a scale word is the step's first (0, and 2 for the second 64 columns of an MX piece).
template <class F, int M, int N>
__device__ constexpr uint32_t idesc_scaled(int sub) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((F::ID == MOE_FP4_MX ? 1u : 0u) << 23) |
           ((uint32_t)(M >> 4) << 24) | ((uint32_t)(2 * sub) << 4) | ((uint32_t)(2 * sub) << 29);
}

// 32 consecutive columns of an output row that starts on 16 bytes, in its type.
template <typename T> __device__ __forceinline__ T out_round(float v);
template <> __device__ __forceinline__ float out_round<float>(float v) { return v; }
template <> __device__ __forceinline__ __half out_round<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 out_round<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <typename T>
__device__ __forceinline__ void store_row(T* dst, const float* v, float al, int n) {
    constexpr int PER = 16 / sizeof(T);
#pragma unroll
    for (int c = 0; c < 32; c += PER) {
        alignas(16) T o[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = out_round<T>(v[c + i] * al);
        if (c + PER <= n) {
            *reinterpret_cast<uint4*>(dst + c) = *reinterpret_cast<const uint4*>(o);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (c + i < n) dst[c + i] = o[i];
        }
    }
}
// A box of 32 rows x 64 bytes of the output through the warp's staging buffer `stg` (the layout of 64-byte swizzling: 16-byte
// chunk c of row r at chunk c ^ (r / 2 % 4)) and one TMA store: whole sectors reach L2, where a thread's own 16-byte stores
// touch half a sector of each of 32 rows. v: the 64 bytes' values of this lane's row.
template <typename T>
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t stg, const float* v, float al, int col, int row0) {
    constexpr int PER = 16 / sizeof(T);
    const int lane = threadIdx.x & 31;
    if (lane == 0) bulk_wait_read_all();             // the previous box has left the buffer
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        alignas(16) T o[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = out_round<T>(v[c * PER + i] * al);
        const uint4 w = *reinterpret_cast<const uint4*>(o);
        st_shared_v4u(stg + lane * 64u + ((uint32_t)(c ^ (lane >> 1 & 3)) << 4), w.x, w.y, w.z, w.w);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
        tma_store_2d(map, stg, col, row0);
        bulk_commit();
    }
}
template <typename T>
__device__ __forceinline__ void store_boxes(const CUtensorMap* map, uint32_t stg, const float* v, float al, int col, int n, int row0) {
    constexpr int COLS = 64 / sizeof(T);
#pragma unroll
    for (int c = 0; c < 64; c += COLS)
        if (c < n) store_box<T>(map, stg, v + c, al, col + c, row0);
}

// Rows that start on no boundary: 64 bytes of each of the warp's 32 rows at a time through the staging buffer, from where the
// lanes write neighbouring columns (1003 x 1001 fp32 rows stored by a lane each touched 32 sectors a store).
template <typename T>
__device__ __forceinline__ void store_loose(T* out, long long ldo, uint32_t stg, const float* v, float al, int col, int n, int row0,
                                            int rows) {
    constexpr int PER = 16 / sizeof(T), COLS = 64 / sizeof(T);
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int g = 0; g < 64; g += COLS) {
        if (g >= n) break;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            alignas(16) T o[PER];
#pragma unroll
            for (int i = 0; i < PER; ++i) o[i] = out_round<T>(v[g + c * PER + i] * al);
            const uint4 w = *reinterpret_cast<const uint4*>(o);
            st_shared_v4u(stg + lane * 64u + ((uint32_t)(c ^ (lane >> 1 & 3)) << 4), w.x, w.y, w.z, w.w);
        }
        __syncwarp();
        const int c = lane % COLS;
#pragma unroll 4
        for (int r = lane / COLS; r < rows; r += 32 / COLS) {
            const uint32_t a = stg + r * 64u + ((uint32_t)((c / PER) ^ (r >> 1 & 3)) << 4) + (uint32_t)(c % PER) * sizeof(T);
            if (g + c < n) {
                if constexpr (sizeof(T) == 4) {
                    float x;
                    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
                    out[(row0 + r) * ldo + col + g + c] = x;
                } else {
                    uint16_t x;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(a) : "memory");
                    reinterpret_cast<uint16_t*>(out)[(row0 + r) * ldo + col + g + c] = x;
                }
            }
        }
        __syncwarp();
    }
}

// Chunk of 64 accumulator columns at column c0 of the tile's output, this thread's row r of the tile (live: one of its
// rows). `read` runs once the chunk's columns are in registers.
template <class F, int EPI, typename Fn>
__device__ __forceinline__ void epilogue_chunk(const Params& p, const CUtensorMap* map, uint32_t stg, const Work& wk, uint32_t tcol,
                                               int c0, int r, bool live, Fn read) {
    const int row = wk.row0 + r;
    float v[64];
    tmem_ld32(tcol, *reinterpret_cast<float (*)[32]>(v));
    tmem_ld32(tcol + 32, *reinterpret_cast<float (*)[32]>(v + 32));
    read();
    if constexpr (EPI == EPI_SWIGLU) {
        if (!live) return;
        const float ag = p.alpha ? __ldg(p.alpha + wk.g) : 1.f, au = p.alpha_up ? __ldg(p.alpha_up + wk.g) : 1.f;
        const float gs = p.act_gscale ? __ldg(p.act_gscale) : 1.f;
        const int f0 = c0 / 2;                   // first column of act
        // g / (1 + exp(-g)) * u, each step but the exponential rounded as written, so that an activation at a rounding tie of
        // its code mostly goes the way that the plain fp32 formula takes: with the quotient as g times the MUFU's reciprocal,
        // two codes in a million went the other way. The exponential is the MUFU's of the rounded g log2(e), off by
        // about 2^-22 + 1.25 |g| 2^-24 of it; expf cost the FFN of 16384 tokens and 128 experts 384 -> 402 us.
        float* u = v + 32;
        float far = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 2) mul2(v + i, v + i, ag);
#pragma unroll
        for (int i = 0; i < 32; ++i) far = max_nan(far, fabsf(v[i]));
        if (far < FAR_GATE) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float t[2], d[2], r[2];
                mul2(t, v + i, -1.44269504f);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    asm("ex2.approx.f32 %0, %1;" : "=f"(d[j]) : "f"(t[j]));
                    d[j] = 1.f + d[j];
                    asm("rcp.approx.f32 %0, %1;" : "=f"(r[j]) : "f"(d[j]));
                }
                quotient2v(v + i, d, r);
            }
        } else {
            // a gate far from 0, infinite or NaN among the 32: exp(-g) would overflow, and the correction of an infinite
            // quotient is NaN. As g exp(-|g|) / (1 + exp(-|g|)), without the numerator's exponential from 0 on. (Rolled, through local
            // memory: unrolled, the code that hardly runs cost the FFN of 16384 tokens and 128 experts 383 -> 388 us.)
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = v[i];
#pragma unroll 1
            for (int i = 0; i < 32; ++i) {
                const float e = expf(-fabsf(x[i]));
                float r;
                asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
                x[i] = (x[i] < 0.f ? x[i] * e : x[i]) * r;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = x[i];
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            mul2(u + i, u + i, au);
            mul2v(u + i, v + i, u + i);
            mul2(u + i, u + i, gs);
        }
        uint32_t w[4], bytes = 0u;
#pragma unroll
        for (int b = 0; b < 32 / F::BLK; ++b) {
            float amax = 0.f, s, rc;
#pragma unroll
            for (int i = 0; i < F::BLK; ++i) amax = max_nan(amax, fabsf(u[b * F::BLK + i]));
            bytes |= block_scale<F>(amax, s, rc) << (8 * b);
            block_codes<F>(u + b * F::BLK, amax, s, rc, w + b * (F::BLK / 8));
        }
        *reinterpret_cast<uint4*>(p.act_codes + (size_t)row * p.act_pitch + f0 / 2) = make_uint4(w[0], w[1], w[2], w[3]);
        const int b0 = f0 / F::BLK;
        uint8_t* sf = p.act_sf + (size_t)wk.tile * p.act_kst * SF_BYTES<F> + (size_t)(b0 >> 2) * 512 + (r & 31) * 16 +
                      (r >> 5) * 4 + (b0 & 3);
        if constexpr (F::ID == MOE_FP4_NV) *reinterpret_cast<uint16_t*>(sf) = (uint16_t)bytes;
        else *sf = (uint8_t)bytes;
    } else {
        const float al = p.alpha ? __ldg(p.alpha + wk.g) : 1.f;
        const int n = p.N - c0;
        if (n <= 0) return;
        if (p.boxed && wk.row0 + (r & ~31) + 31 < wk.row1) {     // all of the warp's rows (the map drops pieces past N)
            const int base = wk.row0 + (r & ~31);
            if (p.out_dtype == MOE_F32) store_boxes<float>(map, stg, v, al, c0, n, base);
            else if (p.out_dtype == MOE_BF16) store_boxes<__nv_bfloat16>(map, stg, v, al, c0, n, base);
            else store_boxes<__half>(map, stg, v, al, c0, n, base);
            return;
        }
        if (!p.vec) {
            const int base = wk.row0 + (r & ~31), rows = min(32, wk.row1 - base);
            if (p.out_dtype == MOE_F32) store_loose(static_cast<float*>(p.out), p.ldo, stg, v, al, c0, n, base, rows);
            else if (p.out_dtype == MOE_BF16) store_loose(static_cast<__nv_bfloat16*>(p.out), p.ldo, stg, v, al, c0, n, base, rows);
            else store_loose(static_cast<__half*>(p.out), p.ldo, stg, v, al, c0, n, base, rows);
            return;
        }
        if (!live) return;
        const int el = p.out_dtype == MOE_F32 ? 4 : 2;
        uint8_t* dst = static_cast<uint8_t*>(p.out) + ((size_t)row * p.ldo + c0) * el;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (n - 32 * h <= 0) break;
            if (p.out_dtype == MOE_F32) store_row(reinterpret_cast<float*>(dst) + 32 * h, v + 32 * h, al, n - 32 * h);
            else if (p.out_dtype == MOE_BF16)
                store_row(reinterpret_cast<__nv_bfloat16*>(dst) + 32 * h, v + 32 * h, al, n - 32 * h);
            else store_row(reinterpret_cast<__half*>(dst) + 32 * h, v + 32 * h, al, n - 32 * h);
        }
    }
}

template <class F, class C, int EPI>
__global__ void __launch_bounds__(THREADS, 1)
fp4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                const __grid_constant__ CUtensorMap tmO, Params p) {
    constexpr int BN = C::BN, STAGES = C::STAGES, B_BYTES = C::B_BYTES, SFS = C::template SFS<F>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sA = smem_u32(smem), sB = sA + STAGES * A_BYTES, sO = sB + STAGES * B_BYTES,
                   sS = sO + EPI_WARPS * BOX_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * (A_BYTES + B_BYTES + SFS) + EPI_WARPS * BOX_BYTES);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
    auto tempty = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
    const uint32_t mma_done = bar0 + 8u * (2 * STAGES + 4);
    auto sfull = [&](int b) { return bar0 + 8u * (2 * STAGES + 5 + b); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5 + SF_BUFS);
    const Groups gs = groups_at(bars + 32);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
        for (int a = 0; a < 2; ++a) { mbar_init(tfull(a), 1); mbar_init(tempty(a), EPI_WARPS); }
        for (int b = 0; b < SF_BUFS; ++b) mbar_init(sfull(b), SF_WARPS);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmA32);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    find_groups(p, gs);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (a programmatic dependent of the kernel that writes the row operand: the groups, the weights and everything above do
    // not wait for it)
    const int total = uniform(gs.first[p.G] * p.NT);
    if (warp != 0) {
        pdl_wait();
        pdl_trigger();
    }

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0, issued = 0, last_par = 0;
        bool ok = true, ready = false;              // ready: the next ring stage was seen free
        int at = 0;
        for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
            const Work wk = map_work(p, gs, w, at);
            const int n = uniform(wk.n), g = uniform(wk.g), tile = uniform(wk.tile), row0 = uniform(wk.row0);
            const int boxes = uniform((wk.row1 - wk.row0 + 31) >> 5);
            const int nb = min(BN / 64, p.NB64 - n * (BN / 64));
            const int t0 = n * BN / 128, nt = min((n * BN + BN + 127) / 128, p.NB128) - t0;
            const uint8_t* w0 = p.w + (size_t)g * p.kst * p.NB64 * 8192 + (size_t)n * (BN / 64) * 8192;
            const uint8_t* s0 = p.w_sf + ((size_t)g * p.kst * p.NB128 + t0) * SF_BYTES<F>;
            const uint8_t* a0 = p.a_sf + (size_t)tile * p.kst * SF_BYTES<F>;
            const uint32_t tx = (uint32_t)(boxes * 4096 + nb * 8192 + (1 + nt) * SF_BYTES<F>);
            auto weights = [&](int st, int kb) {
                expect_elected(full(st), tx);
                bulk_elected(sB + st * B_BYTES, w0 + (size_t)kb * p.NB64 * 8192, nb * 8192, full(st));
                bulk_elected(sS + st * SFS + SF_BYTES<F>, s0 + (size_t)kb * p.NB128 * SF_BYTES<F>, nt * SF_BYTES<F>, full(st));
            };
            int early = 0;                          // stages whose weights are on their way before the row operand is there
            if (w == (int)blockIdx.x) {
                for (; early < min(STAGES, p.kst); ++early) weights(early, early);
                pdl_wait();
                pdl_trigger();
            }
            for (int kb = 0; kb < p.kst; ++kb) {
                if (kb >= early) {
                    if (!ready) ok = wait_warp(empty(stage), phase ^ 1u, p.wait_limit, abort_flag, p.err, 0x210u);
                    if (!ok) break;
                    weights(stage, kb);
                }
                const uint32_t f = full(stage), sa = sA + stage * A_BYTES;
                if (boxes == 4) tma_elected(sa, &tmA, kb * (SEG_K / 2), row0, f);
                else
                    for (int b = 0; b < boxes; ++b) tma_elected(sa + b * 4096, &tmA32, kb * (SEG_K / 2), row0 + 32 * b, f);
                bulk_elected(sS + stage * SFS, a0 + (size_t)kb * SF_BYTES<F>, SF_BYTES<F>, f);
                issued |= 1u << stage;
                last_par = (last_par & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                ready = kb + 1 >= early && test_warp(empty(stage), phase ^ 1u);
            }
        }
        if (lane == 0)
            for (int s = 0; s < STAGES; ++s)        // every issued copy has landed before the CTA exits
                if (issued & (1u << s)) drain_phase(full(s), (last_par >> s) & 1u, p.err, 0x211u);
        __syncwarp();
    } else if (warp == 1) {
        constexpr int PIECES = SF_PIECES<F>;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        int stage = 0, b = 0, acc = 0;
        uint32_t phase = 0, bphase = 0, aphase = 1;
        bool ok = true, ready = false;              // ready: all that the stage waits for was seen complete
        for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
            for (int kb = 0; kb < p.kst; ++kb) {
                if (!ready)
                    ok = (kb > 0 || wait_warp(tempty(acc), aphase, p.wait_limit, abort_flag, p.err, 0x220u)) &&
                         wait_warp(full(stage), phase, p.wait_limit, abort_flag, p.err, 0x221u) &&
                         wait_warp(sfull(b), bphase, p.wait_limit, abort_flag, p.err, 0x223u);
                if (!ok) break;
                tc_fence_after();
                const uint32_t s0 = stage, b0 = b, a0 = acc;
                const bool last = kb + 1 == p.kst;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                if (++b == SF_BUFS) { b = 0; bphase ^= 1u; }
                if (last && ++acc == 2) { acc = 0; aphase ^= 1u; }
                const bool t0 = test_phase(full(stage), phase), t1 = test_phase(sfull(b), bphase),
                           t2 = test_phase(tempty(acc), aphase);
                const uint64_t da = sw128_desc(sA + s0 * A_BYTES), db = sw128_desc(sB + s0 * B_BYTES);
                const uint32_t d = tm + a0 * BN, sfa = tm + C::SF_COL + b0 * C::template SF_COLS<F>, sfb = sfa + PIECES * 4;
                const int n = min(4, p.steps - 4 * kb);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (k < n) {
                        const int q = F::ID == MOE_FP4_NV ? k : k / 2;
                        const uint32_t id = idesc_scaled<F, BM, BN>(F::ID == MOE_FP4_NV ? 0 : k & 1);
                        mma_scaled<F>(d, da + 2 * k, db + 2 * k, id, sfa + 4 * q, sfb + C::B_COLS * q, (kb | k) != 0);
                    }
                }
                commit_elected(empty(s0));
                if (last) commit_elected(tfull(a0));
                ready = __all_sync(0xffffffffu, t0 && t1 && (t2 || !last));
            }
        }
        commit_elected(mma_done);                   // all MMAs finished before the columns are freed
        if (lane == 0) drain_phase(mma_done, 0, p.err, 0x222u);
        __syncwarp();
    } else if (warp >= 2 + EPI_WARPS) {
        // Stage i's scales go to buffer i % SF_BUFS once the MMAs of stage i - SF_BUFS have completed (they free its ring
        // stage too). A tile that starts in the middle of a 128-row scale tile takes the second half of the first one.
        constexpr int PIECES = SF_PIECES<F>, COLS = C::template SF_COLS<F>, BC = C::B_COLS;
        const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
        int stage = 0, b = 0, old = STAGES - SF_BUFS;
        uint32_t phase = 0, ophase = 1;             // (the rounds before the first count as complete)
        bool ok = true, loaded = false, freed = false;
        int at = 0;
        for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
            const bool odd = BN % 128 == 64 && (map_work(p, gs, w, at).n & 1);
            for (int kb = 0; kb < p.kst; ++kb) {
                if (!loaded) ok = wait_warp(full(stage), phase, p.wait_limit, abort_flag, p.err, 0x241u);
                if (!ok) break;
                const bool t0 = test_phase(empty(old), ophase);
                uint32_t v[COLS];
                const uint32_t src = sS + stage * SFS + lane * 16;
#pragma unroll
                for (int q = 0; q < PIECES; ++q) {
                    ld_shared_v4(src + q * 512, v + 4 * q);
                    uint32_t x[4 * C::SF_BLOCKS];
#pragma unroll
                    for (int t = 0; t < C::SF_BLOCKS; ++t) ld_shared_v4(src + (1 + t) * SF_BYTES<F> + q * 512, x + 4 * t);
#pragma unroll
                    for (int c = 0; c < BC; ++c) v[4 * PIECES + BC * q + c] = odd ? x[(c + 2) % (4 * C::SF_BLOCKS)] : x[c];
                }
                freed = __all_sync(0xffffffffu, t0);
                if (!freed) ok = wait_warp(empty(old), ophase, p.wait_limit, abort_flag, p.err, 0x240u);
                if (!ok) break;
                tc_fence_after();
                const uint32_t dst = tmem + quarter + C::SF_COL + b * COLS;
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
                    if (c + 16 <= COLS) tmem_st16(dst + c, v + c);
                    else if (c + 8 <= COLS) {
                        tmem_st8(dst + c, v + c);
                        if (c + 12 <= COLS) tmem_st4(dst + c + 8, v + c + 8);
                    } else tmem_st4(dst + c, v + c);
                }
                const uint32_t sb = sfull(b);
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                if (++old == STAGES) { old = 0; ophase ^= 1u; }
                if (++b == SF_BUFS) b = 0;
                const bool t1 = test_phase(full(stage), phase);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                loaded = __all_sync(0xffffffffu, t1);
                if (lane == 0) mbar_arrive(sb);
            }
        }
    } else {
        const int quarter = 32 * (warp & 3), half = (warp - 2) >> 2, r = quarter + lane;
        int iter = 0, at = 0;
        for (int w = blockIdx.x; w < total; w += gridDim.x, ++iter) {
            const int a = iter & 1;
            const Work wk = map_work(p, gs, w, at);
            if (!wait_warp(tfull(a), (iter >> 1) & 1, p.wait_limit, abort_flag, p.err, 0x230u)) break;
            tc_fence_after();
            const uint32_t tbase = tmem + a * BN + ((uint32_t)quarter << 16);
            if (wk.row0 + quarter < wk.row1) {
                const int nb = min(BN / 64, p.NB64 - wk.n * (BN / 64));
#pragma unroll 1
                for (int q = (half + iter) & 1; q < nb; q += 2)
                    epilogue_chunk<F, EPI>(p, &tmO, sO + (warp - 2) * BOX_BYTES, wk, tbase + 64 * q, wk.n * BN + 64 * q, r,
                                           wk.row0 + r < wk.row1, [] {});
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty(a));
        }
        if (lane == 0) bulk_wait_read_all();         // every box read out of shared memory before the CTA exits
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------------------------------
// two SMs to a tile: a cluster of two CTAs computes 256 rows x 256 columns with tcgen05.mma.cta_group::2
// ---------------------------------------------------------------------------------------------------
// The one-SM kernel waits for its operands: a stage of four MMAs (N = 192) takes 385 cycles and needs 47 KB, and with 150 to
// 190 KB under way some 55 bytes a cycle arrive. In a pair each SM holds its own 128 rows of A and half of the weight rows
// (and the scales of all of them, which its tensor core needs): 38 KB for MMAs a third larger, and five stages of them.
// 16384 skewed rows by 8 x 14336 x 4096 (NV): 456 us by single SMs, 343 by pairs with the quantisation of 41 in both (short
// runs; in long ones, under the power cap, pairs take 375); 300 of the pairs' time at 6.4 PFLOP/s. The MMAs alone, without
// loads and epilogue, took 233. (8192 rows by 4 x 12288 x 4096: 6.2 PFLOP/s, the tensor pipe 64 % busy.)
// The even CTA issues the MMAs for both. Every copy of a CTA completes on its own barrier; the odd CTA's scale warps, which
// wait for it, pass the news on with their arrival on the even CTA's scale barrier, so that barrier tells of both CTAs'
// operands. A pair takes two consecutive tiles of one group; where the second does not exist the odd CTA computes the
// first one again and stores nothing.
// The scales of the weight rows come from the scale warps, those of A's rows by tcgen05.cp from the MMA warp: four copies
// a stage fit beside four MMAs of 256 columns at no cost, and leave tensor memory for three stages of the others.
// Tensor memory has no room for two accumulators of 256 columns next to the scales: they share 128 columns. The epilogue
// reads the shared columns into registers first and frees them at once, so the next tile's MMAs wait for a read of two of
// its four chunks and not for their conversion and stores.
constexpr int PB_BYTES = 128 * SEG_K / 2;        // a CTA's half of the weight rows
constexpr int P_BN = 256, P_SF_BUFS = 3, P_ACC2 = 128, P_SF_COL = P_ACC2 + P_BN, P_SFA_COL = P_SF_COL + 96;
template <class F> constexpr int P_SFS = 3 * SF_BYTES<F>;
// The loads' latency needs the bytes under way: five stages instead of four, for staging buffers of 2 KB instead of 4, took
// the product above from 381 to 350 us and the FFN of 8192 tokens through 8 experts of 14336 from 1007 to 915.
template <int EPI> constexpr int P_STAGES = 5;
template <int EPI> constexpr int P_BOX = EPI == EPI_OUT ? BOX_BYTES : 0;
template <class F, int EPI>
constexpr int P_SMEM = 1024 + EPI_WARPS * P_BOX<EPI> + P_STAGES<EPI> * (A_BYTES + PB_BYTES + P_SFS<F>) + 256 + GROUPS_BYTES + (MAX_G + 1) * 4;
template <class F> constexpr int P_COLS = SF_PIECES<F> * 8;      // scale columns of the weight rows in a stage
static_assert(P_SF_BUFS * P_COLS<Nv> <= 96 && P_SFA_COL + 2 * SF_PIECES<Nv> * 4 <= TMEM_COLS, "tensor memory columns");
static_assert(P_SMEM<Nv, EPI_OUT> + 64 <= 227 * 1024, "shared memory per CTA");

template <class F>
__device__ __forceinline__ void mma_scaled_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                uint32_t accumulate) {
    if constexpr (F::ID == MOE_FP4_NV)
        asm volatile(
            "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) : "memory");
}
// 32 rows of 16 bytes (8-row groups 128 bytes apart) of each CTA's shared memory -> the same 4 columns of each quarter of
// its tensor memory lanes.
__device__ __forceinline__ void sf_copy_pair(uint32_t taddr, uint32_t saddr) {
    const uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 32 | (uint64_t)1 << 46;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(d) : "memory");
}
// On both CTAs' barrier at this offset.
__device__ __forceinline__ void commit_pair_elected(uint32_t bar) {
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
                 ::"r"(bar), "h"((uint16_t)3) : "memory");
}
__device__ __forceinline__ void arrive_pair(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// (What the other CTA's arrivals tell of lies in tensor memory and in asynchronously filled shared memory, ordered by the
// tcgen05 fences on both sides; an acquire at cluster scope, which orders ordinary loads too, cost 450 cycles a wait.)
__device__ __forceinline__ bool wait_warp_pair(uint32_t bar, uint32_t parity, long long limit, volatile int* abort_flag,
                                               uint32_t peer_abort, unsigned* err, unsigned site) {
    for (long long i = 0; i < limit; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if (__any_sync(0xffffffffu, *abort_flag)) return false;
    }
    if ((threadIdx.x & 31) == 0) {
        *abort_flag = 1;
        st_cluster(peer_abort, 1u);
        latch_device_error(err, kDevErrTimeout, site);
    }
    __syncwarp();
    return false;
}

// Item w: group by group, n-tile next, pair fastest. tile, arow: what this CTA loads; row0, row1: what it stores.
struct PairItem { Work wk; int arow, rows; };
__device__ __forceinline__ int pairs_of(const int* first, int g) { return (first[g + 1] - first[g] + 1) >> 1; }
// pp[g]: pairs before group g.
__device__ __forceinline__ PairItem map_pair_item(const Params& p, const Groups& gs, const int* pp, int w, int rank, int& g) {
    g = group_of(pp, p.G, p.NT, w, g);
    const int np = pp[g + 1] - pp[g], local = w - pp[g] * p.NT;
    const int n = local / np, q = local - n * np;
    const int p0 = gs.first[g], mt = gs.first[g + 1] - p0;
    const bool has = 2 * q + rank < mt;
    const int m = 2 * q + (has ? rank : 0), row0 = gs.beg[g] + m * BM, row1 = min(row0 + BM, gs.end[g]);
    return PairItem{Work{g, p0 + m, has ? row0 : 0, has ? row1 : 0, n}, row0, row1 - row0};
}

template <class F, int EPI>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
fp4_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA32,
                     const __grid_constant__ CUtensorMap tmO, Params p) {
    constexpr int STAGES = P_STAGES<EPI>, SFS = P_SFS<F>, PIECES = SF_PIECES<F>, COLS = P_COLS<F>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sA = smem_u32(smem), sB = sA + STAGES * A_BYTES, sO = sB + STAGES * PB_BYTES, sS = sO + EPI_WARPS * P_BOX<EPI>;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * (A_BYTES + PB_BYTES + SFS) + EPI_WARPS * P_BOX<EPI>);
    const uint32_t bar0 = smem_u32(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto sfull = [&](int b) { return bar0 + 8u * (2 * STAGES + b); };
    const uint32_t tfull = bar0 + 8u * (2 * STAGES + P_SF_BUFS), tempty = tfull + 8u, mma_done = tempty + 8u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + P_SF_BUFS + 3);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const Groups gs = groups_at(bars + 32);
    int* pp = gs.first + 3 * MAX_G + 1;

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
        for (int b = 0; b < P_SF_BUFS; ++b) mbar_init(sfull(b), 2 * SF_WARPS);
        mbar_init(tfull, 1);
        mbar_init(tempty, 2 * EPI_WARPS);
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tmap(&tmA);
        prefetch_tmap(&tmA32);
    }
    // (a programmatic dependent of the kernel that writes the row operand: the groups, the weights and the set-up do not wait
    // for it)
    find_groups(p, gs);
    if (warp == 2) {                             // pairs of tiles of each group, summed up
        int carry = 0;
        if (lane == 0) pp[0] = 0;
        for (int base = 0; base < p.G; base += 32) {
            const int g = base + lane;
            int v = g < p.G ? pairs_of(gs.first, g) : 0;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, v, off);
                if (lane >= off) v += t;
            }
            if (g < p.G) pp[g + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tc_fence_before();
    cluster_sync_all();                          // barriers initialised and both CTAs' tensor memory allocated
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t peer_abort = map_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u);
    const int NC = gridDim.x >> 1, cid = blockIdx.x >> 1, total = uniform(pp[p.G] * p.NT);
    if (warp != 0) {
        pdl_wait();
        pdl_trigger();
    }

    if (warp == 0) {
        int stage = 0;
        uint32_t phase = 0, issued = 0, last_par = 0;
        bool ok = true, ready = false;
        int at = 0;
        for (int w = cid; w < total && ok; w += NC) {
            const PairItem it = map_pair_item(p, gs, pp, w, rank, at);
            const int n = uniform(it.wk.n), g = uniform(it.wk.g), tile = uniform(it.wk.tile), arow = uniform(it.arow);
            const int boxes = uniform((it.rows + 31) >> 5), half = uniform((int)rank);
            const int nb = min(2, max(0, p.NB64 - n * 4 - 2 * half)), nt = min(2, p.NB128 - 2 * n);
            const uint8_t* w0 = p.w + (size_t)g * p.kst * p.NB64 * 8192 + (size_t)(n * 4 + 2 * half) * 8192;
            const uint8_t* s0 = p.w_sf + ((size_t)g * p.kst * p.NB128 + 2 * n) * SF_BYTES<F>;
            const uint8_t* a0 = p.a_sf + (size_t)tile * p.kst * SF_BYTES<F>;
            const uint32_t tx = (uint32_t)(boxes * 4096 + nb * 8192 + (1 + nt) * SF_BYTES<F>);
            auto weights = [&](int st, int kb) {
                expect_elected(full(st), tx);
                if (nb) bulk_elected(sB + st * PB_BYTES, w0 + (size_t)kb * p.NB64 * 8192, nb * 8192, full(st));
                bulk_elected(sS + st * SFS + SF_BYTES<F>, s0 + (size_t)kb * p.NB128 * SF_BYTES<F>, nt * SF_BYTES<F>, full(st));
            };
            int early = 0;
            if (w == cid) {
                for (; early < min(STAGES, p.kst); ++early) weights(early, early);
                pdl_wait();
                pdl_trigger();
            }
            for (int kb = 0; kb < p.kst; ++kb) {
                if (kb >= early) {
                    if (!ready) ok = wait_warp_pair(empty(stage), phase ^ 1u, p.wait_limit, abort_flag, peer_abort, p.err, 0x250u);
                    if (!ok) break;
                    weights(stage, kb);
                }
                const uint32_t f = full(stage), sa = sA + stage * A_BYTES;
                if (boxes == 4) tma_elected(sa, &tmA, kb * (SEG_K / 2), arow, f);
                else
                    for (int b = 0; b < boxes; ++b) tma_elected(sa + b * 4096, &tmA32, kb * (SEG_K / 2), arow + 32 * b, f);
                bulk_elected(sS + stage * SFS, a0 + (size_t)kb * SF_BYTES<F>, SF_BYTES<F>, f);
                issued |= 1u << stage;
                last_par = (last_par & ~(1u << stage)) | (phase << stage);
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                ready = kb + 1 >= early && test_warp(empty(stage), phase ^ 1u);
            }
        }
        if (lane == 0)
            for (int s = 0; s < STAGES; ++s)        // every issued copy has landed before the CTA exits
                if (issued & (1u << s)) drain_phase(full(s), (last_par >> s) & 1u, p.err, 0x251u);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            int stage = 0, b = 0, iter = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true, ready = false;
            for (int w = cid; w < total && ok; w += NC, ++iter) {
                for (int kb = 0; kb < p.kst; ++kb) {
                    if (!ready)
                        ok = (kb > 0 || wait_warp_pair(tempty, (iter & 1) ^ 1u, p.wait_limit, abort_flag, peer_abort, p.err, 0x260u)) &&
                             wait_warp_pair(sfull(b), bphase, p.wait_limit, abort_flag, peer_abort, p.err, 0x263u) &&
                             (test_warp(full(stage), phase) ||
                              wait_warp_pair(full(stage), phase, p.wait_limit, abort_flag, peer_abort, p.err, 0x261u));
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t s0 = stage, b0 = b;
                    const bool last = kb + 1 == p.kst;
                    const uint64_t da = sw128_desc(sA + s0 * A_BYTES), db = sw128_desc(sB + s0 * PB_BYTES);
                    const uint32_t d = tm + (iter & 1) * P_ACC2, sfb = tm + P_SF_COL + b0 * COLS,
                                   sfa = tm + P_SFA_COL + (kb & 1) * PIECES * 4;
#pragma unroll
                    for (int q = 0; q < PIECES; ++q) sf_copy_pair(sfa + 4 * q, sS + s0 * SFS + q * 512);
                    const int n = min(4, p.steps - 4 * kb);
                    auto step = [&](int k) {
                        if (k < n) {
                            const int q = F::ID == MOE_FP4_NV ? k : k / 2;
                            const uint32_t id = idesc_scaled<F, 2 * BM, P_BN>(F::ID == MOE_FP4_NV ? 0 : k & 1);
                            mma_scaled_pair<F>(d, da + 2 * k, db + 2 * k, id, sfa + 4 * q, sfb + 8 * q, (kb | k) != 0);
                        }
                    };
                    step(0);
                    step(1);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (++b == P_SF_BUFS) { b = 0; bphase ^= 1u; }
                    const bool t0 = test_phase(full(stage), phase), t1 = test_phase(sfull(b), bphase);
                    step(2);
                    step(3);
                    commit_pair_elected(empty(s0));
                    if (last) commit_pair_elected(tfull);
                    ready = __all_sync(0xffffffffu, t0 && t1 && !last);
                }
            }
            commit_pair_elected(mma_done);          // both CTAs learn when every MMA has finished
        }
    } else if (warp >= 2 + EPI_WARPS) {
        const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16, sfull0 = map_rank(sfull(0), 0);
        int stage = 0, b = 0, old = STAGES - P_SF_BUFS;
        uint32_t phase = 0, ophase = 1;             // (the rounds before the first count as complete)
        bool ok = true, loaded = false;
        for (int w = cid; w < total && ok; w += NC) {
            for (int kb = 0; kb < p.kst; ++kb) {
                if (!loaded) ok = wait_warp_pair(full(stage), phase, p.wait_limit, abort_flag, peer_abort, p.err, 0x271u);
                if (!ok) break;
                const bool t0 = test_phase(empty(old), ophase);
                uint32_t v[COLS];
                const uint32_t src = sS + stage * SFS + SF_BYTES<F> + lane * 16;
#pragma unroll
                for (int q = 0; q < PIECES; ++q) {
                    ld_shared_v4(src + q * 512, v + 8 * q);
                    ld_shared_v4(src + SF_BYTES<F> + q * 512, v + 8 * q + 4);
                }
                if (!__all_sync(0xffffffffu, t0))
                    ok = wait_warp_pair(empty(old), ophase, p.wait_limit, abort_flag, peer_abort, p.err, 0x270u);
                if (!ok) break;
                tc_fence_after();
                const uint32_t dst = tmem + quarter + P_SF_COL + b * COLS;
#pragma unroll
                for (int c = 0; c < COLS; c += 16) {
                    tmem_st16(dst + c, v + c);
                }
                const uint32_t sb = sfull0 + 8u * b;
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                if (++old == STAGES) { old = 0; ophase ^= 1u; }
                if (++b == P_SF_BUFS) b = 0;
                const bool t1 = test_phase(full(stage), phase);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                loaded = __all_sync(0xffffffffu, t1);
                if (lane == 0) arrive_pair(sb);
            }
        }
    } else {
        const int quarter = 32 * (warp & 3), half = (warp - 2) >> 2, r = quarter + lane;
        const uint32_t tempty0 = map_rank(tempty, 0);
        int iter = 0, at = 0;
        for (int w = cid; w < total; w += NC, ++iter) {
            const Work wk = map_pair_item(p, gs, pp, w, rank, at).wk;
            if (!wait_warp_pair(tfull, iter & 1, p.wait_limit, abort_flag, peer_abort, p.err, 0x280u)) break;
            tc_fence_after();
            const uint32_t tbase = tmem + (iter & 1) * P_ACC2 + ((uint32_t)quarter << 16);
            const int nb = min(4, p.NB64 - wk.n * 4);
            auto hand_back = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_pair(tempty0);
            };
            // the chunks whose columns the next tile shares come first: the last two of an even tile, the first two of an odd
            const int first = (iter & 1 ? 0 : 2) + half, second = first ^ 2;
            const bool rows = wk.row0 + quarter < wk.row1, live = wk.row0 + r < wk.row1;
            if (rows && first < nb)
                epilogue_chunk<F, EPI>(p, &tmO, sO + (warp - 2) * P_BOX<EPI>, wk, tbase + 64 * first, wk.n * P_BN + 64 * first, r, live,
                                       hand_back);
            else hand_back();
            if (rows && second < nb)
                epilogue_chunk<F, EPI>(p, &tmO, sO + (warp - 2) * P_BOX<EPI>, wk, tbase + 64 * second, wk.n * P_BN + 64 * second, r, live,
                                       [] {});
        }
        if (lane == 0) bulk_wait_read_all();         // every box read out of shared memory before the CTA exits
    }
    cluster_sync_all();                          // every role of both CTAs has left its loop
    if (warp == 1 && lane == 0) drain_phase(mma_done, 0, p.err, 0x262u);
    tc_fence_before();
    cluster_sync_all();                      // MMAs done, both CTAs' copies landed, all arrivals on the other CTA made
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}


// ---------------------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------------------
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// Codes [rows][pitch bytes], boxes of box_rows x 128 bytes with 128-byte swizzling; zero past the pitch and the rows.
static int codes_map(CUtensorMap* m, const void* base, long long rows, int pitch, int box_rows) {
    auto fn = encode_fn();
    MOE_REQUIRE(fn, MOE_ERR_CUDA, "cuTensorMapEncodeTiled unavailable from the driver");
    cuuint64_t dims[2] = {(cuuint64_t)pitch, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)pitch};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    MOE_REQUIRE(r == CUDA_SUCCESS, MOE_ERR_CUDA, "cuTensorMapEncodeTiled (codes) failed (%d) rows=%lld pitch=%d", (int)r,
                rows, pitch);
    return MOE_OK;
}

// Output [rows][N] of any supported type, boxes of 32 rows x 64 bytes.
static int out_map(CUtensorMap* m, void* base, long long rows, int N, long long ldo, int dtype) {
    auto fn = encode_fn();
    MOE_REQUIRE(fn, MOE_ERR_CUDA, "cuTensorMapEncodeTiled unavailable from the driver");
    const int el = dtype == MOE_F32 ? 4 : 2;
    cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ldo * el};
    cuuint32_t box[2] = {(cuuint32_t)(64 / el), 32};
    cuuint32_t estr[2] = {1, 1};
    const CUresult r = fn(m, dtype == MOE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : dtype == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    MOE_REQUIRE(r == CUDA_SUCCESS, MOE_ERR_CUDA, "cuTensorMapEncodeTiled (output) failed (%d) rows=%lld N=%d", (int)r, rows, N);
    return MOE_OK;
}

// The tensor maps of a launch; the output is stored by TMA where its rows allow a map (16-byte aligned rows).
template <int EPI>
static int make_maps(const void* a_codes, long long rows, int K, Params& p, CUtensorMap* m, CUtensorMap* m32, CUtensorMap* mo) {
    const int pitch = pad64(K) / 2;
    if (int rc = codes_map(m32, a_codes, rows, pitch, 32)) return rc;
    *m = *m32;                                   // (no tile of 128 rows: the map of whole tiles is not used)
    if (rows > 96)
        if (int rc = codes_map(m, a_codes, rows, pitch, BM)) return rc;
    *mo = *m;
    if (EPI == EPI_OUT) {
        const int el = p.out_dtype == MOE_F32 ? 4 : 2;
        p.vec = aligned16(p.out) && (long long)p.ldo * el % 16 == 0;
        // (a box that its map cuts is written in whole 16-byte pieces: 45 fp32 columns in rows of 48 came with three zeros)
        p.boxed = p.vec && rows >= 32 && (long long)p.N * el % 16 == 0;
        if (p.boxed)
            if (int rc = out_map(mo, p.out, rows, p.N, p.ldo, p.out_dtype)) return rc;
    }
    return MOE_OK;
}

template <class F, class C, int EPI>
static int launch(const void* a_codes, long long rows, int K, Params p, cudaStream_t s) {
    constexpr int smem = C::template SMEM<F>;
    static_assert(smem <= 227 * 1024, "shared memory per CTA");
    static unsigned long long attr_ctx[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return set_error(MOE_ERR_CUDA, "fp4 product: no usable current device");
    const unsigned long long ctx = context_id();
    if (ctx == 0 || attr_ctx[dev] != ctx) {
        const cudaError_t e = cudaFuncSetAttribute(fp4_gemm_kernel<F, C, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "fp4 product smem attribute: %s", cudaGetErrorString(e));
        attr_ctx[dev] = context_id();
    }
    CUtensorMap m, m32, mo;
    if (int rc = make_maps<EPI>(a_codes, rows, K, p, &m, &m32, &mo)) return rc;
    p.NT = cdiv(p.NB64, C::BN / 64);
    return check_launch(launch_pdl(fp4_gemm_kernel<F, C, EPI>, dim3(num_sms()), dim3(THREADS), smem, s, m, m32, mo, p),
                        EPI == EPI_SWIGLU ? "fp4_gemm_kernel<swiglu>" : "fp4_gemm_kernel");
}

template <class F, int EPI>
static int launch_pair(const void* a_codes, long long rows, int K, Params p, cudaStream_t s) {
    constexpr int smem = P_SMEM<F, EPI>;
    static int clusters[64];                     // resident pairs, in the context they were asked for
    static unsigned long long attr_ctx[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return set_error(MOE_ERR_CUDA, "fp4 product: no usable current device");
    const unsigned long long ctx = context_id();
    if (!clusters[dev] || ctx == 0 || attr_ctx[dev] != ctx) {
        cudaError_t e = cudaFuncSetAttribute(fp4_gemm_pair_kernel<F, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "fp4 product smem attribute: %s", cudaGetErrorString(e));
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (num_sms() / 2));
        cfg.blockDim = dim3(THREADS);
        cfg.dynamicSmemBytes = smem;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, fp4_gemm_pair_kernel<F, EPI>, &cfg);
        if (e != cudaSuccess || n <= 0)
            return set_error(MOE_ERR_CUDA, "fp4 product: no resident cluster of two CTAs (%s)", cudaGetErrorString(e));
        clusters[dev] = std::min(n, num_sms() / 2);
        attr_ctx[dev] = context_id();
    }
    CUtensorMap m, m32, mo;
    if (int rc = make_maps<EPI>(a_codes, rows, K, p, &m, &m32, &mo)) return rc;
    p.NT = cdiv(p.NB64, 4);
    return check_launch(launch_pdl(fp4_gemm_pair_kernel<F, EPI>, dim3(2 * clusters[dev]), dim3(THREADS), smem, s, m, m32, mo, p),
                        EPI == EPI_SWIGLU ? "fp4_gemm_pair_kernel<swiglu>" : "fp4_gemm_pair_kernel");
}

using Wide = Cfg<192, 4>;
using Mid = Cfg<128, 5>;
using Narrow = Cfg<64, 7>;

// The tile by the time that its waves take on the SMs there are: a stage takes the MMA warp 490, 500 or 530 cycles (64, 128,
// 192 columns; a pair 560), and its bytes about one cycle for each 55, a tile's start and end 2000. The host does not know
// the groups' sizes: a group is taken to end in the middle of a tile. With few rows a call is bound by the weights' bytes,
// and a narrow tile moves too few of them a stage: one token through 8 of 32 experts of 7168 x 2048, gate and up, 36 us with
// 64 columns and 26 with 128; 8192 rows by 8 x 4096 x 12288 (MX), 225 us with 192 columns and 185 by pairs. Pairs are left out
// below 128 rows a group on average, where most groups fill half a pair: with them at 127 rows by 128 x 1536 x 2048 (NV)
// 70 -> 76 us, by 32 x 4096 x 4096 70 -> 75; six groups of 2500 and 122 of 8, which the average leaves out too, 91 either way.
template <class F, int EPI>
static int product(const void* a_codes, long long rows, int G, int K, const Params& p, cudaStream_t s) {
    MOE_REQUIRE((long long)sched_max_tiles(rows, G) * p.NB64 < (1LL << 31), MOE_ERR_INVALID_ARG,
                "4-bit product: %lld rows by %d columns are over 2^31 tiles", rows, p.NB64 * 64);
    const long long used = std::min<long long>(rows, G), kst = stages_of(K), sms = num_sms();
    const long long tiles = std::max(used, used / 2 + rows / BM), pairs = std::max(used, used / 2 + rows / (2 * BM));
    const long long a_bytes = std::min<long long>(4, cdiv(rows, 32 * tiles)) * 4096 + SF_BYTES<F>;
    auto cost = [&](long long m, int blocks, long long units, long long issue, long long b_bytes) {
        return (m * cdiv(p.NB64, blocks) + units - 1) / units * (kst * std::max(issue, (a_bytes + b_bytes) / 55) + 2000);
    };
    const long long c1 = cost(tiles, 1, sms, 490, 8192 + SF_BYTES<F>), c2 = cost(tiles, 2, sms, 500, 16384 + SF_BYTES<F>),
                    c3 = cost(tiles, 3, sms, 530, 24576 + 2 * SF_BYTES<F>);
    const long long c4 = rows >= 128LL * G ? cost(pairs, 4, std::max(1LL, sms / 2), 560, 16384 + 2 * SF_BYTES<F>) : c3 + 1;
    const long long best = std::min(std::min(c1, c2), std::min(c3, c4));
    if (c4 == best) return launch_pair<F, EPI>(a_codes, rows, K, p, s);
    if (c3 == best) return launch<F, Wide, EPI>(a_codes, rows, K, p, s);
    if (c2 == best) return launch<F, Mid, EPI>(a_codes, rows, K, p, s);
    return launch<F, Narrow, EPI>(a_codes, rows, K, p, s);
}

static Params params_for(const int32_t* offsets, const int32_t* sched, unsigned* err, int G, int rows, const void* a_sf, const void* packed, const WeightLayout& L,
                         int K) {
    Params p{};
    p.offsets = offsets;
    p.sched = sched;
    p.G = G;
    p.rows = rows;
    p.max_tiles = (int)sched_max_tiles(rows, G);
    p.a_sf = static_cast<const uint8_t*>(a_sf);
    p.w = static_cast<const uint8_t*>(packed);
    p.w_sf = p.w + L.sf_off;
    p.steps = (K + 63) / 64;
    p.kst = L.KST;
    p.NB64 = L.NB64;
    p.NB128 = L.NB128;
    p.err = err;
    p.wait_limit = wait_limit();
    return p;
}

// Workspace: the schedule of the groups (when the caller has none), each operand's codes and scales, and x's rows quantised
// once where src names them several times.
struct LinearWs { size_t sched, codes, sf, once, total; };
static LinearWs linear_ws(int G, int K, int rows, int fmt) {
    LinearWs w;
    w.sched = 0;
    w.codes = align_up(sched_words(rows, G) * sizeof(int32_t), 1024);
    w.sf = w.codes + operand_codes_bytes(rows, K);
    w.once = w.sf + operand_sf_bytes(rows, G, K, fmt);
    w.total = w.once + gathered_bytes(rows / 2, K, fmt);     // (x has at most rows / 2 rows where they are quantised once)
    return w;
}
struct FfnWs { LinearWs x; size_t act_codes, act_sf, total; };
static FfnWs ffn_ws(int E, int h, int F, int rows, int fmt) {
    FfnWs w;
    w.x = linear_ws(E, h, rows, fmt);
    w.act_codes = w.x.total;
    w.act_sf = w.act_codes + operand_codes_bytes(rows, F);
    w.total = w.act_sf + operand_sf_bytes(rows, E, F, fmt);
    return w;
}

}  // namespace fp4
}  // namespace moe

using namespace moe;
using namespace moe::fp4;

static bool fp4_dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }
static int fp4_el(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// The checks that the product and the FFN share. K: x's columns, N: the output's.
static int check_call(const char* who, const void* x, long long ldx, int x_rows, const int32_t* src, const int32_t* offsets,
                      const int32_t* tile_sched, const void* packed, int G, int N, int K, int rows, int fmt, int dtype,
                      const void* out, long long ldo, int out_dtype, const void* ws) {
    MOE_REQUIRE(fp4_dtype_ok(dtype) && fp4_dtype_ok(out_dtype), MOE_ERR_UNSUPPORTED, "%s: dtype %d, out_dtype %d", who, dtype,
                out_dtype);
    MOE_REQUIRE(fmt == MOE_FP4_NV || fmt == MOE_FP4_MX, MOE_ERR_UNSUPPORTED, "%s: format %d", who, fmt);
    MOE_REQUIRE(G >= 1 && G <= 1024 && N >= 1 && N <= MOE_FP4_MAX_K && K >= 1 && K <= MOE_FP4_MAX_K && rows >= 0 &&
                    rows <= MOE_FP4_MAX_ROWS && x_rows >= 0,
                MOE_ERR_INVALID_ARG, "%s: groups=%d N=%d K=%d rows=%d x_rows=%d", who, G, N, K, rows, x_rows);
    MOE_REQUIRE(ldx >= K && ldo >= N && ldo <= 0x7FFFFFFFLL, MOE_ERR_INVALID_ARG, "%s: ldx=%lld ldo=%lld", who, ldx, ldo);
    MOE_REQUIRE(src || x_rows >= rows, MOE_ERR_INVALID_ARG, "%s: x has %d rows, %d wanted", who, x_rows, rows);
    MOE_REQUIRE((offsets != nullptr) != (tile_sched != nullptr), MOE_ERR_INVALID_ARG,
                "%s: offsets or tile_sched, one of the two", who);
    if (rows == 0) return MOE_OK;
    MOE_REQUIRE((x || x_rows == 0) && packed && out && ws, MOE_ERR_INVALID_ARG, "%s: null pointer", who);
    MOE_REQUIRE(aligned16(packed) && (!tile_sched || aligned16(tile_sched)) &&
                    (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && reinterpret_cast<uintptr_t>(x) % fp4_el(dtype) == 0 &&
                    reinterpret_cast<uintptr_t>(out) % fp4_el(out_dtype) == 0,
                MOE_ERR_INVALID_ARG, "%s: packed and tile_sched must be 16-byte aligned, ws 256-byte, x and out to their type",
                who);
    return MOE_OK;
}

extern "C" size_t moe_fp4_linear_workspace_size(int G, int K, int rows, int fmt) {
    if (G < 1 || G > 1024 || K < 1 || K > MOE_FP4_MAX_K || rows < 0 || rows > MOE_FP4_MAX_ROWS) return 0;
    return linear_ws(G, K, rows, fmt).total;
}

extern "C" int moe_fp4_linear(const void* x, long long ldx, int x_rows, const int32_t* src, const int32_t* offsets,
                              const int32_t* tile_sched, const void* packed, const float* alpha, const float* gscale, int G,
                              int N, int K, int rows, int fmt, int dtype, void* out, long long ldo, int out_dtype, void* ws,
                              size_t ws_bytes, void* stream) {
    if (int rc = check_call("moe_fp4_linear", x, ldx, x_rows, src, offsets, tile_sched, packed, G, N, K, rows, fmt, dtype, out,
                            ldo, out_dtype, ws))
        return rc;
    if (rows == 0) return MOE_OK;
    const LinearWs L = linear_ws(G, K, rows, fmt);
    MOE_REQUIRE(ws_bytes >= L.total, MOE_ERR_WORKSPACE, "moe_fp4_linear: workspace %zu < %zu", ws_bytes, L.total);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* w = static_cast<uint8_t*>(ws);
    unsigned* err = device_error_word();
    int32_t* sched = offsets ? reinterpret_cast<int32_t*>(w + L.sched) : const_cast<int32_t*>(tile_sched);
    if (int rc = launch_quantize_operand(x, ldx, x_rows, src, offsets, sched, G, rows, K, dtype, fmt, gscale, w + L.codes,
                                         w + L.sf, quantize_once(src, x_rows, rows, K) ? w + L.once : nullptr, err, s))
        return rc;
    Params p = params_for(offsets, sched, err, G, rows, w + L.sf, packed, weight_layout(G, N, K, fmt), K);
    p.N = N;
    p.ldo = (int)ldo;
    p.out = out;
    p.out_dtype = out_dtype;
    p.alpha = alpha;
    return fmt == MOE_FP4_NV ? product<Nv, EPI_OUT>(w + L.codes, rows, G, K, p, s)
                             : product<Mx, EPI_OUT>(w + L.codes, rows, G, K, p, s);
}

extern "C" size_t moe_fp4_expert_ffn_workspace_size(int E, int h, int F, int rows, int fmt) {
    if (E < 1 || E > 1024 || h < 1 || h > MOE_FP4_MAX_K || F < 1 || F > MOE_FP4_MAX_K || rows < 0 || rows > MOE_FP4_MAX_ROWS)
        return 0;
    return ffn_ws(E, h, F, rows, fmt).total;
}

extern "C" int moe_fp4_expert_ffn(const void* x, long long ldx, int x_rows, const int32_t* src, const int32_t* offsets,
                                  const int32_t* tile_sched, const void* packed, const float* alpha_gate,
                                  const float* alpha_up, const float* alpha_down, const float* gscale,
                                  const float* act_gscale, int E, int h, int F, int rows, int fmt, int dtype, void* out,
                                  long long ldo, int out_dtype, void* ws, size_t ws_bytes, void* stream) {
    if (int rc = check_call("moe_fp4_expert_ffn", x, ldx, x_rows, src, offsets, tile_sched, packed, E, h, h, rows, fmt, dtype,
                            out, ldo, out_dtype, ws))
        return rc;
    MOE_REQUIRE(F >= 1 && F <= MOE_FP4_MAX_K, MOE_ERR_INVALID_ARG, "moe_fp4_expert_ffn: F=%d", F);
    if (rows == 0) return MOE_OK;
    const FfnWs L = ffn_ws(E, h, F, rows, fmt);
    MOE_REQUIRE(ws_bytes >= L.total, MOE_ERR_WORKSPACE, "moe_fp4_expert_ffn: workspace %zu < %zu", ws_bytes, L.total);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* w = static_cast<uint8_t*>(ws);
    unsigned* err = device_error_word();
    int32_t* sched = offsets ? reinterpret_cast<int32_t*>(w + L.x.sched) : const_cast<int32_t*>(tile_sched);
    if (int rc = launch_quantize_operand(x, ldx, x_rows, src, offsets, sched, E, rows, h, dtype, fmt, gscale, w + L.x.codes,
                                         w + L.x.sf, quantize_once(src, x_rows, rows, h) ? w + L.x.once : nullptr, err, s))
        return rc;
    const ExpertLayout W = expert_layout(E, h, F, fmt);
    Params p = params_for(offsets, sched, err, E, rows, w + L.x.sf, packed, W.gu, h);
    p.alpha = alpha_gate;
    p.alpha_up = alpha_up;
    p.act_gscale = act_gscale;
    p.act_codes = w + L.act_codes;
    p.act_sf = w + L.act_sf;
    p.act_pitch = pad64(F) / 2;
    p.act_kst = stages_of(F);
    if (int rc = fmt == MOE_FP4_NV ? product<Nv, EPI_SWIGLU>(w + L.x.codes, rows, E, h, p, s)
                                   : product<Mx, EPI_SWIGLU>(w + L.x.codes, rows, E, h, p, s))
        return rc;
    Params d = params_for(offsets, sched, err, E, rows, w + L.act_sf, static_cast<const uint8_t*>(packed) + W.down_off, W.down, F);
    d.N = h;
    d.ldo = (int)ldo;
    d.out = out;
    d.out_dtype = out_dtype;
    d.alpha = alpha_down;
    return fmt == MOE_FP4_NV ? product<Nv, EPI_OUT>(w + L.act_codes, rows, E, F, d, s)
                             : product<Mx, EPI_OUT>(w + L.act_codes, rows, E, F, d, s);
}
