// Routing by groups of experts: softmax or sigmoid scores, a selection bias, the best groups, top-k of their experts,
// gates renormalised and scaled; and the gradient of the logits.
//
//   s = sigmoid(L) or softmax(L);  sel_e = s_e + bias_e, -1e30 where L_e = -inf (a masked expert) or is NaN
//   score of a group = the sum of its `best` (1 or 2) largest sel; the top_groups best groups stay, equal scores: lower index
//   the k experts of those groups with the largest sel, equal ones: lower index
//   gate_j = scale * s_j, or scale * s_j / (sum of the chosen s) (0 where all of them are below e^-700)
// The choice is that of exact scores: two scores that 32 bits cannot tell apart are compared in 64. Without a bias the
// experts are ranked by the logits themselves (both scores rise with them), masked ones last, which needs no such comparison.
//
// One warp to a token. A group is a run of lpg lanes, a power of two, and a lane holds npl of its group's experts in a row (the last
// lanes of a group fewer), so that equal scores go to the lowest lane. Where that were over 32 experts to a lane (9 groups of 100), lane l
// holds the experts l npl .. l npl + npl - 1 and the groups' scores go through shared memory.
// (16384 tokens by 8 groups of 37: 67 us that way, 43 with runs of lanes; 4 of 50: 57 and 29; 16 of 48: 166 and 96.)
#include <math.h>
#include <algorithm>
#include "common.cuh"
#include "group_router.cuh"
#include "router.cuh"

namespace moe {

namespace {
constexpr int kWarps = 8;
constexpr int kMaxBlocks = 1024;             // rows of the per-block partial sums in the workspace
constexpr int kMaxK = 16, kMaxGroups = 32, kMaxE = 1024;
constexpr int kMaxT = 1 << 30;               // (a warp's steps through the tokens stay within an int)
constexpr float kMasked = -1e30f;

struct Args {
    const float* logits;                     // the sum of nparts parts, part_stride apart
    int nparts;
    size_t part_stride;
    const float* bias;                       // or null
    int T, E, k, groups, per, top_groups, best, npl, lpg, lpg_log;   // per: experts of a group; lpg: lanes of a group, or 0
    bool sigmoid, renorm, vec;
    float scale;
    float* logits_out;                       // or null
    int32_t* ids;
    float* gates;
    float* partial_P;
    int32_t* partial_C;
    unsigned* ticket;
    int32_t* counts;                         // null, or of a single block that finalizes too: counts, f, P, aux
    float *f, *P, *aux;
    float alpha;
};

// A lane's first expert, and how many it holds.
struct Held { int e0, n; };
__device__ __forceinline__ Held held_by(const Args& a, int lane) {
    if (!a.lpg) return Held{lane * a.npl, min(max(a.E - lane * a.npl, 0), a.npl)};
    const int at = (lane & (a.lpg - 1)) * a.npl, g = lane >> a.lpg_log;
    return Held{g * a.per + at, g < a.groups ? min(max(a.per - at, 0), a.npl) : 0};
}

__device__ __forceinline__ unsigned key_of(float v) {
    const unsigned u = __float_as_uint(v + 0.f);               // (-0 as 0)
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// What follows runs for a token in some thousands, by one warp, and its latency is the call's: 64-bit arithmetic takes sixteen cycles an
// instruction to issue and some sixty until its result, so scores are computed four at a time and compared as whole numbers (compared
// and summed in turn as doubles, one such token made the call 40 us longer).
// A selection score in 64 bits; m and z: softmax's largest logit and sum (z 0: sigmoid).
__device__ __forceinline__ double exact_sel(float l, float bias, double m, double z) {
    if (!(l > -INFINITY)) return (double)kMasked;
    const double e = exp(z == 0.0 ? -(double)l : (double)l - m), v = (z == 0.0 ? 1.0 : e) / (z == 0.0 ? 1.0 + e : z) + (double)bias;
    return v == v ? v : (double)kMasked;
}
// Its order as a whole number, and back.
__device__ __forceinline__ long long order_of(double v) {
    const long long b = __double_as_longlong(v + 0.0);
    return b >= 0 ? b : b ^ 0x7fffffffffffffffLL;
}
__device__ __forceinline__ double of_order(long long b) { return __longlong_as_double(b >= 0 ? b : b ^ 0x7fffffffffffffffLL); }
constexpr long long kLeast = -0x7fffffffffffffffLL - 1;
// The order of a group's score, the sum of the scores in these two places; opposite infinities: as masked.
__device__ __forceinline__ long long order_of_sum(long long b1, long long b2) {
    const double v = of_order(b1) + of_order(b2);
    return order_of(v == v ? v : (double)kMasked);
}

struct Norm { double m, z; };
__device__ __noinline__ Norm exact_norm(const float* L, int npl) {
    float m = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < npl; ++i) m = fmaxf(m, L[i]);
    Norm n{(double)warp_max(m), 0.0};
    double z[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 1
    for (int i = 0; i < npl; i += 4)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] += i + j < npl && L[i + j] > -INFINITY ? exp((double)L[i + j] - n.m) : 0.0;
    n.z = (z[0] + z[1]) + (z[2] + z[3]);
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) n.z += __shfl_xor_sync(0xffffffffu, n.z, o);
    return n;
}

// The groups that stay, in 64 bits: bit g of the result; sel: this lane's scores' order. Whole warp, as the two below; L: this lane's npl
// logits (-inf past E).
__device__ __noinline__ unsigned groups_exact(const Args& a, const float* L, long long* sel) {
    const int lane = threadIdx.x & 31, npl = a.npl;
    const Held h = held_by(a, lane);
    const Norm n = a.sigmoid ? Norm{0.0, 0.0} : exact_norm(L, npl);
#pragma unroll 1
    for (int i = 0; i < npl; i += 4) {
        double v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool live = i + j < h.n;
            v[j] = exact_sel(live ? L[i + j] : 0.f, a.bias && live ? a.bias[h.e0 + i + j] : 0.f, n.m, n.z);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < npl) sel[i + j] = i + j < h.n ? order_of(v[j]) : kLeast;
    }
    long long gscore = kLeast;               // lane g: group g's
    if (a.lpg) {                             // a group is a run of lanes: all at once
        long long t1 = kLeast, t2 = kLeast;
#pragma unroll 1
        for (int i = 0; i < npl; ++i) {
            t2 = max(t2, min(t1, sel[i]));
            t1 = max(t1, sel[i]);
        }
#pragma unroll 1
        for (int o = 1; o < a.lpg; o <<= 1) {
            const long long b1 = __shfl_xor_sync(0xffffffffu, t1, o), b2 = __shfl_xor_sync(0xffffffffu, t2, o);
            t2 = max(min(t1, b1), max(t2, b2));
            t1 = max(t1, b1);
        }
        const long long v = a.best == 2 ? order_of_sum(t1, t2) : t1;
        gscore = __shfl_sync(0xffffffffu, v, min(lane << a.lpg_log, 31));
        if (lane >= a.groups) gscore = kLeast;
    } else
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
        long long t1 = kLeast, t2 = kLeast;
        const int lo = max(g * a.per - h.e0, 0), hi = min((g + 1) * a.per - h.e0, npl);
#pragma unroll 1
        for (int i = lo; i < hi; ++i) {
            t2 = max(t2, min(t1, sel[i]));
            t1 = max(t1, sel[i]);
        }
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) {
            const long long b1 = __shfl_xor_sync(0xffffffffu, t1, o), b2 = __shfl_xor_sync(0xffffffffu, t2, o);
            t2 = max(min(t1, b1), max(t2, b2));
            t1 = max(t1, b1);
        }
        if (lane == g) gscore = a.best == 2 ? order_of_sum(t1, t2) : t1;
    }
    int rank = 0;
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
        const long long o = __shfl_sync(0xffffffffu, gscore, g);
        rank += o > gscore || (o == gscore && g < lane);
    }
    return __ballot_sync(0xffffffffu, lane < a.groups && rank < a.top_groups);
}

struct Candidate { float l, bias; int e, pad; };

// The same where a group is a run of lanes and this lane's group has the score gs in 32 bits, t1 and t2 the largest of its selection
// scores v: only the groups with scores in [lo, hi] may stay or not (what is above stays: fewer than top_groups scores can be above its
// own; what is below does not), and of those only the experts within tol of the ones that count are looked at, one to a lane. list: 32 of
// the warp's own. (Every expert in 64 bits, eight to a lane: 4 us of a call's 33.)
__device__ __noinline__ unsigned groups_near(const Args& a, const float* L, const float* v, Candidate* list, float gs, float t1, float t2,
                                             float lo, float hi, float tol) {
    const int lane = threadIdx.x & 31, npl = a.npl, g = lane >> a.lpg_log;
    const Held h = held_by(a, lane);
    const bool is = g < a.groups, first = is && lane == g << a.lpg_log, near = is && gs >= lo && gs <= hi;
    const unsigned near_at = __ballot_sync(0xffffffffu, first && near), above_at = __ballot_sync(0xffffffffu, first && gs > hi);
    unsigned mine = 0u;                      // slots of this lane
    const float least = (a.best == 2 ? t2 : t1) - tol;
#pragma unroll 1
    for (int i = 0; i < h.n; ++i)
        if (near && v[i] >= least) mine |= 1u << i;
    __syncwarp();
    int at = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += n;
    }
    const int n = __shfl_sync(0xffffffffu, at, 31);
    if (n > 32) {
        long long sel[32];
        return groups_exact(a, L, sel);
    }
    for (at -= __popc(mine); mine; mine &= mine - 1, ++at) {
        const int i = __ffs(mine) - 1;
        list[at] = Candidate{L[i], a.bias ? a.bias[h.e0 + i] : 0.f, h.e0 + i, 0};
    }
    const Norm norm = a.sigmoid ? Norm{0.0, 0.0} : exact_norm(L, npl);
    __syncwarp();
    long long x = kLeast, b1 = kLeast, b2 = kLeast;       // lane j: candidate j; lane g: the best of group g
    int of = -1;
    if (lane < n) {
        x = order_of(exact_sel(list[lane].l, list[lane].bias, norm.m, norm.z));
        of = list[lane].e / a.per;
    }
    __syncwarp();
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        const long long o = __shfl_sync(0xffffffffu, x, j);
        if (__shfl_sync(0xffffffffu, of, j) == lane) {
            b2 = max(b2, min(b1, o));
            b1 = max(b1, o);
        }
    }
    const int at_lane = min(lane << a.lpg_log, 31);
    const bool nearg = lane < a.groups && (near_at >> at_lane & 1u), aboveg = lane < a.groups && (above_at >> at_lane & 1u);
    const long long score = nearg ? (a.best == 2 ? order_of_sum(b1, b2) : b1) : kLeast;
    int rank = 0;
#pragma unroll 1
    for (unsigned left = __ballot_sync(0xffffffffu, nearg); left; left &= left - 1) {
        const int j = __ffs(left) - 1;
        const long long o = __shfl_sync(0xffffffffu, score, j);
        rank += o > score || (o == score && j < lane);
    }
    return __ballot_sync(0xffffffffu, aboveg || (nearg && rank < a.top_groups - __popc(above_at)));
}

// The whole choice in 64 bits; returns lane j's choice j.
__device__ __noinline__ int choose_exact(const Args& a, const float* L) {
    const int lane = threadIdx.x & 31, npl = a.npl;
    const Held h = held_by(a, lane);
    long long sel[32];
    const unsigned kept = groups_exact(a, L, sel);
    unsigned taken = 0u;                     // slots of this lane that are out
#pragma unroll 1
    for (int i = 0; i < npl; ++i) {
        if (i >= h.n || !(kept >> ((h.e0 + i) / a.per) & 1u)) taken |= 1u << i;
        if (!a.bias) sel[i] = order_of((double)fmaxf(L[i], -INFINITY));        // (ranked by the logits; a NaN as masked)
    }
    int my_id = 0;
#pragma unroll 1
    for (int j = 0; j < a.k; ++j) {
        long long v = kLeast;
        int id = 0x7fffffff;
#pragma unroll 1
        for (int i = 0; i < npl; ++i)
            if (!(taken >> i & 1u) && (id == 0x7fffffff || sel[i] > v)) { v = sel[i]; id = h.e0 + i; }
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1) {
            const long long ov = __shfl_xor_sync(0xffffffffu, v, o);
            const int oi = __shfl_xor_sync(0xffffffffu, id, o);
            if (oi != 0x7fffffff && (id == 0x7fffffff || ov > v || (ov == v && oi < id))) { v = ov; id = oi; }
        }
        if (id >= h.e0 && id < h.e0 + h.n) taken |= 1u << (id - h.e0);
        if (lane == j) my_id = id;
    }
    return my_id;
}

// The order of n candidates, lane j's being expert `id` with logit l, where only neighbours among them may be exchanged: a lane computes
// its own score. Returns lane j's expert after ordering.
__device__ __noinline__ int order_exact(const Args& a, const float* L, Candidate* list, float l, int id, int n) {
    const int lane = threadIdx.x & 31;
    long long v = kLeast;
    if (a.bias) {
        const Norm norm = a.sigmoid ? Norm{0.0, 0.0} : exact_norm(L, a.npl);
        if (lane < n) v = order_of(exact_sel(l, a.bias[id], norm.m, norm.z));
    } else if (lane < n) {
        v = order_of((double)fmaxf(l, -INFINITY));
    }
    __syncwarp();
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        const long long o = __shfl_sync(0xffffffffu, v, j);
        const int oi = __shfl_sync(0xffffffffu, id, j);
        rank += o > v || (o == v && oi < id);
    }
    list[lane].e = id;                       // (candidates are different, and ranks a permutation)
    __syncwarp();
    if (lane < n) list[rank].e = id;
    __syncwarp();
    const int out = lane < n ? list[lane].e : id;
    __syncwarp();
    return out;
}

// 2^x and 1 / x of the special-function units: within 2 and 1 units in the last place (0 below the normal range: a score of 2^-126 is
// none).
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.44269504f;

// A sum of scores below this, 2^-40, loses some of them (they are 0 below 2^-126), and its reciprocal may be infinite. Shares in it are
// formed from exp(L - the largest L) instead, to which scores that small are proportional (1 + exp(L) is 1), if the largest score is
// above e^kNoScore. Tokens with such a sum, but for a router's gates, are noted and seen to after the others: in their place the branches
// held up every token (backward of 16384 x 256 9.5 -> 10.5 us).
constexpr float kSmallSum = 9.094947e-13f, kNoScore = -700.f;
// The share of this lane's logit (-inf: none) in the sum of the warp's scores; unit: the logit whose score would be 1.
__device__ __forceinline__ float share_of(float l, float unit) {
    if (!__any_sync(0xffffffffu, l > -INFINITY)) return 0.f;
    const float top = warp_max(l), s = top - unit > kNoScore ? ex2((l - top) * kLog2e) : 0.f, sum = warp_sum(s);
    return sum == 0.f ? 0.f : s * rcp(sum);
}

// Keys by falling order (Batcher's merge exchange).
template <int N>
__device__ __forceinline__ void sort_keys(unsigned (&key)[N]) {
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const unsigned x = key[i + j], y = key[i + j + k];
                        key[i + j] = max(x, y);
                        key[i + j + k] = min(x, y);
                    }
}

// A lane sorts the keys of its experts once, the slot in a key's lowest bits (so that a comparison is a maximum and a minimum), and the
// k rounds compare the lanes' heads without those bits: equal ones go to the lowest lane, and within a lane to the lowest slot. What
// the missing bits, and the roundings of the scores, may have confused is found afterwards from the chosen keys' differences, each lane
// looking at one, and put right in 64 bits.
// (16384 tokens by 256 experts, k 8 of 4 of 8 groups: 25 us with the finalize, from a graph; bound by instructions, 850 a token. When it was
// 29, 2 of them were the tokens that 64 bits decide, and two or four blocks an SM instead of three took 30 and 31. An argmax over
// unsorted slots in every round, with libm's exponential and division, took 45 us of scores and rounds; the whole choice in 64 bits
// 50 us for the one token of some thousands that needs it.)
// FULL: every lane holds NPL experts.
template <int NPL, bool FULL>
__global__ void __launch_bounds__(kWarps * 32, NPL <= 8 ? 3 : NPL <= 16 ? 2 : 1)
group_gate_kernel(const __grid_constant__ Args a) {
    constexpr int SB = NPL == 1 ? 0 : NPL == 2 ? 1 : NPL <= 4 ? 2 : NPL <= 8 ? 3 : NPL <= 16 ? 4 : 5;     // bits of a slot
    constexpr unsigned SLOT = (1u << SB) - 1;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    __shared__ __align__(16) Candidate s_list[kWarps][32];
    float* s_P = reinterpret_cast<float*>(smem_raw);                   // [warps][E]; a warp's row holds its selection scores before
    int* s_hist = reinterpret_cast<int*>(s_P + (size_t)kWarps * a.E);
    pdl_wait();
    pdl_trigger();                            // the finalize may launch now (it waits for this kernel's partials)
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Held h = FULL ? Held{lane * NPL, NPL} : held_by(a, lane);
    const int e0 = h.e0;
    auto live = [&](int i) { return FULL || i < h.n; };
    float* row = s_P + (size_t)warp * a.E;
    float Pacc[NPL], bias[NPL], most = 0.f;  // most: the largest finite magnitude of the bias
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        Pacc[i] = 0.f;
        bias[i] = a.bias && live(i) ? a.bias[e0 + i] : 0.f;
        if (fabsf(bias[i]) < INFINITY) most = fmaxf(most, fabsf(bias[i]));
    }
    if (a.bias) most = warp_max(most);
    bool empty = false;                       // a token whose scores have a small sum
    for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps) {
        alignas(16) float L[NPL];                                    // logits (16 bytes of them a load)
        float s[NPL];                                                // scores
        const float* src = a.logits + (size_t)t * a.E;
#pragma unroll
        for (int i = 0; i < NPL; ++i) L[i] = -INFINITY;
        if (NPL % 4 == 0 && a.vec) {
            if (FULL || h.n > 0) {
#pragma unroll
                for (int i = 0; i < NPL; i += 4) *reinterpret_cast<float4*>(L + i) = *reinterpret_cast<const float4*>(src + e0 + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (live(i)) L[i] = src[e0 + i];
        }
        for (int q = 1; q < a.nparts; ++q) {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (live(i)) L[i] += src[q * a.part_stride + e0 + i];
        }
        if (a.logits_out) {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (live(i)) a.logits_out[(size_t)t * a.E + e0 + i] = L[i];
        }
        // scores (0 of what is masked or past E)
        float total = 0.f, m = 0.f, smax = 1.f;
        if (!a.sigmoid) {
            m = L[0];
#pragma unroll
            for (int i = 1; i < NPL; ++i) m = fmaxf(m, L[i]);
            m = warp_max(m);
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            if (a.sigmoid) s[i] = rcp(1.f + ex2(-kLog2e * L[i]));
            else s[i] = L[i] != -INFINITY ? ex2((L[i] - m) * kLog2e) : 0.f;
            total += s[i];
        }
        total = warp_sum(total);
        const float inv = total < kSmallSum ? 0.f : rcp(total);      // (softmax's total is 1 or more, or 0 where all are masked)
        if (total < kSmallSum) {
            bool some = false;
#pragma unroll
            for (int i = 0; i < NPL; ++i) some = some || L[i] > kNoScore;
            empty = __any_sync(0xffffffffu, some) || empty;
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) Pacc[i] += s[i] * inv;
        if (!a.sigmoid) {
            smax = inv;
#pragma unroll
            for (int i = 0; i < NPL; ++i) s[i] *= inv;
        }
        // Selection scores; the group's score is of s + bias, the experts' order without a bias that of the logits. The error of s: sigmoid's
        // exponential and reciprocal, 2^-22 and 2^-24 of it and the rounding of -L log2(e) (|L| s (1 - s) is below 0.3); softmax's
        // adds the rounded difference of the logits and the sum.
        const float serr = a.sigmoid ? 3e-7f : 1e-6f * smax + 6e-8f;
        float t1 = -INFINITY, t2 = -INFINITY;
        unsigned key[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const float v = s[i] + bias[i];
            const bool in = L[i] > -INFINITY && v == v;
            const float sel = in ? v : kMasked;
            // (without a bias: the logit, and for what is masked one below all of them)
            key[i] = live(i) ? (key_of(a.bias ? sel : in ? L[i] : -INFINITY) & ~SLOT) | (SLOT - i) : 0u;
            if (live(i)) {
                t2 = fmaxf(t2, fminf(t1, sel));
                t1 = fmaxf(t1, sel);
                if (!FULL && !a.lpg) row[e0 + i] = sel;
            }
        }
        if (a.top_groups < a.groups) {
            int g = lane;                     // this lane's group
            if (FULL || a.lpg) {
                g = lane >> a.lpg_log;
                for (int o = 1; o < a.lpg; o <<= 1) {
                    const float b1 = __shfl_xor_sync(0xffffffffu, t1, o), b2 = __shfl_xor_sync(0xffffffffu, t2, o);
                    t2 = fmaxf(fminf(t1, b1), fmaxf(t2, b2));
                    t1 = fmaxf(t1, b1);
                }
            } else {
                __syncwarp();
                t1 = t2 = -INFINITY;
                if (lane < a.groups)
                    for (int i = 0; i < a.per; ++i) {
                        const float v = row[lane * a.per + i];
                        t2 = fmaxf(t2, fminf(t1, v));
                        t1 = fmaxf(t1, v);
                    }
                __syncwarp();
            }
            const float two = t1 + t2, gs = a.best == 1 ? t1 : two == two ? two : kMasked;      // (opposite infinities: as masked)
            int rank = 0;
            for (int o = 0; o < a.groups; ++o) {
                const float v = __shfl_sync(0xffffffffu, gs, FULL || a.lpg ? o << a.lpg_log : o);
                rank += v > gs || (v == gs && o < g);
            }
            const bool is = g < a.groups;
            bool stays = is && rank < a.top_groups;
            const float x = value_of(__reduce_min_sync(0xffffffffu, stays ? key_of(gs) : 0xffffffffu)),
                        y = value_of(__reduce_max_sync(0xffffffffu, is && !stays ? key_of(gs) : 0u));
            // the last that stays and the first that does not: two scores' errors each, and the roundings of their sums with the bias (which
            // may leave a small sum of large terms) and of the groups'.
            // (Finite: infinite sums are equal, and above all others.)
            // Without a bias the errors are relative to the scores: 5e-7 for the exponential, the quotient and the sums; and the exponential's
            // argument is off by 7.3e-8 of itself (sigmoid: log2(e) and the product, rounded) or 1.35e-7 (softmax: the difference of the logits
            // too), which is the error of its power for each unit. The argument is the score's logarithm, at most one more
            // than that of the group's; an exponential below 2^-126 is 0. (The differences of all groups above or below these two are larger than
            // their errors likewise: the error grows more slowly than the score.)
            const float below = fmaxf(-__log2f(fmaxf(y, 1.2e-38f)), 0.f);        // bits of y below 1
            const float tol = a.bias ? fminf(4.f * (serr + 7e-8f * (1.f + most)) + 1.3e-7f * (fabsf(x) + fabsf(y)), 3e38f)
                                     : (1.6e-6f + (a.sigmoid ? 1.4e-7f : 2.5e-7f) * below) * x + 5e-38f;
            // (groups without a live expert, or with one less than `best`, have whole multiples of the masked score: equal)
            bool undecided = !(x - y > tol) && x > 0.1f * kMasked;
            if (undecided && (FULL || a.lpg) && x == y) {
                // equal scores: decided if the logits and biases of the token are all the same (a router at its start)
                bool same = true;
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    const float l0 = __shfl_sync(0xffffffffu, L[0], 0), b0 = __shfl_sync(0xffffffffu, bias[0], 0);
                    if (live(i)) same = same && L[i] == l0 && bias[i] == b0;
                }
                undecided = !__all_sync(0xffffffffu, same);
            }
            unsigned kept = 0u;
            if (undecided) {
                float l[NPL], v[NPL];         // (copies: what they are of stays in registers)
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    l[i] = L[i];
                    v[i] = L[i] > -INFINITY ? s[i] + bias[i] : kMasked;
                }
                if (FULL || a.lpg) {
                    kept = groups_near(a, l, v, s_list[warp], gs, t1, t2, y - tol, x + tol, tol);
                } else {
                    long long sel[32];
                    kept = groups_exact(a, l, sel);
                }
                stays = is && (kept >> g & 1u);
            } else if (!FULL && !a.lpg) {
                kept = __ballot_sync(0xffffffffu, stays);
            }
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (FULL || a.lpg ? !stays : !(kept >> ((e0 + i) / a.per) & 1u)) key[i] = 0u;
        }
        if constexpr (NPL > 1) sort_keys(key);
        // The next best: lane j takes it as its choice. Equal heads go to the lowest lane.
        unsigned my_key = 0u;
        int my_owner = 0;
        auto take = [&](int j) {
            const unsigned head = key[0] >> SB, top = __reduce_max_sync(0xffffffffu, head);
            const int owner = __ffs(__ballot_sync(0xffffffffu, head == top)) - 1;
            const unsigned got = __shfl_sync(0xffffffffu, key[0], owner);
            if (lane == j) {
                my_key = got;
                my_owner = owner;
            }
            const bool pop = lane == owner;
#pragma unroll
            for (int i = 0; i + 1 < NPL; ++i) key[i] = pop ? key[i + 1] : key[i];
            key[NPL - 1] = pop ? 0u : key[NPL - 1];
            return got;
        };
        const int left = a.top_groups * a.per;                    // experts of the kept groups
        int n = min(a.k + 1, left);                               // the k, and the first that is left out
#pragma unroll 2
        for (int j = 0; j < n; ++j) take(j);
        auto id_of = [&] { return (FULL ? my_owner * NPL : held_by(a, my_owner).e0) + (int)(SLOT - (my_key & SLOT)); };
        int my_id = id_of();
        // whether two neighbours' order may be another than their keys'
        auto near = [&](unsigned hi, unsigned lo) {
            if (!a.bias) return (hi >> SB) == (lo >> SB);
            const float x = value_of(hi & ~SLOT), y = value_of(lo & ~SLOT);
            return !(x - y > 2.f * serr + (6.1e-8f + 1.2e-7f * (SLOT + 1)) * (fabsf(x) + fabsf(y))) && x > 0.1f * kMasked;
        };
        auto logit_of = [&](int e) {                              // the parts in their order
            float l = src[e];
            for (int q = 1; q < a.nparts; ++q) l += src[q * a.part_stride + e];
            return l;
        };
        const unsigned next = __shfl_down_sync(0xffffffffu, my_key, 1);      // (by all lanes, not behind a condition)
        const bool close = lane + 1 < n && near(my_key, next);
        float my_l = lane < n ? logit_of(my_id) : -INFINITY;
        if (__any_sync(0xffffffffu, close)) {
            // equal logits with equal biases are equal, and in order; the rest is looked at in 64 bits
            const float b = a.bias && lane < n ? a.bias[my_id] : 0.f;
            const float nl = __shfl_down_sync(0xffffffffu, my_l, 1), nb = __shfl_down_sync(0xffffffffu, b, 1);
            const unsigned bad = __ballot_sync(0xffffffffu, close && !(nl == my_l && nb == b));
            // what is left out may be above something chosen: if the first left out is near the last chosen, unless all that are
            // near one another about there (those before the last from the first gap on; any after it) are equal
            const unsigned chosen = (2u << (a.k - 1)) - 1u, near_bits = __ballot_sync(0xffffffffu, close);
            const bool border = (near_bits >> (a.k - 1) & 1u) != 0;
            const unsigned gaps = ~near_bits & chosen, run = gaps ? chosen & ~((2u << (31 - __clz(gaps))) - 1u) : chosen;
            bool more = border && (bad & run) != 0;
            if (border && !more) {
                const unsigned last = __shfl_sync(0xffffffffu, my_key, a.k - 1);
                const float ll = __shfl_sync(0xffffffffu, my_l, a.k - 1), lb = __shfl_sync(0xffffffffu, b, a.k - 1);
                float l[NPL];
#pragma unroll
                for (int i = 0; i < NPL; ++i) l[i] = L[i];
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    const int slot = (int)(SLOT - (key[i] & SLOT));
                    if (key[i] && near(last, key[i])) more = more || l[slot] != ll || (a.bias && a.bias[e0 + slot] != lb);
                }
                more = __any_sync(0xffffffffu, more);
            }
            if (bad || more) {
                // candidates until a clear distance, if one is within the warp's lanes
                unsigned last = __shfl_sync(0xffffffffu, my_key, n - 1);
                while (more && n < min(left, 32)) {
                    const unsigned got = take(n);
                    ++n;
                    more = near(last, got);
                    last = got;
                }
                float l[NPL];
#pragma unroll
                for (int i = 0; i < NPL; ++i) l[i] = L[i];
                my_id = id_of();
                if (lane < n) my_l = logit_of(my_id);
                my_id = more && n < left ? choose_exact(a, l) : order_exact(a, l, s_list[warp], my_l, my_id, n);
                if (lane < a.k) my_l = logit_of(my_id);
            }
        }
        float my_s = 0.f;
        if (lane < a.k && !(my_l == -INFINITY)) my_s = a.sigmoid ? rcp(1.f + ex2(-kLog2e * my_l)) : ex2((my_l - m) * kLog2e) * inv;
        if (a.renorm) {
            const float sum = warp_sum(my_s);
            if (sum < kSmallSum) my_s = share_of(lane < a.k ? my_l : -INFINITY, a.sigmoid ? 0.f : m);
            else my_s *= rcp(sum);
        }
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = my_id;
            a.gates[(size_t)t * a.k + lane] = my_s * a.scale;
            atomicAdd(&s_hist[my_id], 1);
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        if (live(i)) row[e0 + i] = Pacc[i];
    if (empty && a.sigmoid) {                 // the shares of such tokens' scores
        for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps) {
            const float* src = a.logits + (size_t)t * a.E;
            float l[NPL], top = -INFINITY, total = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                l[i] = live(i) ? src[e0 + i] : -INFINITY;
                for (int q = 1; q < a.nparts; ++q)
                    if (live(i)) l[i] += src[q * a.part_stride + e0 + i];
                top = fmaxf(top, l[i]);
                total += rcp(1.f + ex2(-kLog2e * l[i]));             // (as above)
            }
            top = warp_max(top);
            if (!(warp_sum(total) < kSmallSum) || !(top > kNoScore)) continue;
            total = 0.f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) total += l[i] = ex2((l[i] - top) * kLog2e);
            total = rcp(warp_sum(total));
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (live(i)) row[e0 + i] += l[i] * total;
        }
    }
    __syncthreads();
    if (a.counts) {                           // the only block: counts, f, P and aux as well
        __shared__ float s_term[kWarps];
        float term = 0.f;
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            float v = 0.f;
            for (int w = 0; w < kWarps; ++w) v += s_P[(size_t)w * a.E + e];
            const float P = v / (float)a.T, f = (float)s_hist[e] / ((float)a.k * (float)a.T);
            a.counts[e] = s_hist[e];
            a.f[e] = f;
            a.P[e] = P;
            term += f * P;
        }
        term = warp_sum(term);
        if (lane == 0) s_term[warp] = term;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int w = 1; w < kWarps; ++w) term += s_term[w];
            a.aux[0] = a.alpha * (float)a.E * term;
        }
        return;
    }
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += s_P[(size_t)w * a.E + e];
        a.partial_P[(size_t)blockIdx.x * a.E + e] = v;
        a.partial_C[(size_t)blockIdx.x * a.E + e] = s_hist[e];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0u;          // the finalize runs after this kernel
}

// d_logits of a token by one warp, lane l holding the experts l, l + 32, ... (whole lines are read and written):
//   ds_j = scale d_g_j, or with renormalised gates scale (d_g_j - sum_i d_g_i s_i / S) / S, S = sum_i s_i (0 where S is 0)
//   c_e = d_aux alpha E f_e / T;  softmax: dp = ds + c, d_logits = p (dp - <dp, p>)
//   sigmoid: d_logits = (ds + (c - <c, q>) / sum s) s (1 - s), q = s / sum s
// The ds reach their experts through a row of shared memory that is zero but for them (compared with every slot of every lane instead, and the
// scores taken from the lanes that hold them, a token cost 920 instructions: 16384 x 256 in 19.6 us).
constexpr int kBwdWarps = 8;
// A token whose S is small, or under sigmoid the sum of all its s (so large or infinite ds): t_j = scale (s_j / S) (d_g_j - sum_i d_g_i s_i / S) from the
// shares s_j / S, or scale s_j d_g_j, in place of ds s; under softmax of p (ds - <ds, p>) too, since the t add up to 0. Some expert has a
// score. id, dg: of lane j, choice j and its gate's gradient.
__device__ __forceinline__ void group_gate_backward_small(const float* src, const float* f, int E, int k, int id, float dg, bool sigmoid, bool renorm,
                                                          float scale, float coef, float* out) {
    const int lane = threadIdx.x & 31;
    if (id < 0 || id >= E) id = -1;
    const float l = id >= 0 ? src[id] : -INFINITY;
    float top = -INFINITY, total = 0.f, cq = 0.f;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) top = fmaxf(top, src[e]);
    top = warp_max(top);
    const bool tiny = sigmoid && top < -30.f;
    // scores, of softmax and tiny ones multiples
    auto score = [&](float x) { return sigmoid && !tiny ? rcp(1.f + ex2(-kLog2e * x)) : ex2((x - top) * kLog2e); };
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
        const float s = score(src[e]);
        total += s;
        cq += coef * f[e] * s;
    }
    total = warp_sum(total);
    const float inv = total == 0.f ? 0.f : rcp(total);
    cq = warp_sum(cq) * inv;
    float t = ex2(l * kLog2e) * dg;                                  // (all scores are small: exp(L))
    if (renorm) {
        const float share = share_of(l, sigmoid ? 0.f : top);
        if (id < 0) dg = 0.f;
        t = share * (dg - warp_sum(share * dg));
    }
    t *= scale;
#pragma unroll 1
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        const float x = e < E ? src[e] : -INFINITY;
        float d = e < E ? score(x) * inv * (coef * f[e] - cq) : 0.f;
#pragma unroll 1
        for (int j = 0; j < k; ++j) {
            const int at = __shfl_sync(0xffffffffu, id, j);
            const float v = __shfl_sync(0xffffffffu, t, j);
            if (at == e) d += v;
        }
        if (e < E) out[e] = sigmoid ? d * rcp(1.f + ex2(kLog2e * x)) : d;
    }
}
// (Four blocks an SM are launched, and are all resident up to 256 experts.)
template <int NPL>
__global__ void __launch_bounds__(kBwdWarps * 32, NPL <= 8 ? 4 : 1)
group_gate_backward_kernel(const float* logits, const int32_t* ids, const float* d_gates, const float* f, int T, int E, int k, bool sigmoid,
                           bool renorm, float scale, float coef, float* d_logits, unsigned* err) {
    __shared__ float s_ds[kBwdWarps][32 * NPL];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* row = s_ds[warp];
    float c[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        c[i] = lane + 32 * i < E ? coef * f[lane + 32 * i] : 0.f;
        row[lane + 32 * i] = 0.f;
    }
    __syncwarp();
    const int step = gridDim.x * kBwdWarps;
    for (int t0 = blockIdx.x * kBwdWarps + warp; t0 < T; t0 += 32 * step) {
        unsigned small = 0u, bit = 1u;
        for (int t = t0; t < T && bit; t += step, bit <<= 1) {
            const float* src = logits + (size_t)t * E;
            float s[NPL], n[NPL];                                        // score, 1 - score
#pragma unroll
            for (int i = 0; i < NPL; ++i) s[i] = lane + 32 * i < E ? src[lane + 32 * i] : -INFINITY;
            int id = -1;
            float dg = 0.f, mine = 0.f;                                  // lane j: choice j, its gate's gradient and its score
            if (lane < k) {
                id = ids[(size_t)t * k + lane];
                dg = d_gates[(size_t)t * k + lane];
                if (id < 0 || id >= E) { latch_device_error(err, kDevErrBadIndex, 0x300u); id = -1; }
                if (id >= 0) mine = src[id];
                else dg = 0.f;
            }
            float total = 0.f, m = 0.f, top = -INFINITY;                 // (top: this lane's)
#pragma unroll
            for (int i = 0; i < NPL; ++i) top = fmaxf(top, s[i]);
            if (sigmoid) {
                // e = exp(-|L|): s and 1 - s are 1 / (1 + e) and e / (1 + e), neither a difference
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    const float e = ex2(-kLog2e * fabsf(s[i])), inv = rcp(1.f + e), b = e * inv;
                    const bool up = s[i] >= 0.f;
                    n[i] = up ? b : inv;
                    s[i] = up ? inv : b;
                    total += s[i];
                }
                mine = id >= 0 ? rcp(1.f + ex2(-kLog2e * mine)) : 0.f;
            } else {
                m = warp_max(top);
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    s[i] = s[i] != -INFINITY ? ex2((s[i] - m) * kLog2e) : 0.f;
                    total += s[i];
                }
                mine = id >= 0 && mine != -INFINITY ? ex2((mine - m) * kLog2e) : 0.f;
            }
            total = warp_sum(total);
            const float tinv = total == 0.f ? 0.f : rcp(total);
            if (!sigmoid) {
                mine *= tinv;
#pragma unroll
                for (int i = 0; i < NPL; ++i) s[i] *= tinv;
            }
            float ds = scale * dg, S = total;
            if (renorm) {
                S = warp_sum(mine);
                const float w = warp_sum(mine * dg);
                const float inv = S == 0.f ? 0.f : 1.f / S;
                ds = scale * (dg - w * inv) * inv;
            }
            // a choice that is there twice (no route has one) is added in the choices' order
            const unsigned same = __match_any_sync(0xffffffffu, id >= 0 ? id : -1 - lane);
            const bool first = id >= 0 && lane == __ffs(same) - 1;
            if (__any_sync(0xffffffffu, __popc(same) > 1)) {
                float sum = 0.f;
                for (int j = 0; j < k; ++j) {
                    const float v = __shfl_sync(0xffffffffu, ds, j);
                    if (same >> j & 1u) sum += v;
                }
                ds = sum;
            }
            if (first) row[id] = ds;
            __syncwarp();
            float d[NPL];                                                // gradient of the score
            if (sigmoid) {
                float cq = 0.f;
#pragma unroll
                for (int i = 0; i < NPL; ++i) cq += c[i] * s[i];
                cq = warp_sum(cq) * tinv;
#pragma unroll
                for (int i = 0; i < NPL; ++i) d[i] = row[lane + 32 * i] + (c[i] - cq) * tinv;
#pragma unroll
                for (int i = 0; i < NPL; ++i) d[i] = d[i] * s[i] * n[i];
            } else {
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < NPL; ++i) {
                    d[i] = row[lane + 32 * i] + c[i];
                    dot += d[i] * s[i];
                }
                dot = warp_sum(dot);
#pragma unroll
                for (int i = 0; i < NPL; ++i) d[i] = s[i] * (d[i] - dot);
            }
            __syncwarp();
            if (first) row[id] = 0.f;
            __syncwarp();
            // (its row is not written yet: d_logits may be logits; of tokens without any score all is 0)
            const bool is_small = S < kSmallSum && __any_sync(0xffffffffu, top > (sigmoid ? kNoScore : -INFINITY));
            if (is_small) small |= bit;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (lane + 32 * i < E && !is_small) __stcs(d_logits + (size_t)t * E + lane + 32 * i, d[i]);
        }
        for (; small; small &= small - 1) {
            const size_t t = t0 + (__ffs(small) - 1) * step;
            group_gate_backward_small(logits + t * E, f, E, k, lane < k ? ids[t * k + lane] : -1, lane < k ? d_gates[t * k + lane] : 0.f, sigmoid, renorm, scale,
                                      coef, d_logits + t * E);
        }
    }
}

int grid_of(int T) { return std::max(1, std::min(cdiv(T, kWarps), kMaxBlocks)); }

struct Ws { float* partial_P; int32_t* partial_C; unsigned* ticket; float* term_part; size_t bytes; };
Ws ws_layout(void* ws, int T, int E) {
    Ws w{};
    const size_t G = grid_of(T);
    char* base = static_cast<char*>(ws);
    size_t off = 0;
    w.partial_P = reinterpret_cast<float*>(base + off); off = align_up(off + G * E * 4, 256);
    w.partial_C = reinterpret_cast<int32_t*>(base + off); off = align_up(off + G * E * 4, 256);
    w.ticket = reinterpret_cast<unsigned*>(base + off); off = align_up(off + 4, 256);
    w.term_part = reinterpret_cast<float*>(base + off); off = align_up(off + (size_t)finalize_grid(T, E) * 4, 256);
    w.bytes = off;
    return w;
}

// Launches on as many blocks as are resident at once (into *G; one that finalizes too where a.counts is set). What the runtime says of a
// kernel is kept: asked in every call, it cost a small one two microseconds. (The shared memory is below 48 KB for any E.)
template <int NPL, bool FULL>
int launch_gate(Args& a, int* G, cudaStream_t s) {
    static int per_sm[64];
    static unsigned long long of_ctx[64];
    const auto kernel = group_gate_kernel<NPL, FULL>;
    auto smem_of = [](int E) { return (size_t)kWarps * E * sizeof(float) + (size_t)E * sizeof(int); };
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return set_error(MOE_ERR_CUDA, "group routing: no usable current device");
    const unsigned long long ctx = context_id();
    if (ctx == 0 || of_ctx[dev] != ctx || !per_sm[dev]) {
        int n = 0;
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kWarps * 32, smem_of(32 * NPL));
        per_sm[dev] = e == cudaSuccess && n > 0 ? n : 1;
        of_ctx[dev] = context_id();
    }
    const size_t smem = smem_of(a.E);
    a.vec = a.npl == NPL && NPL % 4 == 0 && a.E % 4 == 0 && aligned16(a.logits) && a.per == a.lpg * NPL;
    *G = a.counts ? 1 : std::min(grid_of(a.T), per_sm[dev] * num_sms());
    return check_launch(launch_pdl(kernel, dim3(*G), dim3(kWarps * 32), smem, s, a), "group_gate_kernel");
}

int check_spec(const char* fn, int T, int E, int k, int groups, int top_groups, int score, int best, float scale) {
    MOE_REQUIRE(score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SOFTMAX, MOE_ERR_UNSUPPORTED, "%s: score %d", fn, score);
    MOE_REQUIRE(T >= 0 && T <= kMaxT && E >= 1 && E <= kMaxE && groups >= 1 && groups <= kMaxGroups && E % groups == 0,
                MOE_ERR_INVALID_ARG, "%s: T=%d E=%d groups=%d (need T <= 2^30, E <= 1024, groups <= 32 of equal size)", fn, T, E, groups);
    MOE_REQUIRE(top_groups >= 1 && top_groups <= groups && (best == 1 || best == 2) && best <= E / groups, MOE_ERR_INVALID_ARG,
                "%s: top_groups=%d best=%d of %d groups of %d", fn, top_groups, best, groups, E / groups);
    MOE_REQUIRE(k >= 1 && k <= kMaxK && k <= top_groups * (E / groups), MOE_ERR_INVALID_ARG,
                "%s: k=%d (need 1 <= k <= 16 and no more than the kept groups' %d experts)", fn, k, top_groups * (E / groups));
    MOE_REQUIRE(isfinite(scale), MOE_ERR_INVALID_ARG, "%s: scale is not finite", fn);
    return MOE_OK;
}
}  // namespace

size_t group_gate_ws_bytes(int T, int E) { return ws_layout(nullptr, T, E).bytes; }

int launch_group_gate(const GroupGate& g, void* ws, cudaStream_t s) {
    const Ws w = ws_layout(ws, g.T, g.E);
    int G = 0;
    if (g.T > 0) {
        Args a{};
        a.logits = g.logits; a.nparts = g.nparts; a.part_stride = g.part_stride;
        a.bias = g.bias; a.logits_out = g.logits_out;
        a.T = g.T; a.E = g.E; a.k = g.k; a.groups = g.groups; a.per = g.E / g.groups; a.top_groups = g.top_groups; a.best = g.best;
        a.sigmoid = g.score == MOE_SCORE_SIGMOID; a.renorm = g.renorm; a.scale = g.scale;
        a.ids = g.ids; a.gates = g.gates; a.partial_P = w.partial_P; a.partial_C = w.partial_C; a.ticket = w.ticket;
        if (a.top_groups == a.groups) {           // no choice of groups
            a.groups = a.top_groups = 1;
            a.per = a.E;
        }
        a.lpg_log = 0;
        while (a.groups << (a.lpg_log + 1) <= 32) ++a.lpg_log;
        a.lpg = 1 << a.lpg_log;
        a.npl = cdiv(a.per, a.lpg);
        if (a.npl > 32) {
            a.lpg = a.lpg_log = 0;
            a.npl = cdiv(a.E, 32);
        }
        // up to two tokens a warp of one block: a second block and the finalize's launch cost more
        if (g.T <= 2 * kWarps) {
            a.counts = g.counts; a.f = g.f; a.P = g.P; a.aux = g.aux; a.alpha = g.alpha;
        }
        const bool full = a.lpg && g.E == 32 * a.npl;
#define MOE_GATE(N) (full && a.npl == N ? launch_gate<N, true>(a, &G, s) : launch_gate<N, false>(a, &G, s))
        // (3 and 5: 96 and 160 experts, without predicates)
        const int rc = a.npl <= 1 ? MOE_GATE(1) : a.npl <= 2 ? MOE_GATE(2) : full && a.npl == 3 ? launch_gate<3, true>(a, &G, s)
                     : a.npl <= 4 ? MOE_GATE(4) : full && a.npl == 5 ? launch_gate<5, true>(a, &G, s) : a.npl <= 6 ? MOE_GATE(6)
                     : a.npl <= 8 ? MOE_GATE(8) : a.npl <= 12 ? MOE_GATE(12) : a.npl <= 16 ? MOE_GATE(16)
                     : a.npl <= 24 ? MOE_GATE(24) : MOE_GATE(32);
#undef MOE_GATE
        if (rc) return rc;
        if (a.counts) return MOE_OK;
    }
    return launch_router_finalize(w.partial_P, w.partial_C, G, g.T, g.E, g.k, g.alpha, g.counts, g.f, g.P, g.aux, w.term_part,
                                  w.ticket, s);
}

int check_group_gate(const char* fn, const GroupGate& g) {
    if (int rc = check_spec(fn, g.T, g.E, g.k, g.groups, g.top_groups, g.score, g.best, g.scale)) return rc;
    MOE_REQUIRE(g.counts && g.f && g.P && g.aux && (g.T == 0 || (g.ids && g.gates)), MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" size_t moe_group_route_workspace_size(int T, int E) {
    if (T < 0 || T > kMaxT || E <= 0) return 0;
    return group_gate_ws_bytes(T, E);
}

extern "C" int moe_group_route(const float* logits, const float* bias, int T, int E, int k, int groups, int top_groups, int score,
                               int best, int renorm, float scale, float alpha, int32_t* topk_ids, float* gates, int32_t* counts,
                               float* f, float* P, float* aux, void* ws, size_t ws_bytes, void* stream) {
    GroupGate g{};
    g.logits = logits; g.nparts = 1; g.bias = bias;
    g.T = T; g.E = E; g.k = k; g.groups = groups; g.top_groups = top_groups; g.score = score; g.best = best;
    g.renorm = renorm != 0; g.scale = scale; g.alpha = alpha;
    g.ids = topk_ids; g.gates = gates; g.counts = counts; g.f = f; g.P = P; g.aux = aux;
    if (int rc = check_group_gate("moe_group_route", g)) return rc;
    MOE_REQUIRE(T == 0 || logits, MOE_ERR_INVALID_ARG, "moe_group_route: null logits");
    const size_t need = group_gate_ws_bytes(T, E);
    MOE_REQUIRE(ws && aligned16(ws) && ws_bytes >= need, MOE_ERR_WORKSPACE, "moe_group_route: workspace %zu < %zu bytes (16-byte aligned)",
                ws_bytes, need);
    return launch_group_gate(g, ws, static_cast<cudaStream_t>(stream));
}

extern "C" int moe_group_route_backward(const float* logits, const int32_t* topk_ids, const float* d_gates, const float* f, int T,
                                        int E, int k, int score, int renorm, float scale, float alpha, float d_aux,
                                        float* d_logits, void* stream) {
    const char* fn = "moe_group_route_backward";
    if (int rc = check_spec(fn, T, E, k, 1, 1, score, 1, scale)) return rc;
    if (T == 0) return MOE_OK;
    MOE_REQUIRE(logits && topk_ids && d_gates && f && d_logits, MOE_ERR_INVALID_ARG, "%s: null pointer", fn);
    unsigned* err = device_error_word();
    MOE_REQUIRE(err, MOE_ERR_CUDA, "%s: device error word unavailable", fn);
    const float coef = d_aux * alpha * (float)E / (float)T;
    const int G = std::min(cdiv(T, kBwdWarps), 4 * num_sms());
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
#define MOE_GROUP_BWD(N)                                                                                                    \
    e = launch_pdl(group_gate_backward_kernel<N>, dim3(G), dim3(kBwdWarps * 32), 0, s, logits, topk_ids, d_gates, f, T, E, k, \
                   score == MOE_SCORE_SIGMOID, renorm != 0, scale, coef, d_logits, err)
    const int n = cdiv(E, 32);
    if (n <= 1) MOE_GROUP_BWD(1);
    else if (n <= 2) MOE_GROUP_BWD(2);
    else if (n <= 4) MOE_GROUP_BWD(4);
    else if (n <= 8) MOE_GROUP_BWD(8);
    else if (n <= 16) MOE_GROUP_BWD(16);
    else MOE_GROUP_BWD(32);
#undef MOE_GROUP_BWD
    return check_launch(e, "group_gate_backward_kernel");
}
