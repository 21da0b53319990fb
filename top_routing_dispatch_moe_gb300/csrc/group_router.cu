// Routing by groups of experts: softmax or sigmoid scores, a selection bias, the best groups, top-k of their experts,
// gates renormalised and scaled; and the gradient of the logits.
//
//   s = sigmoid(L) or softmax(L);  sel_e = s_e + bias_e, -1e30 where L_e = -inf (a masked expert) or is NaN
//   score of a group = the sum of its `best` (1 or 2) largest sel; the top_groups best groups stay, equal scores: lower index
//   the k experts of those groups with the largest sel, equal ones: lower index
//   gate_j = scale * s_j, or scale * s_j / (sum of the chosen s) (0 where that sum is 0)
// The choice is that of exact scores: two scores that 32 bits cannot tell apart are compared in 64. Without a bias the
// experts are ranked by the logits themselves (both scores rise with them), which needs no such comparison.
//
// One warp to a token, lane l holding the experts l npl .. l npl + npl - 1, so that a group is a run of lanes (where its
// size is a multiple of npl; through shared memory otherwise) and equal scores go to the lowest lane.
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
constexpr float kMasked = -1e30f;

struct Args {
    const float* logits;                     // the sum of nparts parts, part_stride apart
    int nparts;
    size_t part_stride;
    const float* bias;                       // or null
    int T, E, k, groups, per, top_groups, best, npl, lpg;   // per: experts of a group; lpg: lanes of a group (0: no whole lanes)
    bool sigmoid, renorm, vec;
    float scale;
    float* logits_out;                       // or null
    int32_t* ids;
    float* gates;
    float* partial_P;
    int32_t* partial_C;
    unsigned* ticket;
};

__device__ __forceinline__ unsigned key_of(float v) {
    const unsigned u = __float_as_uint(v == 0.f ? 0.f : v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(unsigned key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// The choice in 64 bits, for a token with scores that are next to each other. Whole warp; returns lane j's choice j.
__device__ __noinline__ int choose_exact(const Args& a, const float* L, const float* bias, int npl) {
    const int lane = threadIdx.x & 31, e0 = lane * npl;
    double sel[32];
    double m = -INFINITY, z = 1.0;
    if (!a.sigmoid) {
        for (int i = 0; i < npl; ++i)
            if (e0 + i < a.E) m = fmax(m, (double)L[i]);
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        z = 0.0;
        for (int i = 0; i < npl; ++i)
            if (e0 + i < a.E && L[i] > -INFINITY) z += exp((double)L[i] - m);
        for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    for (int i = 0; i < npl; ++i) {
        sel[i] = -INFINITY;
        if (e0 + i < a.E) {
            const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)L[i])) : exp((double)L[i] - m) / z;
            const double v = s + (bias ? (double)bias[e0 + i] : 0.0);
            sel[i] = L[i] > -INFINITY && v == v ? v : (double)kMasked;
        }
    }
    double gscore = 0.0;                     // lane g: group g's
    for (int g = 0; g < a.groups; ++g) {
        double t1 = -INFINITY, t2 = -INFINITY;
        for (int i = 0; i < npl; ++i) {
            const int e = e0 + i;
            if (e < g * a.per || e >= (g + 1) * a.per) continue;
            if (sel[i] > t1) { t2 = t1; t1 = sel[i]; } else if (sel[i] > t2) t2 = sel[i];
        }
        for (int o = 16; o > 0; o >>= 1) {
            const double b1 = __shfl_xor_sync(0xffffffffu, t1, o), b2 = __shfl_xor_sync(0xffffffffu, t2, o);
            const double lo = fmin(t1, b1);
            t1 = fmax(t1, b1);
            t2 = fmax(lo, fmax(t2, b2));
        }
        if (lane == g) gscore = a.best == 2 ? t1 + t2 : t1;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
        const double o = __shfl_sync(0xffffffffu, gscore, g);
        rank += o > gscore || (o == gscore && g < lane);
    }
    const unsigned kept = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.top_groups);
    unsigned taken = 0u;                     // slots of this lane that are out
    for (int i = 0; i < npl; ++i)
        if (e0 + i >= a.E || !(kept >> ((e0 + i) / a.per) & 1u)) taken |= 1u << i;
    int my_id = 0;
    for (int j = 0; j < a.k; ++j) {
        double v = -INFINITY;
        int id = 0x7fffffff;
        for (int i = 0; i < npl; ++i)
            if (!(taken >> i & 1u) && (id == 0x7fffffff || sel[i] > v)) { v = sel[i]; id = e0 + i; }
        for (int o = 16; o > 0; o >>= 1) {
            const double ov = __shfl_xor_sync(0xffffffffu, v, o);
            const int oi = __shfl_xor_sync(0xffffffffu, id, o);
            if (oi != 0x7fffffff && (id == 0x7fffffff || ov > v || (ov == v && oi < id))) { v = ov; id = oi; }
        }
        if (id / npl == lane) taken |= 1u << (id - e0);
        if (lane == j) my_id = id;
    }
    return my_id;
}

// The order of the chosen and the next best where only neighbours among them lie that near (sigmoid scores: each lane j <= k computes
// its own in 64 bits, a hundredth of what the whole choice costs). id, l: lane j's expert and its logit, of
// `n` in all; returns lane j's expert after ordering.
__device__ __noinline__ int order_exact(float l, const float* bias, int id, int n) {
    const int lane = threadIdx.x & 31;
    double v = -INFINITY;
    if (lane < n) {
        v = l > -INFINITY ? 1.0 / (1.0 + exp(-(double)l)) + (double)bias[id] : (double)kMasked;
        if (!(v == v)) v = (double)kMasked;
    }
    int rank = 0;
    for (int j = 0; j < n; ++j) {
        const double o = __shfl_sync(0xffffffffu, v, j);
        const int oi = __shfl_sync(0xffffffffu, id, j);
        rank += o > v || (o == v && oi < id);
    }
    int out = id;
    for (int j = 0; j < n; ++j) {
        const int r = __shfl_sync(0xffffffffu, rank, j), oi = __shfl_sync(0xffffffffu, id, j);
        if (lane == r) out = oi;
    }
    return out;
}

template <int NPL>
__global__ void __launch_bounds__(kWarps * 32)
group_gate_kernel(const Args a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    float* s_P = reinterpret_cast<float*>(smem_raw);                   // [warps][E]; a warp's row holds its selection scores before
    int* s_hist = reinterpret_cast<int*>(s_P + (size_t)kWarps * a.E);
    pdl_wait();
    pdl_trigger();                            // the finalize may launch now (it waits for this kernel's partials)
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) s_hist[e] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int npl = a.npl, e0 = lane * npl;
    float* row = s_P + (size_t)warp * a.E;
    float Pacc[NPL], bias[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        Pacc[i] = 0.f;
        bias[i] = a.bias && i < npl && e0 + i < a.E ? a.bias[e0 + i] : 0.f;
    }
    for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps) {
        float L[NPL], s[NPL], r[NPL];                                // logits, scores, what the experts are ranked by
        bool live[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            live[i] = i < npl && e0 + i < a.E;
            L[i] = -INFINITY;
        }
        const float* src = a.logits + (size_t)t * a.E;
        if (NPL % 4 == 0 && a.vec) {
            if (e0 < a.E) {
#pragma unroll
                for (int i = 0; i < NPL; i += 4) *reinterpret_cast<float4*>(L + i) = *reinterpret_cast<const float4*>(src + e0 + i);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (live[i]) L[i] = src[e0 + i];
        }
        for (int q = 1; q < a.nparts; ++q) {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (live[i]) L[i] += src[q * a.part_stride + e0 + i];
        }
        if (a.logits_out) {
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (live[i]) a.logits_out[(size_t)t * a.E + e0 + i] = L[i];
        }
        // scores
        float total = 0.f;
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                s[i] = live[i] ? 1.f / (1.f + expf(-L[i])) : 0.f;
                total += s[i];
            }
            total = warp_sum(total);
            const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
            for (int i = 0; i < NPL; ++i) Pacc[i] += s[i] * inv;
        } else {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < NPL; ++i) m = fmaxf(m, L[i]);
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                s[i] = L[i] != -INFINITY ? expf(L[i] - m) : 0.f;
                total += s[i];
            }
            total = warp_sum(total);
            const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                s[i] *= inv;
                Pacc[i] += s[i];
            }
        }
        // selection scores; the group's score is of s + bias, the experts' order without a bias that of the logits
        float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const float v = s[i] + bias[i];
            const bool out = !(L[i] > -INFINITY) || !(v == v);
            const float sel = out ? kMasked : v;
            r[i] = a.bias || out ? sel : L[i];
            if (live[i]) {
                t2 = fmaxf(t2, fminf(t1, sel));
                t1 = fmaxf(t1, sel);
                if (!a.lpg) row[e0 + i] = sel;
            }
        }
        bool near = false;                    // scores that 32 bits cannot tell apart
        unsigned kept = 0xffffffffu;          // bit g: group g stays
        if (a.top_groups < a.groups) {
            int g = lane;                     // this lane's group
            if (a.lpg) {
                g = lane / a.lpg;
                const int pos = lane - g * a.lpg, g0 = lane - pos;
                if ((a.lpg & (a.lpg - 1)) == 0) {
                    for (int o = 1; o < a.lpg; o <<= 1) {
                        const float b1 = __shfl_xor_sync(0xffffffffu, t1, o), b2 = __shfl_xor_sync(0xffffffffu, t2, o);
                        t2 = fmaxf(fminf(t1, b1), fmaxf(t2, b2));
                        t1 = fmaxf(t1, b1);
                    }
                } else {
                    const float m1 = t1, m2 = t2;
                    for (int o = 1; o < a.lpg; ++o) {
                        const int from = g0 + (pos + o < a.lpg ? pos + o : pos + o - a.lpg);
                        const float b1 = __shfl_sync(0xffffffffu, m1, from & 31), b2 = __shfl_sync(0xffffffffu, m2, from & 31);
                        t2 = fmaxf(fminf(t1, b1), fmaxf(t2, b2));
                        t1 = fmaxf(t1, b1);
                    }
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
            const float gs = a.best == 2 ? t1 + t2 : t1;
            int rank = 0;
            for (int o = 0; o < a.groups; ++o) {
                const float v = __shfl_sync(0xffffffffu, gs, a.lpg ? o * a.lpg : o);
                rank += v > gs || (v == gs && o < g);
            }
            const bool is = g < a.groups, stays = is && rank < a.top_groups;
            const unsigned last = __reduce_min_sync(0xffffffffu, stays ? key_of(gs) : 0xffffffffu),
                           next = __reduce_max_sync(0xffffffffu, is && !stays ? key_of(gs) : 0u);
            const float x = value_of(last), y = value_of(next);
            // error of a group's score: with a bias 2^-21 for the s (all below 1) and the sum's rounding; without one
            // relative to the score (softmax: the logits' difference is rounded too)
            const float tol = a.bias ? 2e-6f + 2.4e-7f * (fabsf(x) + fabsf(y)) : (a.sigmoid ? 1e-6f : 4e-6f) * (x + y);
            // (two masked groups are equal; the largest of a group without a bias is compared exactly below)
            near = !(x - y > tol) && x > 0.1f * kMasked;
            kept = __ballot_sync(0xffffffffu, stays);
            if (a.lpg) kept = stays ? 0xffffffffu : 0u;                   // this lane's experts are all of one group
        }
        unsigned key[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const bool in = live[i] && (kept == 0xffffffffu || (kept >> ((e0 + i) / a.per) & 1u));
            key[i] = in ? key_of(r[i]) : 0u;
        }
        unsigned lmax = key[0];
        int lslot = 0;
        float ls = s[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i)
            if (key[i] > lmax) { lmax = key[i]; lslot = i; ls = s[i]; }
        // k rounds; with a bias one more, and a look at what is left then, which tell how near the scores are that were left out
        int my_id = 0;
        float my_s = 0.f, sum = 0.f, pv_before = 0.f, m_before = 0.f;
        bool close = false, past = false;     // chosen (or the first left out) close to each other; the first two left out
        // what two neighbours' difference has to pass: the error of s (a sigmoid's exponential and two roundings, of which the exponential's
        // counts with 1 - s; softmax: the exponential, the difference of the logits, the sum) and that of adding the bias
        auto near_by = [&](float x, float sx, float y, float sy) {
            const float err = a.sigmoid ? sx * (1.4e-7f + 2.5e-7f * (1.f - sx)) + sy * (1.4e-7f + 2.5e-7f * (1.f - sy)) : 1e-6f * (sx + sy) + 6e-8f;
            return !(x - y > err + 6.1e-8f * (fabsf(x) + fabsf(y))) && x > 0.1f * kMasked;
        };
        const int rounds = a.k + (a.bias ? 1 : 0);
        for (int j = 0; j < rounds; ++j) {
            const unsigned m = __reduce_max_sync(0xffffffffu, lmax);
            if (m == 0u) break;               // (no expert is left after the k)
            const int owner = __ffs(__ballot_sync(0xffffffffu, lmax == m)) - 1;
            const float pv = __shfl_sync(0xffffffffu, ls, owner), mv = value_of(m);
            const int id = __shfl_sync(0xffffffffu, e0 + lslot, owner);
            if (a.bias && j > 0) close |= near_by(m_before, pv_before, mv, pv);
            pv_before = pv;
            m_before = mv;
            if (lane == owner) {
#pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if (i == lslot) key[i] = 0u;
                lmax = key[0];
                lslot = 0;
                ls = s[0];
#pragma unroll
                for (int i = 1; i < NPL; ++i)
                    if (key[i] > lmax) { lmax = key[i]; lslot = i; ls = s[i]; }
            }
            if (lane == j) {
                my_id = id;
                my_s = pv;
            }
            if (j < a.k) sum += pv;
        }
        if (near || close) {
            int n = a.k;                      // the candidates of a cheap ordering: the chosen and the next, if nothing comes near that
            if (close) {
                const unsigned m = __reduce_max_sync(0xffffffffu, lmax);
                const int owner = __ffs(__ballot_sync(0xffffffffu, lmax == m)) - 1;
                if (m != 0u) past = near_by(m_before, pv_before, value_of(m), __shfl_sync(0xffffffffu, ls, owner));
                n = min(rounds, a.top_groups * a.per);
            }
            if (near || past || !a.sigmoid) {
                my_id = choose_exact(a, L, a.bias, npl);
            } else {
                float my_l = 0.f;
                for (int j = 0; j < n; ++j) {
                    const int id = __shfl_sync(0xffffffffu, my_id, j);
                    float v = 0.f;
#pragma unroll
                    for (int i = 0; i < NPL; ++i)
                        if (e0 + i == id && i < npl) v = L[i];
                    v = __shfl_sync(0xffffffffu, v, id / npl);
                    if (lane == j) my_l = v;
                }
                my_id = order_exact(my_l, a.bias, my_id, n);
            }
            // the chosen experts' scores, from the lanes that hold them
            sum = 0.f;
            for (int j = 0; j < a.k; ++j) {
                const int id = __shfl_sync(0xffffffffu, my_id, j);
                float v = 0.f;
#pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if (e0 + i == id && i < npl) v = s[i];
                v = __shfl_sync(0xffffffffu, v, id / npl);
                if (lane == j) my_s = v;
                sum += v;
            }
        }
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = my_id;
            a.gates[(size_t)t * a.k + lane] = a.renorm ? (sum == 0.f ? 0.f : my_s * a.scale / sum) : my_s * a.scale;
            atomicAdd(&s_hist[my_id], 1);
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NPL; ++i)
        if (i < npl && e0 + i < a.E) row[e0 + i] = Pacc[i];
    __syncthreads();
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
template <int NPL>
__global__ void __launch_bounds__(256)
group_gate_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ d_gates,
                           const float* __restrict__ f, int T, int E, int k, bool sigmoid, bool renorm, float scale, float coef,
                           float* __restrict__ d_logits, unsigned* err) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    float c[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) c[i] = lane + 32 * i < E ? coef * f[lane + 32 * i] : 0.f;
    for (int t = blockIdx.x * nw + warp; t < T; t += gridDim.x * nw) {
        float s[NPL], n[NPL], d[NPL];                                // score, 1 - score, gradient of the score
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = lane + 32 * i < E ? __ldcs(logits + (size_t)t * E + lane + 32 * i) : -INFINITY;
        int id = -1;
        float dg = 0.f;
        if (lane < k) {
            id = ids[(size_t)t * k + lane];
            dg = d_gates[(size_t)t * k + lane];
            if (id < 0 || id >= E) { latch_device_error(err, kDevErrBadIndex, 0x300u); id = -1; }
        }
        float total = 0.f, m = 0.f;
        if (sigmoid) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const float e = expf(-fabsf(s[i])), inv = 1.f / (1.f + e), a = e * inv;
                n[i] = s[i] >= 0.f ? a : inv;
                s[i] = s[i] >= 0.f ? inv : a;
                if (lane + 32 * i >= E) s[i] = 0.f;
            }
        } else {
            m = s[0];
#pragma unroll
            for (int i = 1; i < NPL; ++i) m = fmaxf(m, s[i]);
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                s[i] = s[i] != -INFINITY ? expf(s[i] - m) : 0.f;
                n[i] = 0.f;
            }
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) total += s[i];
        total = warp_sum(total);
        const float tinv = total == 0.f ? 0.f : 1.f / total;
        if (!sigmoid) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) s[i] *= tinv;
        }
        float ds = scale * dg;
        if (renorm) {
            float mine = 0.f;                                        // lane j: the score of choice j
            for (int j = 0; j < k; ++j) {
                const int e = __shfl_sync(0xffffffffu, id, j);
                float v = 0.f;
#pragma unroll
                for (int i = 0; i < NPL; ++i)
                    if (lane + 32 * i == e) v = s[i];
                v = __shfl_sync(0xffffffffu, v, e & 31);
                if (lane == j && e >= 0) mine = v;
            }
            const float S = warp_sum(mine), w = warp_sum(mine * dg);
            const float inv = S == 0.f ? 0.f : 1.f / S;
            ds = scale * (dg - w * inv) * inv;
        }
        float cq = 0.f;
        if (sigmoid) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) cq += c[i] * s[i];
            cq = warp_sum(cq) * tinv;
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) d[i] = sigmoid ? (c[i] - cq) * tinv : c[i];
        for (int j = 0; j < k; ++j) {
            const int e = __shfl_sync(0xffffffffu, id, j);
            const float v = __shfl_sync(0xffffffffu, ds, j);
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (lane + 32 * i == e) d[i] += v;
        }
        float dot = 0.f;
        if (!sigmoid) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) dot += d[i] * s[i];
            dot = warp_sum(dot);
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (lane + 32 * i < E)
                __stcs(d_logits + (size_t)t * E + lane + 32 * i, sigmoid ? d[i] * s[i] * n[i] : s[i] * (d[i] - dot));
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

int check_spec(const char* fn, int T, int E, int k, int groups, int top_groups, int score, int best, float scale) {
    MOE_REQUIRE(score == MOE_SCORE_SIGMOID || score == MOE_SCORE_SOFTMAX, MOE_ERR_UNSUPPORTED, "%s: score %d", fn, score);
    MOE_REQUIRE(T >= 0 && E >= 1 && E <= kMaxE && groups >= 1 && groups <= kMaxGroups && E % groups == 0, MOE_ERR_INVALID_ARG,
                "%s: T=%d E=%d groups=%d (need E <= 1024, groups <= 32 of equal size)", fn, T, E, groups);
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
        // experts to a lane: as few as hold E, and a divisor of the group's size where one fits
        const int least = cdiv(g.E, 32);
        a.npl = least;
        a.lpg = 0;
        for (int n = least; n <= std::min(a.per, 32); ++n)
            if (a.per % n == 0 && (n <= 8 || n < 2 * least)) { a.npl = n; a.lpg = a.per / n; break; }
        const size_t smem = (size_t)kWarps * g.E * sizeof(float) + (size_t)g.E * sizeof(int);
        auto launch = [&](auto kernel, int n) {
            a.vec = a.npl == n && n % 4 == 0 && g.E % 4 == 0 && aligned16(g.logits) && g.E % n == 0;
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            int per_sm = 0;
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kWarps * 32, smem) != cudaSuccess || per_sm < 1) per_sm = 1;
            G = std::min(grid_of(g.T), per_sm * num_sms());
            return launch_pdl(kernel, dim3(G), dim3(kWarps * 32), smem, s, a);
        };
        const cudaError_t e = a.npl <= 1 ? launch(group_gate_kernel<1>, 1) : a.npl <= 2 ? launch(group_gate_kernel<2>, 2)
                            : a.npl <= 4 ? launch(group_gate_kernel<4>, 4) : a.npl <= 8 ? launch(group_gate_kernel<8>, 8)
                            : a.npl <= 16 ? launch(group_gate_kernel<16>, 16) : launch(group_gate_kernel<32>, 32);
        if (int rc = check_launch(e, "group_gate_kernel")) return rc;
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
    if (T < 0 || E <= 0) return 0;
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
    const int G = std::min(cdiv(T, 8), 8 * num_sms());
    cudaStream_t s = static_cast<cudaStream_t>(stream);
#define MOE_GROUP_BWD(N)                                                                                              \
    group_gate_backward_kernel<N><<<G, 256, 0, s>>>(logits, topk_ids, d_gates, f, T, E, k, score == MOE_SCORE_SIGMOID, renorm != 0, \
                                                    scale, coef, d_logits, err)
    const int n = cdiv(E, 32);
    if (n <= 1) MOE_GROUP_BWD(1);
    else if (n <= 2) MOE_GROUP_BWD(2);
    else if (n <= 4) MOE_GROUP_BWD(4);
    else if (n <= 8) MOE_GROUP_BWD(8);
    else if (n <= 16) MOE_GROUP_BWD(16);
    else MOE_GROUP_BWD(32);
#undef MOE_GROUP_BWD
    return check_launch("group_gate_backward_kernel");
}
