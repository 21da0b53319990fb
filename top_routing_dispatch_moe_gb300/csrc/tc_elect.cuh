// Operations that a whole warp issues through one elected lane, and waits with the same answer in every lane: the producer
// and MMA warps of the quantised grouped products.
#pragma once
#include "tc_ptx.cuh"

namespace moe {
namespace tc {

// The value of lane 0, known to the compiler to be the same in the warp: branches on it and what depends on it stay uniform.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

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

// ---- a pair of CTAs ----
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

}  // namespace tc
}  // namespace moe
