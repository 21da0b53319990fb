// Router: what other routing kernels share with it.
#pragma once
#include "common.cuh"

namespace moe {

// Blocks of the finalize (the length of its term_part).
int finalize_grid(int T, int E);
// Counts, f, P and aux from the partial sums [G][E] of G gating blocks, block 0 of which zeroed `ticket`; a programmatic
// dependent of the kernel that wrote them. T == 0: no partial sums.
int launch_router_finalize(const float* partial_P, const int32_t* partial_C, int G, int T, int E, int k, float alpha,
                           int32_t* counts, float* f, float* P, float* aux, float* term_part, unsigned* ticket, cudaStream_t s);

}  // namespace moe
