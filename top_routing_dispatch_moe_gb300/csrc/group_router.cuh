// Routing by groups of experts: the gating step on logits.
#pragma once
#include "common.cuh"

namespace moe {

struct GroupGate {
    const float* logits;          // [T][E], the sum of nparts parts, part_stride elements apart
    int nparts;
    size_t part_stride;
    float* logits_out;            // the summed logits, or null
    const float* bias;            // [E] or null
    int T, E, k, groups, top_groups, score, best;
    bool renorm;
    float scale, alpha;
    int32_t* ids;
    float* gates;
    int32_t* counts;
    float *f, *P, *aux;
};
int check_group_gate(const char* fn, const GroupGate& g);
size_t group_gate_ws_bytes(int T, int E);
int launch_group_gate(const GroupGate& g, void* ws, cudaStream_t s);

}  // namespace moe
