// The choice of experts from logits (internal; ep_select.cu, ep_router.cu).
#pragma once

#include <cuda_runtime.h>

#include "ep.h"

namespace ep {

constexpr int kMaxGroups = 64;

// How experts are chosen, and from what.
struct Choice {
    const void *logits;   // [T,E] fp32 (dtype 0) or bf16 (1); or sums of `slices` parts [slices][T][E] fp32 (0)
    int dtype, slices;
    const float *bias;
    int T, E, K;
    int sigmoid, groups, kept, top2, renormalize;
    float scale;
    int64_t *idx;
    float *weights, *sums;   // sums: [T,E] receives the logits, or null
};

// Host errors of the arguments that every entry point of a choice shares.
int choice_status(int E, int K, int scoring, int num_groups, int topk_groups, int group_score);

int launch_choice(const Choice &c, cudaStream_t stream);

}  // namespace ep
