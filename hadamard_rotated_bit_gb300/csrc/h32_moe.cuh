// What the routers share (sm_103a): their limits, and the grouping of the
// (token, choice) rows by expert.
#pragma once

#include "h32_common.cuh"

namespace h32 {

constexpr int kMaxE = 1024;   // experts a router call handles
constexpr int kMaxK = 32;     // choices per token (one lane each)

// topk_id [T][k] -> expert_off [E+1], row_idx [T k], row_of [T][k] (h32_moe.cu)
cudaError_t launch_route_group(const int32_t *topk_id, int T, int E, int k, int32_t *expert_off,
                               int32_t *row_idx, int32_t *row_of, cudaStream_t s);

}  // namespace h32
