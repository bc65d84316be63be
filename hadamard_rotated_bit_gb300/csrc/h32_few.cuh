// The product of a few tokens (h32_few.cu), called by the tensor-core GEMM's entry
// points once their arguments are checked.
#pragma once

#include "h32_common.cuh"
#include "h32_finish.cuh"

namespace h32 {

constexpr int kFewTokens = 16;   // tokens the kernel takes

// z of q4_0_x_q4_gemm_tc (xbits 4) or q4_0_x_q8_gemm_tc (8) for M <= kFewTokens
// tokens, finished as `fin` says
h32_status launch_few(int xbits, const uint8_t *wp, const float *wsc, int64_t ldws,
                      const uint8_t *xw, const float *xdt, int64_t ldxd, int64_t M, int64_t N,
                      int64_t K, const EpiArgs &fin, int sms, cudaStream_t s);
h32_status few_read_and_clear_status(cudaStream_t s);

}  // namespace h32
