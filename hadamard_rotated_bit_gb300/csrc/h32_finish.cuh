// What a product does to its output before storing it (sm_103a), shared by the
// tensor-core GEMM and the few-token product: bias, activation, residual, one
// rounding.  All in fp32:
//   v = act(z + bias);  y = round(v + residual)
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "../../include/h32.h"

namespace h32 {

struct EpiArgs {
    const float *bias;      // [rows of the weights] or null
    const void *res;        // [M][ldr] or null
    void *y;                // [M][ldy]
    int64_t ldr, ldy;
    int32_t act;            // an h32_epi_act
    uint8_t res_bf16, y_bf16;
};

// z / (1 + exp(-t)): the sigmoid of t times z; exp(-t) = inf gives the limit 0
__device__ __forceinline__ float sigmoid_times(float t, float z) {
    return __fdiv_rn(z, __fadd_rn(1.0f, expf(-t)));
}

__device__ __forceinline__ float swiglu(float gate, float up) {
    return __fmul_rn(sigmoid_times(gate, gate), up);
}

// act(z) of the activations that take one value.  The tanh form of GELU is
// z sigmoid(2 u), u = sqrt(2/pi) (z + 0.044715 z^3), and the erf form
// z erfc(-z / sqrt(2)) / 2: both without the cancellation of 1 + tanh and 1 + erf
// at negative z.
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case H32_EPI_RELU: return z < 0.0f ? 0.0f : z;   // NaN stays
        case H32_EPI_SILU: return sigmoid_times(z, z);
        case H32_EPI_GELU_TANH: {
            const float c = 1.5957691216057308f;   // 2 sqrt(2 / pi)
            return sigmoid_times(c * __fmaf_rn(0.044715f * z * z, z, z), z);
        }
        case H32_EPI_GELU_ERF: return 0.5f * z * erfcf(-0.70710678118654752f * z);
        default: return z;
    }
}

__device__ __forceinline__ float load_value(const void *p, int64_t i, bool bf16) {
    // plain loads: y may be the residual itself
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i])
                : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_value(void *p, int64_t i, bool bf16, float v) {
    if (bf16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<float *>(p)[i] = v;
}

// n token columns m0 + q of output feature j, those with lo <= q < hi: residual and
// store (the loads of all columns in flight together)
template <int n>
__device__ __forceinline__ void finish_columns(const EpiArgs &f, const float *v, int64_t m0, int lo,
                                               int hi, int j) {
    float r[n];
    if (f.res) {
#pragma unroll
        for (int q = 0; q < n; ++q)
            r[q] = (q >= lo && q < hi) ? load_value(f.res, (m0 + q) * f.ldr + j, f.res_bf16) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < n; ++q)
        if (q >= lo && q < hi)
            store_value(f.y, (m0 + q) * f.ldy + j, f.y_bf16, f.res ? __fadd_rn(v[q], r[q]) : v[q]);
}

}  // namespace h32
