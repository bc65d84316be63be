// Residual addition, root-mean-square norm, rotation and quantization in one
// pass over the rows (sm_103a): h32_add_rms_norm_quantize.
//
// What runs between two products of a decoder layer ("509 tokens a second of
// prompt: the Hadamard route ships", section "The rotation": every projection's
// input is rotated and quantized).  Per row of K values:
//   h = x + residual            (fp32, rounded to the residual's type)
//   S = sum h^2                 (fp32, in the fixed order below)
//   r = 1 / sqrt(S / K + eps)   (each step rounded to fp32)
//   n = (h r) w                 (two fp32 roundings)
// then n's 32-blocks are rotated and rounded to codes exactly as by the
// activation quantizers.  The order of S: fma over a block's 32 elements from
// +0, then groups of 32 blocks by the xor tree of strides 1, 2, 4, 8, 16 (absent
// blocks are 0), then the groups in order: the same bits for every launch shape.
//
// Bound: HBM (bf16 in, bf16 residual in and out, one code byte: 7.1 bytes an
// element against about 25 instructions).  One thread owns one 32-block, as in
// the activation quantizers, so the block stays in registers from the load to
// the codes: the row is read once, and the only exchange is the sum.
#include "h32_common.cuh"
#include "h32_quant_block.cuh"

#include <cuda_bf16.h>

namespace h32 {
namespace {

constexpr int kMaxRowThreads = 1024;   // 32-blocks a row (K <= 32768)
// rows of up to 768 blocks run without register spills (80 a thread); longer
// ones in an instance of their own (64 a thread)
constexpr int kRowThreads = 768;

struct NormArgs {
    const void *x, *res, *w;
    void *res_out, *norm_out;
    void *xq;
    float *xd;
    int64_t ldx, ldr, ldro, ldn, ldxd;
    int64_t M;
    int32_t K, nb;
    int32_t lanes;   // threads a row where a warp holds several rows (power of two <= 32)
    float eps;
    uint8_t x_bf16, res_bf16, w_bf16, n_bf16;
};

// Plain loads: x and the residual may be the very rows this kernel writes.
__device__ __forceinline__ void load32(const void *p, int64_t at, bool bf16, float (&v)[32]) {
    if (bf16) {
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 u = q[c];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[8 * c + 2 * i] = __uint_as_float(w[i] << 16);
                v[8 * c + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
        }
    } else {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float4 f = q[c];
            v[4 * c] = f.x;
            v[4 * c + 1] = f.y;
            v[4 * c + 2] = f.z;
            v[4 * c + 3] = f.w;
        }
    }
}

// two fp32 values rounded to bf16 (nearest even), the first in the low half
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// stores 32 values; a bf16 store also rounds v itself, so that what follows
// uses the values as stored
__device__ __forceinline__ void store32(void *p, int64_t at, bool bf16, const float (&v)[32]) {
    if (bf16) {
        uint4 *q = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            q[c] = make_uint4(bf16_pair(v[8 * c], v[8 * c + 1]), bf16_pair(v[8 * c + 2], v[8 * c + 3]),
                              bf16_pair(v[8 * c + 4], v[8 * c + 5]),
                              bf16_pair(v[8 * c + 6], v[8 * c + 7]));
    } else {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + at);
#pragma unroll
        for (int c = 0; c < 8; ++c)
            q[c] = make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
    }
}

// The row's sum of squares in the order above; every thread of the row gets it.
// s_part: one float per warp of the block (rows of more than 32 blocks).
__device__ __forceinline__ float row_sum_sq(const float (&v)[32], const NormArgs &a,
                                            float *s_part) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s = __fmaf_rn(v[i], v[i], s);
    for (int o = 1; o < a.lanes; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    if (a.nb <= 32) return s;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = s;
    __syncthreads();
    s = s_part[0];
    for (int w = 1; w < warps; ++w) s = __fadd_rn(s, s_part[w]);
    return s;
}

// kForm: an h32_act_form, or -1 (norm_out alone)
template <int kForm, int kRot, int kThreads>
__global__ void __launch_bounds__(kThreads) norm_quant_kernel(const NormArgs a) {
    __shared__ float s_part[2][32];
    pdl_wait();
    pdl_trigger();
    // rows of up to 32 blocks: 256 / lanes rows a block; longer rows: one a block
    const int64_t row = a.nb <= 32
                            ? static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.lanes) + threadIdx.x / a.lanes
                            : blockIdx.x;
    const int b = a.nb <= 32 ? threadIdx.x & (a.lanes - 1) : threadIdx.x;
    const bool in = row < a.M && b < a.nb;
    const unsigned mask = __ballot_sync(0xFFFFFFFFu, in);
    float v[32];
    if (in) {
        load32(a.x, row * a.ldx + 32 * b, a.x_bf16, v);
        if (a.res) {
            float u[32];
            load32(a.res, row * a.ldr + 32 * b, a.res_bf16, u);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __fadd_rn(v[i], u[i]);
            if (a.res_bf16) {
                // the norm reads the residual as it is stored
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
            }
            if (a.res_out) store32(a.res_out, row * a.ldro + 32 * b, a.res_bf16, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.0f;
    }
    const float kf = static_cast<float>(a.K);
    float s = row_sum_sq(v, a, s_part[0]);
    float r;
    // (a warp that holds several rows takes both ways where one of them overflows)
    bool over = !(s < INFINITY);
    r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(s, kf), a.eps)));
    if (a.nb <= 32 ? __any_sync(0xFFFFFFFFu, over) : over) {
        // a sum of squares above fp32's range: the row times 2^-80 (exact but for
        // values too small to matter), whose norm is the same; eps is nothing there
        if (over) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __fmul_rn(v[i], 0x1p-80f);
        }
        const float s2 = row_sum_sq(v, a, s_part[1]);
        if (over) r = __frcp_rn(__fsqrt_rn(__fdiv_rn(s2, kf)));
    }
    if (!in) return;
    {
        float w[32];
        load32(a.w, 32 * b, a.w_bf16, w);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __fmul_rn(__fmul_rn(v[i], r), w[i]);
    }
    if (a.norm_out) store32(a.norm_out, row * a.ldn + 32 * b, a.n_bf16, v);
    if constexpr (kForm >= 0) {
        rotate_block<kRot>(v, b, mask);
        const int64_t K = a.K;
        uint8_t *xq = static_cast<uint8_t *>(a.xq);
        float d;
        if constexpr (kForm == H32_ACT_Q4) {
            uint32_t bits[32], w[4];
            d = quant_block_bits<4>(v, bits);
            pack_q4(bits, w);
            *reinterpret_cast<uint4 *>(xq + row * (K / 2) + 16 * b) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (kForm == H32_ACT_Q8) {
            uint32_t bits[32], w[8];
            d = quant_block_bits<8>(v, bits);
            pack_q8(bits, w);
            uint4 *dst = reinterpret_cast<uint4 *>(xq + row * K + 32 * b);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else if constexpr (kForm == H32_ACT_Q8_TC) {
            uint32_t bits[32], wh[8], wl[8];
            d = quant_block_bits<8>(v, bits);
            pack_q8_tc(bits, wh, wl);
            uint4 *dst = reinterpret_cast<uint4 *>(xq + row * 2 * K + 64 * b);
            dst[0] = make_uint4(wh[0], wh[1], wh[2], wh[3]);
            dst[1] = make_uint4(wh[4], wh[5], wh[6], wh[7]);
            dst[2] = make_uint4(wl[0], wl[1], wl[2], wl[3]);
            dst[3] = make_uint4(wl[4], wl[5], wl[6], wl[7]);
        } else {
            uint32_t w[8];
            d = quant_block_tc4<kForm == H32_ACT_Q4_TC_E5M2>(v, w);
            uint4 *dst = reinterpret_cast<uint4 *>(xq + row * K + 32 * b);
            dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
            dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        if constexpr (kForm == H32_ACT_Q4 || kForm == H32_ACT_Q8)
            a.xd[row * a.nb + b] = d;
        else
            a.xd[static_cast<int64_t>(b) * a.ldxd + row] = d;
    }
}

template <int kForm, int kRot>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t s) {
    if (a.nb <= 32) {
        const int rows = 256 / a.lanes;
        return launch_pdl(norm_quant_kernel<kForm, kRot, kRowThreads>,
                          dim3(static_cast<unsigned>((a.M + rows - 1) / rows)), dim3(256), 0, s, a);
    }
    const dim3 grid(static_cast<unsigned>(a.M)), block((a.nb + 31) / 32 * 32);
    if (a.nb <= kRowThreads) return launch_pdl(norm_quant_kernel<kForm, kRot, kRowThreads>, grid, block, 0, s, a);
    return launch_pdl(norm_quant_kernel<kForm, kRot, kMaxRowThreads>, grid, block, 0, s, a);
}

template <int kForm>
cudaError_t launch_norm_rot(const NormArgs &a, int rot, cudaStream_t s) {
    switch (rot) {
        case 0: return launch_norm<kForm, 0>(a, s);
        case 32: return launch_norm<kForm, 32>(a, s);
        case 64: return launch_norm<kForm, 64>(a, s);
        default: return launch_norm<kForm, 128>(a, s);
    }
}

inline bool dtype_ok(h32_in_dtype dt) { return dt == H32_IN_F32 || dt == H32_IN_BF16; }
inline int64_t bytes_of(h32_in_dtype dt) { return dt == H32_IN_BF16 ? 2 : 4; }

}  // namespace
}  // namespace h32

extern "C" h32_status h32_add_rms_norm_quantize(
    const void *x, h32_in_dtype x_dt, int64_t ldx, const void *residual, h32_in_dtype res_dt,
    int64_t ldr, const void *w, h32_in_dtype w_dt, float eps, int64_t M, int64_t K,
    void *residual_out, int64_t ldro, void *norm_out, h32_in_dtype norm_dt, int64_t ldn,
    int32_t form, int rotate, void *xq, float *xd, int64_t ldxd, void *stream) {
    using namespace h32;
    const int rot = rot_points(rotate);
    if (M < 0 || K <= 0 || (K % 32) != 0 || K > 32 * kMaxRowThreads || ldx < K)
        return H32_ERR_INVALID_ARG;
    if (rot < 0 || (rot > 0 && K % rot != 0)) return H32_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !(eps < INFINITY)) return H32_ERR_INVALID_ARG;
    if (!dtype_ok(x_dt) || !dtype_ok(w_dt) || (residual && (!dtype_ok(res_dt) || ldr < K)) ||
        (residual_out && (!residual || ldro < K)) || (norm_out && (!dtype_ok(norm_dt) || ldn < K)))
        return H32_ERR_INVALID_ARG;
    const bool quant = xq || xd;
    const bool tc = form == H32_ACT_Q4_TC || form == H32_ACT_Q8_TC || form == H32_ACT_Q4_TC_E5M2;
    if (quant && (!xq || !xd || (!tc && form != H32_ACT_Q4 && form != H32_ACT_Q8) ||
                  (tc && (ldxd < M || (ldxd % 4) != 0))))
        return H32_ERR_INVALID_ARG;
    if (M == 0) return H32_OK;
    if (!x || !w || (!quant && !norm_out) || M > 0x7FFFFFFFll) return H32_ERR_INVALID_ARG;
    // an output may be an input element for element, not in another type or pitch
    if ((residual_out == x && (x_dt != res_dt || ldx != ldro)) ||
        (residual_out && residual_out == residual && ldro != ldr) ||
        (norm_out && (norm_out == residual_out ||
                      (norm_out == x && (x_dt != norm_dt || ldx != ldn)) ||
                      (norm_out == residual && (res_dt != norm_dt || ldr != ldn)))))
        return H32_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(w) || (ldx * bytes_of(x_dt)) % 16 != 0 ||
        (residual && (!aligned16(residual) || (ldr * bytes_of(res_dt)) % 16 != 0)) ||
        (residual_out && (!aligned16(residual_out) || (ldro * bytes_of(res_dt)) % 16 != 0)) ||
        (norm_out && (!aligned16(norm_out) || (ldn * bytes_of(norm_dt)) % 16 != 0)) ||
        (quant && (!aligned16(xq) || !aligned16(xd))))
        return H32_ERR_ALIGNMENT;
    H32_TRY(check_device(nullptr));
    NormArgs a{};
    a.x = x;
    a.res = residual;
    a.w = w;
    a.res_out = residual_out;
    a.norm_out = norm_out;
    a.xq = xq;
    a.xd = xd;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldro = ldro;
    a.ldn = ldn;
    a.ldxd = ldxd;
    a.M = M;
    a.K = static_cast<int32_t>(K);
    a.nb = static_cast<int32_t>(K / 32);
    a.lanes = 1;
    while (a.lanes < a.nb && a.lanes < 32) a.lanes *= 2;
    a.eps = eps;
    a.x_bf16 = x_dt == H32_IN_BF16;
    a.res_bf16 = res_dt == H32_IN_BF16;
    a.w_bf16 = w_dt == H32_IN_BF16;
    a.n_bf16 = norm_dt == H32_IN_BF16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (!quant) {
        e = launch_norm<-1, 0>(a, s);
    } else {
        switch (form) {
            case H32_ACT_Q4: e = launch_norm_rot<H32_ACT_Q4>(a, rot, s); break;
            case H32_ACT_Q8: e = launch_norm_rot<H32_ACT_Q8>(a, rot, s); break;
            case H32_ACT_Q4_TC: e = launch_norm_rot<H32_ACT_Q4_TC>(a, rot, s); break;
            case H32_ACT_Q8_TC: e = launch_norm_rot<H32_ACT_Q8_TC>(a, rot, s); break;
            default: e = launch_norm_rot<H32_ACT_Q4_TC_E5M2>(a, rot, s); break;
        }
    }
    return launch_status(e != cudaSuccess ? e : cudaGetLastError());
}
