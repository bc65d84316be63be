// Residual addition, root-mean-square norm, rotation and quantization in one
// pass over the rows (sm_103a): h32_add_rms_norm_quantize.
//
// What runs between two products of a decoder layer ("509 tokens a second of
// prompt: the Hadamard route ships", section "The rotation": every projection's
// input is rotated and quantized).  Per row of K values:
//   h = x + residual              (fp32, rounded to the residual's type)
//   S = sum h^2                   (fp32, in the fixed order below)
//   r = 1 / sqrt(S fl(1/K) + eps) (product, sum and reciprocal root each rounded)
//   n = (h r) w                   (two fp32 roundings)
// then n's 32-blocks are rotated and rounded to codes exactly as by the
// activation quantizers.  The order of S: over 16 consecutive values two fma
// chains from +0, the even and the odd places, added; 32 such sums by the xor tree
// of strides 1 .. 16 (absent ones 0); 32 of those the same way; then what is left
// in order.  The same bits for every launch shape.
//
// Bound: HBM (bf16 in, bf16 residual in and out, one code byte: 7.1 bytes an
// element).  Two adjacent lanes hold one 32-block, 16 values each: four of the
// five butterfly stages stay in the lane, the fifth is one exchange, and a warp
// touches 32-byte runs.  (One lane a block, the activation quantizers' layout,
// touches 64-byte runs, 128 for fp32: with the norm's four arrays the L1's
// wavefronts bound it, 75% busy at half the copy rate, 179 us for 16384 x 5120.)
// Blocks of threads walk the rows, so the weights stay in registers; products,
// sums and butterflies work on packed pairs.
#include "h32_common.cuh"
#include "h32_epilogue.cuh"
#include "h32_quant_block.cuh"

#include <cuda_bf16.h>

namespace h32 {
namespace {

constexpr int kMaxRow = 32768;      // K: 1024 threads of two 16-value pieces
constexpr int kOnePiece = 8192;     // up to here a thread holds one piece

struct NormArgs {
    const void *x, *res, *w;
    void *res_out, *norm_out;
    void *xq;
    float *xd;
    int64_t ldx, ldr, ldro, ldn, ldxd;
    int64_t M;
    int32_t K;
    int32_t lanes;   // threads a row where a warp holds several rows (power of two <= 32)
    float eps, inv_k;
    uint8_t x_bf16, res_bf16, w_bf16, n_bf16;
};

__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t pair_f(float lo, float hi) {
    return pair_of(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float lo_f(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float hi_f(uint64_t p) {
    return __uint_as_float(static_cast<uint32_t>(p >> 32));
}

// two fp32 values rounded to bf16 (nearest even), the first in the low half
__device__ __forceinline__ uint32_t bf16_pair(uint64_t p) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo_f(p), hi_f(p));
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ uint64_t widen(uint32_t b) { return pair_of(b << 16, b & 0xFFFF0000u); }

// 16 values from element `at`.  Plain loads: x and the residual may be the very
// rows this kernel writes.
__device__ __forceinline__ void load16(const void *p, int64_t at, bool bf16, uint64_t (&v)[8]) {
    if (bf16) {
        const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + at);
        const uint4 u[2] = {q[0], q[1]};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            v[4 * c] = widen(u[c].x);
            v[4 * c + 1] = widen(u[c].y);
            v[4 * c + 2] = widen(u[c].z);
            v[4 * c + 3] = widen(u[c].w);
        }
    } else {
        const ulonglong2 *q = reinterpret_cast<const ulonglong2 *>(static_cast<const float *>(p) + at);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const ulonglong2 u = q[c];
            v[2 * c] = u.x;
            v[2 * c + 1] = u.y;
        }
    }
}

// 16 values to element `at`, rounded to bf16 or as they are
__device__ __forceinline__ void store16(void *p, int64_t at, bool bf16, const uint64_t (&v)[8]) {
    if (bf16) {
        uint4 *q = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + at);
        q[0] = make_uint4(bf16_pair(v[0]), bf16_pair(v[1]), bf16_pair(v[2]), bf16_pair(v[3]));
        q[1] = make_uint4(bf16_pair(v[4]), bf16_pair(v[5]), bf16_pair(v[6]), bf16_pair(v[7]));
    } else {
        ulonglong2 *q = reinterpret_cast<ulonglong2 *>(static_cast<float *>(p) + at);
#pragma unroll
        for (int c = 0; c < 4; ++c) q[c] = make_ulonglong2(v[2 * c], v[2 * c + 1]);
    }
}

// the piece's sum of squares: the even and the odd places' chains, added
__device__ __forceinline__ float piece_sum(const uint64_t (&v)[8]) {
    uint64_t s = 0ull;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fma_f32x2(v[i], v[i], s);
    return __fadd_rn(lo_f(s), hi_f(s));
}

// The row's sum of squares in the order above; every thread of the row gets it.
// s_part: 64 floats.  kOne: the row is one piece a thread within one warp.
template <int kPieces>
__device__ __forceinline__ float row_sum(const uint64_t (&v)[kPieces][8], const NormArgs &a,
                                         float *s_part) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        float s = piece_sum(v[i]);
        for (int o = 1; o < a.lanes; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
        if (kPieces == 1 && a.K <= 512) return s;
        if (lane == 0) s_part[(threadIdx.x >> 5) + i * warps] = s;
    }
    __syncthreads();
    const int groups = warps * kPieces;
    float s = lane < groups ? s_part[lane] : 0.0f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    if (kPieces > 1 && groups > 32) {
        float t = lane + 32 < groups ? s_part[lane + 32] : 0.0f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) t = __fadd_rn(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
        s = __fadd_rn(s, t);
    }
    return s;
}

// The rotation of a block held by an even lane (elements 0..15) and the odd lane
// after it (16..31); larger rotations pair blocks of adjacent lane pairs.  Stage
// by stage the sums and differences of the activation quantizers' butterfly.
template <int kRot>
__device__ __forceinline__ void rotate_piece(uint64_t (&v)[8], unsigned mask) {
    if constexpr (kRot > 0) {
        const uint64_t minus = pair_f(-1.0f, -1.0f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = lo_f(v[i]), c = hi_f(v[i]);
            v[i] = pair_f(__fadd_rn(a, c), __fsub_rn(a, c));
        }
#pragma unroll
        for (int h = 1; h < 8; h <<= 1) {   // strides 2, 4, 8
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if ((i & h) == 0) {
                    const uint64_t a = v[i], c = v[i + h];
                    v[i] = add_f32x2(a, c);
                    v[i + h] = fma_f32x2(c, minus, a);
                }
            }
        }
#pragma unroll
        for (int hb = 1; hb <= kRot / 32; hb <<= 1) {   // strides 16, 32, 64
            const float sign = (threadIdx.x & hb) ? -1.0f : 1.0f;
            const uint64_t sg = pair_f(sign, sign);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float clo = __shfl_xor_sync(mask, lo_f(v[i]), hb);
                const float chi = __shfl_xor_sync(mask, hi_f(v[i]), hb);
                v[i] = fma_f32x2(v[i], sg, pair_f(clo, chi));   // lower: v + c, upper: c - v
            }
        }
        const float k = kRot == 32 ? kInvSqrt32 : kRot == 64 ? 0.125f : kInvSqrt128;
        const uint64_t sc = pair_f(k, k);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = mul_f32x2(v[i], sc);
    }
}

// Codes and scale of the lane's half of block `unit / 2` of row `row`.
template <int kForm>
__device__ __forceinline__ void quantize_piece(const NormArgs &a, int64_t row, int unit,
                                               const uint64_t (&p)[8], unsigned mask) {
    constexpr int kBits = (kForm == H32_ACT_Q8 || kForm == H32_ACT_Q8_TC) ? 8 : 4;
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = lo_f(p[i]);
        v[2 * i + 1] = hi_f(p[i]);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(v[i]));
    amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 1));
    uint32_t bits[16];
    const float d = quant_bits<kBits>(v, amax, bits);
    const int odd = unit & 1, b = unit >> 1;
    const int64_t K = a.K;
    uint8_t *xq = static_cast<uint8_t *>(a.xq);
    if constexpr (kForm == H32_ACT_Q4_TC || kForm == H32_ACT_Q4_TC_E5M2) {
        // the codes as integer-valued floats, converted exactly by the hardware
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = __fsub_rn(__uint_as_float(bits[4 * k + i]), kRoundMagic);
            w[k] = kForm == H32_ACT_Q4_TC ? e4m3x4_of_ints(c[0], c[1], c[2], c[3])
                                          : e5m2x4_of_ints_x512(c[0], c[1], c[2], c[3]);
        }
        *reinterpret_cast<uint4 *>(xq + row * K + 16 * unit) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = pack_low_bytes(bits[4 * k], bits[4 * k + 1], bits[4 * k + 2], bits[4 * k + 3]);
        if constexpr (kForm == H32_ACT_Q8) {
            *reinterpret_cast<uint4 *>(xq + row * K + 16 * unit) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (kForm == H32_ACT_Q8_TC) {
            uint32_t wh[4], wl[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) tc_bytes_q8(w[k], wh[k], wl[k]);
            uint4 *dst = reinterpret_cast<uint4 *>(xq + row * 2 * K + 64 * b + 16 * odd);
            dst[0] = make_uint4(wh[0], wh[1], wh[2], wh[3]);
            dst[2] = make_uint4(wl[0], wl[1], wl[2], wl[3]);
        } else {
            // byte j = element j (low) | element j + 16 (high): the even lane makes
            // bytes 0..7, the odd lane 8..15
            const uint32_t r0 = __shfl_xor_sync(mask, odd ? w[0] : w[2], 1);
            const uint32_t r1 = __shfl_xor_sync(mask, odd ? w[1] : w[3], 1);
            const uint32_t lo0 = odd ? r0 : w[0], lo1 = odd ? r1 : w[1];
            const uint32_t hi0 = odd ? w[2] : r0, hi1 = odd ? w[3] : r1;
            *reinterpret_cast<uint2 *>(xq + row * (K / 2) + 8 * unit) =
                make_uint2((lo0 & 0x0F0F0F0Fu) | ((hi0 << 4) & 0xF0F0F0F0u),
                           (lo1 & 0x0F0F0F0Fu) | ((hi1 << 4) & 0xF0F0F0F0u));
        }
    }
    if (!odd) {
        if constexpr (kForm == H32_ACT_Q4 || kForm == H32_ACT_Q8)
            a.xd[row * (K / 32) + b] = d;
        else
            a.xd[b * a.ldxd + row] = d;
    }
}

// kForm: an h32_act_form, or -1 (norm_out alone).  A thread holds kPieces pieces
// of 16 values of a row, blockDim.x * 16 values apart.  With one piece a block
// walks rows (its weights stay in registers); with two it takes one row.
template <int kForm, int kRot, int kPieces, int kThreads>
__global__ void __launch_bounds__(kThreads, kPieces == 1 ? 2 : 1) norm_quant_kernel(const NormArgs a) {
    __shared__ float s_part[2][2][64];
    pdl_wait();
    pdl_trigger();
    // rows of at most 512 values: several in a warp
    const bool shared_warp = kPieces == 1 && a.K <= 512;
    const int rows = shared_warp ? blockDim.x / a.lanes : 1;
    const int unit0 = shared_warp ? threadIdx.x & (a.lanes - 1) : threadIdx.x;
    const int units = a.K / 16;
    uint64_t w[kPieces][8];
    if constexpr (kPieces == 1)
        if (unit0 < units) load16(a.w, 16 * unit0, a.w_bf16, w[0]);
    int turn = 0;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows; row0 < a.M;
         row0 += static_cast<int64_t>(gridDim.x) * rows, turn ^= 1) {
        const int64_t row = row0 + (shared_warp ? threadIdx.x / a.lanes : 0);
        uint64_t v[kPieces][8];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int unit = unit0 + i * blockDim.x;
            if (row < a.M && unit < units) {
                load16(a.x, row * a.ldx + 16 * unit, a.x_bf16, v[i]);
                if (a.res) {
                    uint64_t u[8];
                    load16(a.res, row * a.ldr + 16 * unit, a.res_bf16, u);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] = add_f32x2(v[i][j], u[j]);
                    if (a.res_out) store16(a.res_out, row * a.ldro + 16 * unit, a.res_bf16, v[i]);
                    if (a.res_bf16) {
                        // the norm reads the residual as it is stored
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[i][j] = widen(bf16_pair(v[i][j]));
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0ull;
            }
        }
        const float s = row_sum(v, a, s_part[turn][0]);
        float r = __frsqrt_rn(__fadd_rn(__fmul_rn(s, a.inv_k), a.eps));
        // a sum of squares above fp32's range: the row times 2^-80 (exact but for
        // values too small to matter), whose norm is the same; eps is nothing there
        // (a warp that holds several rows goes along where one of them overflows)
        const bool over = !(s < INFINITY);
        if (shared_warp ? __any_sync(0xFFFFFFFFu, over) : over) {
            const uint64_t down = pair_f(over ? 0x1p-80f : 1.0f, over ? 0x1p-80f : 1.0f);
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = mul_f32x2(v[i][j], down);
            const float s2 = row_sum(v, a, s_part[turn][1]);
            if (over) r = __frsqrt_rn(__fmul_rn(s2, a.inv_k));
        }
        const uint64_t rr = pair_f(r, r);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int unit = unit0 + i * blockDim.x;
            const bool in = row < a.M && unit < units;
            const unsigned mask = __ballot_sync(0xFFFFFFFFu, in);
            if (in) {
                if constexpr (kPieces > 1) load16(a.w, 16 * unit, a.w_bf16, w[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = mul_f32x2(mul_f32x2(v[i][j], rr), w[i][j]);
                if (a.norm_out) store16(a.norm_out, row * a.ldn + 16 * unit, a.n_bf16, v[i]);
                if constexpr (kForm >= 0) {
                    rotate_piece<kRot>(v[i], mask);
                    quantize_piece<kForm>(a, row, unit, v[i], mask);
                }
            }
        }
    }
}

// Blocks of up to 512 threads share an SM (64 registers a thread hold 1024 of
// them); rows beyond 8192 values take two pieces a thread, beyond 24576 in an
// instance of their own (1024 threads).
template <int kForm, int kRot>
cudaError_t launch_norm(const NormArgs &a, int sms, cudaStream_t s) {
    const int units = a.K / 16;
    if (a.K <= kOnePiece) {
        const int threads = a.K <= 512 ? 256 : (units + 31) / 32 * 32;
        const int64_t rows = a.K <= 512 ? threads / a.lanes : 1;
        int64_t grid = (a.M + rows - 1) / rows;
        const int64_t most = static_cast<int64_t>(sms) * (1024 / threads);
        if (grid > most) grid = most;
        return launch_pdl(norm_quant_kernel<kForm, kRot, 1, 512>, dim3(static_cast<unsigned>(grid)),
                          dim3(threads), 0, s, a);
    }
    const dim3 grid(static_cast<unsigned>(a.M)), block((units / 2 + 31) / 32 * 32);
    if (block.x <= 768) return launch_pdl(norm_quant_kernel<kForm, kRot, 2, 768>, grid, block, 0, s, a);
    return launch_pdl(norm_quant_kernel<kForm, kRot, 2, 1024>, grid, block, 0, s, a);
}

template <int kForm>
cudaError_t launch_norm_rot(const NormArgs &a, int rot, int sms, cudaStream_t s) {
    switch (rot) {
        case 0: return launch_norm<kForm, 0>(a, sms, s);
        case 32: return launch_norm<kForm, 32>(a, sms, s);
        case 64: return launch_norm<kForm, 64>(a, sms, s);
        default: return launch_norm<kForm, 128>(a, sms, s);
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
    if (M < 0 || K <= 0 || (K % 32) != 0 || K > kMaxRow || ldx < K)
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
    int sms = 0;
    H32_TRY(check_device(&sms));
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
    a.lanes = 2;
    while (a.lanes < K / 16 && a.lanes < 32) a.lanes *= 2;
    a.eps = eps;
    a.inv_k = 1.0f / static_cast<float>(K);
    a.x_bf16 = x_dt == H32_IN_BF16;
    a.res_bf16 = res_dt == H32_IN_BF16;
    a.w_bf16 = w_dt == H32_IN_BF16;
    a.n_bf16 = norm_dt == H32_IN_BF16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (!quant) {
        e = launch_norm<-1, 0>(a, sms, s);
    } else {
        switch (form) {
            case H32_ACT_Q4: e = launch_norm_rot<H32_ACT_Q4>(a, rot, sms, s); break;
            case H32_ACT_Q8: e = launch_norm_rot<H32_ACT_Q8>(a, rot, sms, s); break;
            case H32_ACT_Q4_TC: e = launch_norm_rot<H32_ACT_Q4_TC>(a, rot, sms, s); break;
            case H32_ACT_Q8_TC: e = launch_norm_rot<H32_ACT_Q8_TC>(a, rot, sms, s); break;
            default: e = launch_norm_rot<H32_ACT_Q4_TC_E5M2>(a, rot, sms, s); break;
        }
    }
    return launch_status(e != cudaSuccess ? e : cudaGetLastError());
}
