// Quantizers of the 8-bit floating-point products (sm_103a): e4m3 codes with one fp32
// scale for each 128 values of an activation row, or for each 128 x 128 block of weights.
//
// Per group: v = the rotated values (H of 0, 32, 64 or 128 points, as in h32_quant.cu),
// d = amax|v| / 448, code = the e4m3 number nearest to v * fl(1/d), ties to even.
// 448 is e4m3's largest number, so the largest value of a group gets it.
//
// Both keep 32-blocks in each thread's registers, activations one (the layout of h32_quant.cu:
// the butterfly's strides 1..16 need no exchange, 32 and 64 one shuffle each), weights two,
// and read every value once.  Bound: HBM, 3 bytes a bf16 value, 5 an fp32 one (16384 x 5120 bf16 activations,
// no rotation: 41 us, 92% of the measured copy rate, 128 points 58; weights below); one token by its
// launch, 2.1 us.
#include "h32_common.cuh"
#include "h32_quant_block.cuh"

namespace h32 {
namespace {

__device__ uint32_t g_f8q_status;   // kStatusGuard: a gathered row index out of range

constexpr float kMax = 448.0f;

__device__ __forceinline__ float block_amax(const float (&v)[32]) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) a = fmaxf(a, fabsf(v[i]));
    return a;
}

// four values -> four e4m3 bytes, round to nearest even; beyond 448: 448, NaN: 0x7F
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n.reg .b16 lo, hi;\ncvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\nmov.b32 %0, {lo, hi};\n}\n"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// The block's codes for a group of largest magnitude amax; returns the scale.  Where
// 1/d is not finite (d below 2^-128) the quotient is an IEEE divide instead, as in the
// 4-bit quantizers' degenerate blocks.
__device__ __forceinline__ float f8_codes(const float (&v)[32], float amax, uint32_t (&w)[8]) {
    const float d = __fdiv_rn(amax, kMax);
    const float id = d != 0.0f ? __frcp_rn(d) : 0.0f;
    float q[32];
    if (isinf(id)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) q[i] = __fdiv_rn(v[i], d);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) q[i] = __fmul_rn(v[i], id);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = e4m3x4(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
    return d;
}

// rotate_block of h32_quant_block.cuh with one fma a value for the strides across lanes:
// v + c in the lower block, c - v in the upper one, the same bits (the product is exact)
template <int kRot>
__device__ __forceinline__ void rotate(float (&v)[32], uint32_t pos) {
    if constexpr (kRot <= 32) {
        rotate_block<kRot>(v, pos, 0xFFFFFFFFu);
    } else {
        butterfly32(v);
#pragma unroll
        for (int hb = 1; hb < kRot / 32; hb <<= 1) {
            const float sign = (pos & hb) == 0 ? 1.0f : -1.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __fmaf_rn(v[i], sign, __shfl_xor_sync(0xFFFFFFFFu, v[i], hb));
        }
        const float sc = kRot == 64 ? 0.125f : kInvSqrt128;
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __fmul_rn(v[i], sc);
    }
}

// the same for two blocks in a thread, `upper` in a row's upper half: the stride 32 needs no exchange
template <int kRot>
__device__ __forceinline__ void rotate_pair(float (&v)[2][32], uint32_t upper) {
    if constexpr (kRot <= 32) {
        rotate_block<kRot>(v[0], 0, 0xFFFFFFFFu);
        rotate_block<kRot>(v[1], 0, 0xFFFFFFFFu);
    } else {
        butterfly32(v[0]);
        butterfly32(v[1]);
        const float sign = upper ? -1.0f : 1.0f, sc = kRot == 64 ? 0.125f : kInvSqrt128;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float a = __fadd_rn(v[0][i], v[1][i]), b = __fsub_rn(v[0][i], v[1][i]);
            v[0][i] = a;
            v[1][i] = b;
        }
        if constexpr (kRot == 128) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 32; ++i) v[k][i] = __fmaf_rn(v[k][i], sign, __shfl_xor_sync(0xFFFFFFFFu, v[k][i], 1));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[k][i] = __fmul_rn(v[k][i], sc);
    }
}

template <bool kBf16>
__device__ __forceinline__ void load_block(const void *x, int64_t at, float (&v)[32]) {
    if constexpr (kBf16) load_block_bf16(static_cast<const uint16_t *>(x) + at, v);
    else load_block_f32(static_cast<const float *>(x) + at, v);
}

__device__ __forceinline__ void store_codes(uint8_t *p, const uint32_t (&w)[8]) {
    uint4 *dst = reinterpret_cast<uint4 *>(p);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// A warp takes 4 rows x 8 blocks (lane = 8 r + j), as quant_act_tc_kernel: a group is
// four adjacent lanes, and its scale goes to the group-major array.  row_idx (nullable):
// output row r is input row row_idx[r].
template <bool kBf16, int kRot>
__global__ void __launch_bounds__(256) act_f8_kernel(const void *__restrict__ x, uint32_t M, uint32_t nb,
                                                     int64_t ldx, const int32_t *__restrict__ row_idx,
                                                     int64_t T, uint8_t *__restrict__ xq,
                                                     float *__restrict__ xd, int64_t ldxd) {
    pdl_wait();
    pdl_trigger();
    const uint32_t tiles_b = (nb + 7) / 8, ntiles = ((M + 3) / 4) * tiles_b;
    const uint32_t lane = threadIdx.x & 31, nwarps = gridDim.x * (blockDim.x >> 5);
    for (uint32_t t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < ntiles; t += nwarps) {
        const uint32_t tr = t / tiles_b, tb = t - tr * tiles_b;
        const uint32_t row = tr * 4 + (lane >> 3), b = tb * 8 + (lane & 7);
        bool in = row < M && b < nb;
        const bool out = in;
        int64_t src = row;
        if (row_idx && in) {
            src = __ldg(row_idx + row);
            if (src < 0 || src >= T) {
                atomicOr(&g_f8q_status, kStatusGuard);
                in = false;   // zero codes, a zero scale
            }
        }
        float v[32];
        if (in) {
            load_block<kBf16>(x, src * ldx + 32 * b, v);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        }
        rotate<kRot>(v, b);
        float amax = block_amax(v);
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        uint32_t w[8];
        const float d = f8_codes(v, amax, w);
        if (out) {
            store_codes(xq + (int64_t(row) * nb + b) * 32, w);
            if ((b & 3) == 0) xd[int64_t(b >> 2) * ldxd + row] = d;
        }
    }
}

// One 128 x 128 block after another: two lanes hold a row's 128 values, 256 threads the block, and
// the next one is copied while this one is rotated and rounded.  It comes through shared memory
// (16-byte copies of whole lines: a thread reading its own 128 bytes directly took 264 us for 34816
// x 5120 fp32 and 128 points, staged ones 190, copied ahead 172, all with four lanes a row; two
// lanes, with half the exchange, 159; a lane 162; without a rotation 133, the measured copy rate),
// swizzled so that the eight lanes of a quarter warp, four rows of two halves, read eight different
// bank groups.
__device__ __forceinline__ void copy16(void *smem_dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}

template <bool kBf16>
struct WeightTile {
    static constexpr int kPieces = kBf16 ? 16 : 32;   // 16-byte pieces of a row's 128 values
    static constexpr int kBytes = 128 * kPieces * 16;
    // where piece p of row r stands: its half of the row and the row's low bits move it within
    // the line
    static __device__ __forceinline__ int at(int r, int p) {
        return (r * kPieces + (p ^ (p / (kPieces / 2) + 2 * (r & 3)))) * 16;
    }
};

template <bool kBf16, int kRot>
__global__ void __launch_bounds__(256, 2) weights_f8_kernel(const void *__restrict__ w, uint32_t N, uint32_t nb,
                                                            uint32_t groups, int64_t ldw,
                                                            uint8_t *__restrict__ wq, float *__restrict__ wd) {
    using T = WeightTile<kBf16>;
    extern __shared__ __align__(128) uint8_t s_tile[];
    __shared__ float s_amax[8];
    constexpr int kSize = kBf16 ? 2 : 4, kRows = 256 / T::kPieces;   // rows a round of copies covers
    const int p = threadIdx.x % T::kPieces, r0 = threadIdx.x / T::kPieces;
    const auto copy = [&](uint32_t t) {
        const uint32_t tile_n = t / groups, g = t - tile_n * groups;
        const uint8_t *base = static_cast<const uint8_t *>(w) + (int64_t(tile_n) * 128 * ldw + g * 128) * kSize + p * 16;
        const bool col_in = g * 128 + p * (16 / kSize) < nb * 32;
#pragma unroll
        for (int i = 0; i < 128 / kRows; ++i) {
            const int r = i * kRows + r0;
            const bool in = col_in && tile_n * 128 + r < N;
            copy16(s_tile + T::at(r, p), in ? base + r * ldw * kSize : w, in);
        }
    };
    const uint32_t tiles = (N + 127) / 128 * groups;
    const uint32_t r = threadIdx.x >> 1, j = threadIdx.x & 1;
    copy(blockIdx.x);
    for (uint32_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const uint32_t tile_n = t / groups, g = t - tile_n * groups, row = tile_n * 128 + r, b = g * 4 + 2 * j;
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        float v[2][32];
#pragma unroll
        for (int i = 0; i < T::kPieces / 2; ++i) {
            const uint4 u = *reinterpret_cast<const uint4 *>(s_tile + T::at(r, j * (T::kPieces / 2) + i));
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
            constexpr int kIn = kBf16 ? 8 : 4;   // values of a piece
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float *dst = v[i / (T::kPieces / 4)] + i % (T::kPieces / 4) * kIn + kIn / 4 * q;
                if constexpr (kBf16) {
                    dst[0] = __uint_as_float(x[q] << 16);
                    dst[1] = __uint_as_float(x[q] & 0xFFFF0000u);
                } else {
                    dst[0] = __uint_as_float(x[q]);
                }
            }
        }
        __syncthreads();
        if (t + gridDim.x < tiles) copy(t + gridDim.x);   // (under this block's arithmetic)
        rotate_pair<kRot>(v, j);
        float amax = fmaxf(block_amax(v[0]), block_amax(v[1]));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = amax;
        __syncthreads();   // (its next write is two barriers on)
        amax = s_amax[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) amax = fmaxf(amax, s_amax[i]);
        float d = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t c[8];
            d = f8_codes(v[i], amax, c);
            if (row < N && b + i < nb) store_codes(wq + (int64_t(row) * nb + b + i) * 32, c);
        }
        if (threadIdx.x == 0) wd[t] = d;
    }
}

// what both quantizers ask of their sizes, types and rotation: rows and K below 2^31, as the
// products (the kernels number rows, blocks and a row's values in 32 bits)
h32_status quant_args(h32_in_dtype dt, int64_t rows, int64_t K, int64_t ld, int rotate) {
    constexpr int64_t kMost = 0x7FFFFFFFll - 256;
    if (rows < 0 || rows > kMost || K <= 0 || K > kMost || K % 32 != 0 || ld < K) return H32_ERR_INVALID_ARG;
    const int rot = rot_points(rotate);
    if (rot < 0 || (rot > 0 && K % rot != 0)) return H32_ERR_INVALID_ARG;
    if (dt != H32_IN_F32 && dt != H32_IN_BF16) return H32_ERR_INVALID_ARG;
    return H32_OK;
}

template <bool kBf16>
auto act_kernel(int rotate) {
    switch (rot_points(rotate)) {
        case 0: return act_f8_kernel<kBf16, 0>;
        case 32: return act_f8_kernel<kBf16, 32>;
        case 64: return act_f8_kernel<kBf16, 64>;
        default: return act_f8_kernel<kBf16, 128>;
    }
}
template <bool kBf16>
auto weights_kernel(int rotate) {
    switch (rot_points(rotate)) {
        case 0: return weights_f8_kernel<kBf16, 0>;
        case 32: return weights_f8_kernel<kBf16, 32>;
        case 64: return weights_f8_kernel<kBf16, 64>;
        default: return weights_f8_kernel<kBf16, 128>;
    }
}

}  // namespace

__device__ uint32_t g_f8q_status_taken;
__global__ void take_g_f8q_status() { g_f8q_status_taken = atomicExch(&g_f8q_status, 0u); }

h32_status f8q_read_and_clear_status(cudaStream_t s) {
    bool ok = false;
    const uint32_t v = take_status(take_g_f8q_status, g_f8q_status_taken, s, &ok);
    if (!ok) return H32_ERR_CUDA;
    return (v & kStatusGuard) ? H32_ERR_DEVICE_GUARD : H32_OK;
}

}  // namespace h32

extern "C" h32_status h32_quantize_act_f8(const void *x, h32_in_dtype dt, int64_t T, int64_t K, int64_t ldx,
                                          const int32_t *row_idx, int64_t R, uint8_t *xq, float *xd,
                                          int64_t ldxd, int rotate, void *stream) {
    using namespace h32;
    H32_TRY(quant_args(dt, T, K, ldx, rotate));
    if (R < 0 || R > 0x7FFFFFFFll || ldxd < R || ldxd % 4 != 0 || (!row_idx && R != T)) return H32_ERR_INVALID_ARG;
    if (R == 0) return H32_OK;
    if (!x || !xq || !xd || T == 0) return H32_ERR_INVALID_ARG;
    const int64_t esize = dt == H32_IN_BF16 ? 2 : 4;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(xd) || (ldx * esize) % 16 != 0 ||
        (row_idx && reinterpret_cast<uintptr_t>(row_idx) % 4 != 0))
        return H32_ERR_ALIGNMENT;
    if (R * (K / 32) > 0x7FFFFFFFll) return H32_ERR_INVALID_ARG;
    int sms = 0;
    H32_TRY(check_device(&sms));
    const uint32_t nb = static_cast<uint32_t>(K / 32);
    const int64_t tiles = (R + 3) / 4 * ((nb + 7) / 8), want = (tiles + 7) / 8;
    if (tiles > 0x7FFFFFFFll) return H32_ERR_INVALID_ARG;
    const int grid = static_cast<int>(want < int64_t(sms) * 8 ? want : int64_t(sms) * 8);
    const auto kernel = dt == H32_IN_BF16 ? act_kernel<true>(rotate) : act_kernel<false>(rotate);
    const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), x,
                                     static_cast<uint32_t>(R), nb, ldx, row_idx, T, xq, xd, ldxd);
    return launch_status(e != cudaSuccess ? e : cudaGetLastError());
}

extern "C" h32_status h32_quantize_weights_f8(const void *w, h32_in_dtype dt, int64_t N, int64_t K, int64_t ldw,
                                              int rotate, uint8_t *wq, float *wd, void *stream) {
    using namespace h32;
    H32_TRY(quant_args(dt, N, K, ldw, rotate));
    if (N == 0) return H32_OK;
    if (!w || !wq || !wd) return H32_ERR_INVALID_ARG;
    const int64_t esize = dt == H32_IN_BF16 ? 2 : 4;
    if (!aligned16(w) || !aligned16(wq) || !aligned16(wd) || (ldw * esize) % 16 != 0) return H32_ERR_ALIGNMENT;
    const int64_t groups = (K + 127) / 128, tiles = (N + 127) / 128 * groups;
    if (tiles > 0x7FFFFFFFll) return H32_ERR_INVALID_ARG;
    int sms = 0;
    H32_TRY(check_device(&sms));
    const auto kernel = dt == H32_IN_BF16 ? weights_kernel<true>(rotate) : weights_kernel<false>(rotate);
    const int smem = dt == H32_IN_BF16 ? WeightTile<true>::kBytes : WeightTile<false>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return launch_status(e);
    kernel<<<static_cast<int>(tiles < 2 * sms ? tiles : 2 * sms), 256, smem, reinterpret_cast<cudaStream_t>(stream)>>>(
        w, static_cast<uint32_t>(N), static_cast<uint32_t>(K / 32), static_cast<uint32_t>(groups), ldw, wq, wd);
    return launch_status(cudaGetLastError());
}
