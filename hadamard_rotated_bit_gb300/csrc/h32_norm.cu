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
// Blocks of threads walk the rows, so the weights stay in registers, and one thread
// copies the rows to come into shared memory (bulk copies), which keeps the reads
// going while a row is summed and rounded; products, sums and butterflies work on
// packed pairs.  16384 x 5120, bf16 with a bf16 residual, 4-bit codes: 100 us,
// 6.0 TB/s of the 7.1 bytes an element, 90% of the measured copy rate (without the
// copies ahead 136 us).
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
    uint8_t res_bf16, w_bf16, n_bf16;
    int32_t form, rot;   // an h32_act_form or -1 (norm_out alone); points
    uint64_t wait_limit;
};

__device__ uint32_t g_norm_status;   // kStatusTimeout: a wait for a row's copy gave up
constexpr uint64_t kDrainPolls = 1ull << 22;

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

// 16 values, bf16 or fp32.  Plain loads: x and the residual may be the very rows
// this kernel writes.
template <bool kBf16>
__device__ __forceinline__ void load_piece(const uint8_t *p, uint64_t (&v)[8]) {
    if constexpr (kBf16) {
        const uint4 u[2] = {reinterpret_cast<const uint4 *>(p)[0], reinterpret_cast<const uint4 *>(p)[1]};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            v[4 * c] = widen(u[c].x);
            v[4 * c + 1] = widen(u[c].y);
            v[4 * c + 2] = widen(u[c].z);
            v[4 * c + 3] = widen(u[c].w);
        }
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const ulonglong2 u = reinterpret_cast<const ulonglong2 *>(p)[c];
            v[2 * c] = u.x;
            v[2 * c + 1] = u.y;
        }
    }
}

// sum of two bf16 pairs, each rounded once: the same as the fp32 sum rounded to
// bf16 (an fp32 sum of two bf16 values is inexact only when they are 16 binades
// apart, and then far from a bf16 tie)
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint4 add_bf16x8(const uint4 &a, const uint4 &b) {
    return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z),
                      add_bf16x2(a.w, b.w));
}

// 16 values rounded to bf16 or as they are
__device__ __forceinline__ void store_piece(uint8_t *p, bool bf16, const uint64_t (&v)[8]) {
    if (bf16) {
        uint4 *q = reinterpret_cast<uint4 *>(p);
        q[0] = make_uint4(bf16_pair(v[0]), bf16_pair(v[1]), bf16_pair(v[2]), bf16_pair(v[3]));
        q[1] = make_uint4(bf16_pair(v[4]), bf16_pair(v[5]), bf16_pair(v[6]), bf16_pair(v[7]));
    } else {
        ulonglong2 *q = reinterpret_cast<ulonglong2 *>(p);
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
// s_part: 64 floats.
template <int kPieces>
__device__ __forceinline__ float row_sum(const uint64_t (&v)[kPieces][8], const NormArgs &a,
                                         float *s_part) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        float s = piece_sum(v[i]);
        if (kPieces == 1 && a.K <= 512) {
            for (int o = 1; o < a.lanes; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
            return s;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
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
__device__ __forceinline__ void rotate_piece(uint64_t (&v)[8], int rot, unsigned mask) {
    if (rot == 0) return;
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
    for (int hb = 1; hb <= rot >> 5; hb <<= 1) {   // strides 16, 32, 64
        const float sign = (threadIdx.x & hb) ? -1.0f : 1.0f;
        const uint64_t sg = pair_f(sign, sign);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float clo = __shfl_xor_sync(mask, lo_f(v[i]), hb);
            const float chi = __shfl_xor_sync(mask, hi_f(v[i]), hb);
            v[i] = fma_f32x2(v[i], sg, pair_f(clo, chi));   // lower: v + c, upper: c - v
        }
    }
    const float k = rot == 32 ? kInvSqrt32 : rot == 64 ? 0.125f : kInvSqrt128;
    const uint64_t sc = pair_f(k, k);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = mul_f32x2(v[i], sc);
}

// Codes and scale of the lane's half of block `unit / 2` of row `row`: the steps of
// quant_bits (h32_quant_block.cuh) on packed pairs.
template <int kForm>
__device__ __forceinline__ void quantize_piece(const NormArgs &a, int64_t row, int unit,
                                               const uint64_t (&p)[8], unsigned mask) {
    constexpr int kBits = (kForm == H32_ACT_Q8 || kForm == H32_ACT_Q8_TC) ? 8 : 4;
    constexpr float kQmax = kBits == 4 ? 7.0f : 127.0f, kQmin = kBits == 4 ? -8.0f : -127.0f;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(lo_f(p[i])), fabsf(hi_f(p[i]))));
    amax = fmaxf(amax, __shfl_xor_sync(mask, amax, 1));
    const float d = __fdiv_rn(amax, kQmax);
    const float id = (d != 0.0f) ? __frcp_rn(d) : 0.0f;
    const uint64_t magic = pair_f(kRoundMagic, kRoundMagic);
    uint64_t t[8];   // code + 1.5 * 2^23
    if (!(amax < INFINITY) || isinf(id)) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = add_f32x2(pair_f(degenerate_code(lo_f(p[i]), d, kQmin, kQmax),
                                    degenerate_code(hi_f(p[i]), d, kQmin, kQmax)),
                             magic);
    } else {
        // the product rounded by itself (scalar: the compiler joins a packed product and
        // the sum after it into one fma, which moves a tie)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            t[i] = add_f32x2(pair_f(__fmul_rn(lo_f(p[i]), id), __fmul_rn(hi_f(p[i]), id)), magic);
    }
    const int odd = unit & 1, b = unit >> 1;
    const int64_t K = a.K;
    uint8_t *xq = static_cast<uint8_t *>(a.xq);
    if constexpr (kForm == H32_ACT_Q4_TC || kForm == H32_ACT_Q4_TC_E5M2) {
        // the codes as integer-valued floats, converted exactly by the hardware
        const uint64_t back = pair_f(-kRoundMagic, -kRoundMagic);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t c = add_f32x2(t[2 * k], back), e = add_f32x2(t[2 * k + 1], back);
            w[k] = kForm == H32_ACT_Q4_TC ? e4m3x4_of_ints(lo_f(c), hi_f(c), lo_f(e), hi_f(e))
                                          : e5m2x4_of_ints_x512(lo_f(c), hi_f(c), lo_f(e), hi_f(e));
        }
        *reinterpret_cast<uint4 *>(xq + row * K + 16 * unit) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            w[k] = pack_low_bytes(static_cast<uint32_t>(t[2 * k]), static_cast<uint32_t>(t[2 * k] >> 32),
                                  static_cast<uint32_t>(t[2 * k + 1]),
                                  static_cast<uint32_t>(t[2 * k + 1] >> 32));
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

constexpr int kNoRes = 0, kResF32 = 1, kResBf16 = 2;

// the piece of a row: x + residual, stored and rounded as the residual is, and
// widened to fp32
template <bool kXB, int kRes>
__device__ __forceinline__ void load_sum(const uint8_t *x, const uint8_t *r, uint8_t *out,
                                         uint64_t (&v)[8]) {
    if constexpr (kXB && kRes == kResBf16) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint4 h = add_bf16x8(reinterpret_cast<const uint4 *>(x)[c],
                                       reinterpret_cast<const uint4 *>(r)[c]);
            if (out) reinterpret_cast<uint4 *>(out)[c] = h;
            v[4 * c] = widen(h.x);
            v[4 * c + 1] = widen(h.y);
            v[4 * c + 2] = widen(h.z);
            v[4 * c + 3] = widen(h.w);
        }
    } else {
        load_piece<kXB>(x, v);
        if constexpr (kRes != kNoRes) {
            uint64_t u[8];
            load_piece<kRes == kResBf16>(r, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = add_f32x2(v[j], u[j]);
            if constexpr (kRes == kResBf16) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 h = make_uint4(bf16_pair(v[4 * c]), bf16_pair(v[4 * c + 1]),
                                               bf16_pair(v[4 * c + 2]), bf16_pair(v[4 * c + 3]));
                    if (out) reinterpret_cast<uint4 *>(out)[c] = h;
                    v[4 * c] = widen(h.x);
                    v[4 * c + 1] = widen(h.y);
                    v[4 * c + 2] = widen(h.z);
                    v[4 * c + 3] = widen(h.w);
                }
            } else if (out) {
                store_piece(out, false, v);
            }
        }
    }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const uint8_t *src, uint32_t bytes,
                                          uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

constexpr int kSlots = 2;   // rows a block has in flight ahead

// A thread holds kPieces pieces of 16 values of a row, blockDim.x * 16 values apart.
// With one piece a block walks rows (its weights stay in registers) and, with
// kAhead, one thread copies the rows to come into shared memory; with two pieces it
// takes one row.  Types are compiled in (they decide the registers), the form and
// the rotation are branches the whole launch takes alike.
template <bool kXB, int kRes, int kPieces, bool kAhead, int kThreads>
__global__ void __launch_bounds__(kThreads, kPieces == 1 ? 2 : 1) norm_quant_kernel(const NormArgs a) {
    __shared__ float s_part[2][2][64];
    __shared__ uint64_t s_full[kSlots];
    extern __shared__ __align__(16) uint8_t s_rows[];
    constexpr int xs = kXB ? 2 : 4, rs = kRes == kResBf16 ? 2 : 4;   // bytes a value
    // rows of at most 512 values: several in a warp
    const bool shared_warp = kPieces == 1 && !kAhead && a.K <= 512;
    const int rows = shared_warp ? blockDim.x / a.lanes : 1;
    const int unit0 = shared_warp ? threadIdx.x & (a.lanes - 1) : threadIdx.x;
    const int units = a.K / 16;
    const uint32_t x_bytes = a.K * xs, r_bytes = kRes != kNoRes ? a.K * rs : 0;
    if (kAhead) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < kSlots; ++i) mbar_init(&s_full[i], 1);
            fence_barrier_init();
        }
        __syncthreads();
    }
    pdl_wait();
    pdl_trigger();
    const uint8_t *ax = static_cast<const uint8_t *>(a.x), *ar = static_cast<const uint8_t *>(a.res);
    auto copy_row = [&](int64_t row, int slot) {   // one thread
        if (row >= a.M) return;
        const uint32_t to = smem_u32(s_rows) + slot * (x_bytes + r_bytes);
        mbar_arrive_expect_tx(&s_full[slot], x_bytes + r_bytes);
        bulk_load(to, ax + row * a.ldx * xs, x_bytes, &s_full[slot]);
        if (kRes != kNoRes) bulk_load(to + x_bytes, ar + row * a.ldr * rs, r_bytes, &s_full[slot]);
    };
    if (kAhead && threadIdx.x == 0)
        for (int i = 0; i < kSlots; ++i) copy_row(blockIdx.x + static_cast<int64_t>(i) * gridDim.x, i);
    auto load_w = [&](int unit, uint64_t (&w)[8]) {
        if (a.w_bf16) load_piece<true>(static_cast<const uint8_t *>(a.w) + 32 * unit, w);
        else load_piece<false>(static_cast<const uint8_t *>(a.w) + 64 * unit, w);
    };
    uint64_t w[8];
    if (kPieces == 1 && unit0 < units) load_w(unit0, w);
    const int64_t my_row = shared_warp ? threadIdx.x / a.lanes : 0;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * rows;
    int turn = 0;           // the slot, and which half of s_part
    uint32_t phase = 0;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * rows; row0 < a.M; row0 += stride) {
        const int64_t row = row0 + my_row;
        uint64_t v[kPieces][8];
        if (kAhead && !warp_wait_or_look(&s_full[turn], phase, a.wait_limit, nullptr)) {
            // gave up: the block's rows from this one on are undefined; the thread that
            // copies leaves when its copies under way have landed, or after as long again
            if ((threadIdx.x & 31) == 0) atomicOr(&g_norm_status, kStatusTimeout);
            if (threadIdx.x == 0)
                for (int i = 0; i < kSlots; ++i)
                    if (row + i * stride < a.M)
                        mbar_wait_bounded(&s_full[(turn + i) % kSlots],
                                          turn + i < kSlots ? phase : phase ^ 1, kDrainPolls, nullptr);
            return;
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int unit = unit0 + i * blockDim.x;
            if (row < a.M && unit < units) {
                const uint8_t *xp = ax + (row * a.ldx + 16 * unit) * xs;
                const uint8_t *rp = kRes != kNoRes ? ar + (row * a.ldr + 16 * unit) * rs : nullptr;
                if constexpr (kAhead) {
                    xp = s_rows + turn * (x_bytes + r_bytes) + 16 * xs * unit;
                    rp = s_rows + turn * (x_bytes + r_bytes) + x_bytes + 16 * rs * unit;
                }
                uint8_t *out = (kRes != kNoRes && a.res_out)
                                   ? static_cast<uint8_t *>(a.res_out) + (row * a.ldro + 16 * unit) * rs
                                   : nullptr;
                load_sum<kXB, kRes>(xp, rp, out, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0ull;
            }
        }
        const float s = row_sum(v, a, s_part[turn][0]);
        // (the block has met in row_sum: every thread has read its part of the slot)
        if (kAhead && threadIdx.x == 0) copy_row(row + kSlots * stride, turn);
        const float ms = __fadd_rn(__fmul_rn(s, a.inv_k), a.eps);
        float r = __frsqrt_rn(ms);
        // a mean square above fp32's range: the row times 2^-80 (exact but for values too
        // small to matter) and eps times 2^-160 (nothing unless eps is huge), whose norm is
        // the same (a warp that holds several rows goes along where one of them overflows)
        const bool over = !(ms < INFINITY);
        if (shared_warp ? __any_sync(0xFFFFFFFFu, over) : over) {
            const uint64_t down = pair_f(over ? 0x1p-80f : 1.0f, over ? 0x1p-80f : 1.0f);
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = mul_f32x2(v[i][j], down);
            const float s2 = row_sum(v, a, s_part[turn][1]);
            if (over)
                r = __frsqrt_rn(__fadd_rn(__fmul_rn(s2, a.inv_k),
                                          __fmul_rn(__fmul_rn(a.eps, 0x1p-80f), 0x1p-80f)));
        }
        const uint64_t rr = pair_f(r, r);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int unit = unit0 + i * blockDim.x;
            const bool in = row < a.M && unit < units;
            const unsigned mask = __ballot_sync(0xFFFFFFFFu, in);
            if (in) {
                if (kPieces > 1) load_w(unit, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = mul_f32x2(mul_f32x2(v[i][j], rr), w[j]);
                if (a.norm_out)
                    store_piece(static_cast<uint8_t *>(a.norm_out) +
                                    (row * a.ldn + 16 * unit) * (a.n_bf16 ? 2 : 4),
                                a.n_bf16, v[i]);
                if (a.form >= 0) {
                    rotate_piece(v[i], a.rot, mask);
                    switch (a.form) {
                        case H32_ACT_Q4: quantize_piece<H32_ACT_Q4>(a, row, unit, v[i], mask); break;
                        case H32_ACT_Q8: quantize_piece<H32_ACT_Q8>(a, row, unit, v[i], mask); break;
                        case H32_ACT_Q4_TC: quantize_piece<H32_ACT_Q4_TC>(a, row, unit, v[i], mask); break;
                        case H32_ACT_Q8_TC: quantize_piece<H32_ACT_Q8_TC>(a, row, unit, v[i], mask); break;
                        default: quantize_piece<H32_ACT_Q4_TC_E5M2>(a, row, unit, v[i], mask); break;
                    }
                }
            }
        }
        turn ^= 1;
        phase ^= turn == 0;
    }
}

// Blocks of up to 512 threads share an SM (64 registers a thread hold 1024 of
// them); rows beyond 8192 values take two pieces a thread, one block an SM, beyond
// 24576 in an instance of their own (1024 threads).  With four or more rows for
// every block that an SM holds, blocks walk the rows and copy the next ones ahead,
// where the copies have room (16384 x 5120, bf16: 100 us, a block a row 161);
// with fewer, one block takes one row (512 x 5120: 9.0 us, walking 9.7).
template <bool kXB, int kRes, int kPieces, int kThreads>
cudaError_t launch_rows(const NormArgs &a, int threads, int64_t blocks, int64_t most, int per_sm,
                        cudaStream_t s) {
    const int bytes = kSlots * a.K * ((kXB ? 2 : 4) + (kRes == kNoRes ? 0 : kRes == kResBf16 ? 2 : 4));
    const bool ahead = a.K > 512 && blocks >= 4 * most && bytes * per_sm <= 220 * 1024;
    if (!ahead) {
        if (a.K <= 512 && blocks > 4 * most) blocks = 4 * most;
        return launch_pdl(norm_quant_kernel<kXB, kRes, kPieces, false, kThreads>,
                          dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, s, a);
    }
    if (bytes > 40960) {
        const cudaError_t e =
            cudaFuncSetAttribute(norm_quant_kernel<kXB, kRes, kPieces, true, kThreads>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(norm_quant_kernel<kXB, kRes, kPieces, true, kThreads>,
                      dim3(static_cast<unsigned>(most)), dim3(threads), bytes, s, a);
}

template <bool kXB, int kRes>
cudaError_t launch_norm(const NormArgs &a, int sms, cudaStream_t s) {
    const int units = a.K / 16;
    if (a.K <= kOnePiece) {
        const int threads = a.K <= 512 ? 256 : (units + 31) / 32 * 32;
        const int64_t rows = a.K <= 512 ? threads / a.lanes : 1;
        const int per_sm = 1024 / threads;
        return launch_rows<kXB, kRes, 1, 512>(a, threads, (a.M + rows - 1) / rows,
                                              static_cast<int64_t>(sms) * per_sm, per_sm, s);
    }
    const int threads = (units / 2 + 31) / 32 * 32;
    if (threads <= 768) return launch_rows<kXB, kRes, 2, 768>(a, threads, a.M, sms, 1, s);
    return launch_rows<kXB, kRes, 2, 1024>(a, threads, a.M, sms, 1, s);
}

template <bool kXB>
cudaError_t launch_norm_res(const NormArgs &a, int sms, cudaStream_t s) {
    if (!a.res) return launch_norm<kXB, kNoRes>(a, sms, s);
    return a.res_bf16 ? launch_norm<kXB, kResBf16>(a, sms, s) : launch_norm<kXB, kResF32>(a, sms, s);
}

inline bool dtype_ok(h32_in_dtype dt) { return dt == H32_IN_F32 || dt == H32_IN_BF16; }
inline int64_t bytes_of(h32_in_dtype dt) { return dt == H32_IN_BF16 ? 2 : 4; }

}  // namespace

__device__ uint32_t g_norm_status_taken;
__global__ void take_g_norm_status() { g_norm_status_taken = atomicExch(&g_norm_status, 0u); }

h32_status norm_read_and_clear_status(cudaStream_t s) {
    bool ok = false;
    const uint32_t v = take_status(take_g_norm_status, g_norm_status_taken, s, &ok);
    if (!ok) return H32_ERR_CUDA;
    return (v & kStatusTimeout) ? H32_ERR_TIMEOUT : H32_OK;
}

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
    a.wait_limit = wait_limit();
    a.res_bf16 = res_dt == H32_IN_BF16;
    a.w_bf16 = w_dt == H32_IN_BF16;
    a.n_bf16 = norm_dt == H32_IN_BF16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    a.form = quant ? form : -1;
    a.rot = rot;
    const cudaError_t e = x_dt == H32_IN_BF16 ? launch_norm_res<true>(a, sms, s)
                                              : launch_norm_res<false>(a, sms, s);
    return launch_status(e != cudaSuccess ? e : cudaGetLastError());
}
