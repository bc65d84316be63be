// The block-scaled product of a few tokens (sm_103a): one new token of each
// sequence through a projection, with the epilogue of h32_finish.cuh.
//
// Per weight row and token the same definition as the tensor-core GEMM, bit for
// bit: exact integer sums S of 32-blocks, then acc = fma(fl(d_w d_x), S, acc) in
// block order.  The tensor-core GEMM runs 128-row tiles over the whole of K one
// block step after another, which for a few tokens leaves most of the card idle
// (5120 x 5120, one token: 35 us).  Here the sums and the ordered folds are taken
// apart: all warps stream weight rows and form sums, any order, as they are exact;
// one warp a token folds them in order.
//
// Bound: HBM, 1.125 bytes a weight.  A block takes 8 RW rows (RW a warp), in steps
// of 1024 codes.  A lane loads 16 codes (16 bytes) of each row, widens them to fp16
// pairs, and multiplies by the tokens' codes (fp16 in shared memory, widened once a
// step): |w x| <= 64, so 32 products sum exactly in fp16 (|S| <= 2048).  An 8-bit
// activation code is 16 h + l, two such sums (16 h: multiples of 16 up to 8192; l:
// up to 960, a lane), added in fp32.  A register is loaded again for the next step
// as soon as its codes are widened, so each block keeps 8 KB a row pair in flight.
// The sums go to shared memory, two buffers, one barrier a step: while warp m folds
// the step for token m the others form the next one's.
#include "h32_few.cuh"

#include <cuda_fp16.h>

namespace h32 {
namespace {

constexpr int kWarps = 8;
constexpr int kStep = 1024;           // codes a step
constexpr int kBlocks = kStep / 32;   // 32-blocks a step
constexpr int kLoads = kStep / 512;   // 16-byte loads of a row, a lane and step

struct FewArgs {
    const uint8_t *wp, *xw;
    const float *wsc, *xdt;
    int64_t ldws, ldxd;
    int32_t M, N, K;
    EpiArgs fin;
};

// two e4m3 bytes -> an fp16 pair, exact
__device__ __forceinline__ uint32_t half2_of(uint16_t b) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(b));
    return r;
}
__device__ __forceinline__ void widen16(const uint4 &q, uint32_t (&h)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[2 * i] = half2_of(static_cast<uint16_t>(w[i]));
        h[2 * i + 1] = half2_of(static_cast<uint16_t>(w[i] >> 16));
    }
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float half_sum(uint32_t h) {
    const __half2 v = *reinterpret_cast<const __half2 *>(&h);
    return __low2float(v) + __high2float(v);
}

// Shared memory: sums [2][kBlocks][MT][rows + pad], activations [2][MT][kLoads]
// [pairs of 16 bytes][32 lanes], weight scales [2][kBlocks][rows + 1], activation
// scales [2][MT][kBlocks].
template <int XB, int MT, int RW>
struct FewCfg {
    static constexpr int kRows = kWarps * RW;
    // sums: fp16 (4-bit) with 2 halves of padding, or fp32 with one word
    static constexpr int kSumStride = XB == 4 ? (kRows + 2) * 2 : (kRows + 1) * 4;
    static constexpr int kSumBytes = kBlocks * MT * kSumStride;
    static constexpr int kActVecs = 2 * (XB / 4);                       // uint4 a lane and load
    static constexpr int kActBytes = MT * kLoads * kActVecs * 512;
    static constexpr int kDwBytes = kBlocks * (kRows + 1) * 4;
    static constexpr int kDxBytes = MT * kBlocks * 4;
    static constexpr int kOffAct = 2 * ((kSumBytes + 15) & ~15);
    static constexpr int kOffDw = kOffAct + 2 * kActBytes;
    static constexpr int kOffDx = kOffDw + 2 * kDwBytes;
    static constexpr int kSmem = kOffDx + 2 * kDxBytes;
};

template <int XB, int MT, int RW>
__global__ void __launch_bounds__(kWarps * 32, 2) few_kernel(const FewArgs a) {
    using C = FewCfg<XB, MT, RW>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n0 = blockIdx.x * C::kRows;
    const int nb = a.K / 32, steps = (a.K + kStep - 1) / kStep;
    auto s_sum = [&](int buf) { return smem + buf * (C::kOffAct / 2); };
    auto s_act = [&](int buf) { return reinterpret_cast<uint4 *>(smem + C::kOffAct + buf * C::kActBytes); };
    auto s_dw = [&](int buf) { return reinterpret_cast<float *>(smem + C::kOffDw + buf * C::kDwBytes); };
    auto s_dx = [&](int buf) { return reinterpret_cast<float *>(smem + C::kOffDx + buf * C::kDxBytes); };
    pdl_wait();
    pdl_trigger();

    const int row0 = n0 + warp * RW;
    const uint8_t *wrow = a.wp + static_cast<int64_t>(row0) * a.K + lane * 16;
    uint4 wq[kLoads][RW];
    float dw[RW], dx = 0.0f;
    auto load_w = [&](int st, int i) {
        const int k = st * kStep + i * 512 + lane * 16;
#pragma unroll
        for (int r = 0; r < RW; ++r)
            wq[i][r] = (k < a.K && row0 + r < a.N)
                           ? __ldg(reinterpret_cast<const uint4 *>(
                                 wrow + static_cast<int64_t>(r) * a.K + (st * kStep + i * 512)))
                           : make_uint4(0u, 0u, 0u, 0u);
    };
    auto load_scales = [&](int st) {   // a block of the step a lane; a token a warp
        const int b = st * kBlocks + lane;
#pragma unroll
        for (int r = 0; r < RW; ++r)
            dw[r] = (b < nb && row0 + r < a.N) ? __ldg(a.wsc + (row0 + r) * a.ldws + b) : 0.0f;
        if (warp < MT) dx = (warp < a.M && b < nb) ? __ldg(a.xdt + b * a.ldxd + warp) : 0.0f;
    };
    // the step's activations, widened into shared memory
    auto stage_x = [&](int st, int buf) {
        constexpr int kItems = MT * kLoads * 32;
#pragma unroll
        for (int it = 0; it < (kItems + kWarps * 32 - 1) / (kWarps * 32); ++it) {
            const int item = it * kWarps * 32 + tid;
            if (kItems % (kWarps * 32) != 0 && item >= kItems) break;
            const int m = item / (kLoads * 32), i = (item / 32) % kLoads, ln = item & 31;
            const int k = st * kStep + i * 512 + ln * 16;
            const bool in = m < a.M && k < a.K;
            uint4 *dst = s_act(buf) + (m * kLoads + i) * C::kActVecs * 32 + ln;
#pragma unroll
            for (int p = 0; p < XB / 4; ++p) {
                // 4-bit: the codes' bytes; 8-bit: a block's 32 bytes of 16 h, then of l
                const uint8_t *src =
                    XB == 4 ? a.xw + static_cast<int64_t>(m) * a.K + k
                            : a.xw + static_cast<int64_t>(m) * 2 * a.K + (k >> 5) * 64 + p * 32 + (k & 16);
                uint32_t h[8];
                widen16(in ? __ldg(reinterpret_cast<const uint4 *>(src)) : make_uint4(0u, 0u, 0u, 0u), h);
                dst[(2 * p) * 32] = make_uint4(h[0], h[1], h[2], h[3]);
                dst[(2 * p + 1) * 32] = make_uint4(h[4], h[5], h[6], h[7]);
            }
        }
    };

#pragma unroll
    for (int i = 0; i < kLoads; ++i) load_w(0, i);
    load_scales(0);
    stage_x(0, 0);
    __syncthreads();

    float acc = 0.0f;   // of row n0 + lane and token `warp`
    for (int st = 0; st < steps; ++st) {
        const int buf = st & 1;
        uint8_t *sum = s_sum(buf);
#pragma unroll
        for (int r = 0; r < RW; ++r) s_dw(buf)[lane * (C::kRows + 1) + warp * RW + r] = dw[r];
        if (warp < MT) s_dx(buf)[warp * kBlocks + lane] = dx;
        if (st + 1 < steps) load_scales(st + 1);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            uint32_t w[RW][8];
#pragma unroll
            for (int r = 0; r < RW; ++r) widen16(wq[i][r], w[r]);
            if (st + 1 < steps) load_w(st + 1, i);
            const int b = i * 16 + (lane >> 1);   // the lane pair's block within the step
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if (m < a.M) {
                    const uint4 *act = s_act(buf) + (m * kLoads + i) * C::kActVecs * 32 + lane;
                    if constexpr (XB == 4) {
                        const uint4 x0 = act[0], x1 = act[32];
                        const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                        uint32_t s[RW];
#pragma unroll
                        for (int r = 0; r < RW; ++r) {
                            uint32_t t = 0u;
#pragma unroll
                            for (int j = 0; j < 8; ++j) t = hfma2(w[r][j], x[j], t);
                            s[r] = t;
                        }
                        __half *to = reinterpret_cast<__half *>(sum + (b * MT + m) * C::kSumStride) + warp * RW;
                        if constexpr (RW == 1) {
                            const uint32_t t = hadd2(s[0], s[0] >> 16);   // low half: both
                            const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, t, 1);
                            if (!(lane & 1)) {
                                const uint32_t f = hadd2(t, o);
                                to[0] = __ushort_as_half(static_cast<uint16_t>(f));
                            }
                        } else {
                            // two rows' sums as one pair
                            uint32_t f[RW / 2];
#pragma unroll
                            for (int q = 0; q < RW / 2; ++q) {
                                const uint32_t t = hadd2(__byte_perm(s[2 * q], s[2 * q + 1], 0x5410),
                                                         __byte_perm(s[2 * q], s[2 * q + 1], 0x7632));
                                f[q] = hadd2(t, __shfl_xor_sync(0xFFFFFFFFu, t, 1));
                            }
                            if constexpr (RW == 2) {
                                if (!(lane & 1)) *reinterpret_cast<uint32_t *>(to) = f[0];
                            } else {
                                *reinterpret_cast<uint32_t *>(to + 2 * (lane & 1)) = (lane & 1) ? f[1] : f[0];
                            }
                        }
                    } else {
                        float s[RW];
#pragma unroll
                        for (int r = 0; r < RW; ++r) s[r] = 0.0f;
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const uint4 x0 = act[(2 * p) * 32], x1 = act[(2 * p + 1) * 32];
                            const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                            for (int r = 0; r < RW; ++r) {
                                uint32_t t = 0u;
#pragma unroll
                                for (int j = 0; j < 8; ++j) t = hfma2(w[r][j], x[j], t);
                                s[r] += half_sum(t);
                            }
                        }
                        float *to = reinterpret_cast<float *>(sum + (b * MT + m) * C::kSumStride) + warp * RW;
#pragma unroll
                        for (int r = 0; r < RW; ++r) {
                            s[r] += __shfl_xor_sync(0xFFFFFFFFu, s[r], 1);
                            if ((lane & 1) == (r & 1) || (RW == 1 && !(lane & 1))) to[r] = s[r];
                        }
                    }
                }
            }
        }
        if (st + 1 < steps) stage_x(st + 1, buf ^ 1);
        __syncthreads();
        // warp m folds the step for token m, its blocks in order, a row a lane
        if (warp < MT && warp < a.M && lane < C::kRows) {
            const int n = min(kBlocks, nb - st * kBlocks);
            const float *dwp = s_dw(buf) + lane, *dxp = s_dx(buf) + warp * kBlocks;
            const uint8_t *sp = sum + warp * C::kSumStride;
#pragma unroll 8
            for (int b = 0; b < n; ++b) {
                const uint8_t *at = sp + b * MT * C::kSumStride;
                const float S = XB == 4 ? __half2float(reinterpret_cast<const __half *>(at)[lane])
                                        : reinterpret_cast<const float *>(at)[lane];
                acc = __fmaf_rn(__fmul_rn(dwp[b * (C::kRows + 1)], dxp[b]), S, acc);
            }
        }
    }
    if (warp >= MT || warp >= a.M) return;
    // bias, activation, residual: gate and up rows sit in adjacent lanes
    const EpiArgs &f = a.fin;
    const int n = n0 + lane;
    const bool in = lane < C::kRows && n < a.N;
    float z = acc;
    if (f.bias && in) z = __fadd_rn(z, __ldg(f.bias + n));
    int j = n;
    bool out = in;
    if (f.act == H32_EPI_SWIGLU) {
        const float up = __shfl_xor_sync(0xFFFFFFFFu, z, 1);
        z = swiglu(z, up);
        j = n >> 1;
        out = in && !(lane & 1);
    } else {
        z = activate(z, f.act);
    }
    if (out) {
        if (f.res) z = __fadd_rn(z, load_value(f.res, warp * f.ldr + j, f.res_bf16));
        store_value(f.y, warp * f.ldy + j, f.y_bf16, z);
    }
}

template <int XB, int MT, int RW>
cudaError_t launch_few_rows(const FewArgs &a, cudaStream_t s) {
    using C = FewCfg<XB, MT, RW>;
    if (C::kSmem > 49152) {
        const cudaError_t e = cudaFuncSetAttribute(few_kernel<XB, MT, RW>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(few_kernel<XB, MT, RW>, dim3((a.N + C::kRows - 1) / C::kRows), dim3(kWarps * 32),
                      C::kSmem, s, a);
}

// rows a warp: 4 where the blocks still fill the card
template <int XB, int MT>
cudaError_t launch_few_tokens(const FewArgs &a, int sms, cudaStream_t s) {
    if (a.N >= 32 * sms) return launch_few_rows<XB, MT, 4>(a, s);
    if (a.N >= 16 * sms) return launch_few_rows<XB, MT, 2>(a, s);
    return launch_few_rows<XB, MT, 1>(a, s);
}

template <int XB>
cudaError_t launch_few_bits(const FewArgs &a, int sms, cudaStream_t s) {
    if (a.M == 1) return launch_few_tokens<XB, 1>(a, sms, s);
    if (a.M == 2) return launch_few_tokens<XB, 2>(a, sms, s);
    if (a.M <= 4) return launch_few_tokens<XB, 4>(a, sms, s);
    return launch_few_tokens<XB, 8>(a, sms, s);
}

}  // namespace

cudaError_t launch_few(int xbits, const uint8_t *wp, const float *wsc, int64_t ldws,
                       const uint8_t *xw, const float *xdt, int64_t ldxd, int64_t M, int64_t N,
                       int64_t K, const EpiArgs &fin, int sms, cudaStream_t s) {
    FewArgs a{};
    a.wp = wp;
    a.wsc = wsc;
    a.ldws = ldws;
    a.xw = xw;
    a.xdt = xdt;
    a.ldxd = ldxd;
    a.M = static_cast<int32_t>(M);
    a.N = static_cast<int32_t>(N);
    a.K = static_cast<int32_t>(K);
    a.fin = fin;
    return xbits == 4 ? launch_few_bits<4>(a, sms, s) : launch_few_bits<8>(a, sms, s);
}

}  // namespace h32
