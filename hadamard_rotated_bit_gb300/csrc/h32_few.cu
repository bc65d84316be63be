// The block-scaled product of a few tokens (sm_103a): one new token of each
// sequence through a projection, with the epilogue of h32_finish.cuh.
//
// The definition, the operands and the bits of the tensor-core GEMM
// (h32_gemm_tc.cu): per 32-block the exact sum S from one tcgen05.mma of K = 32, then
// acc = fma(fl(d_w d_x), S, acc) in block order.  That kernel's tiles are 128 weight
// rows wide, and it hands two blocks at a time from the MMA to the epilogue, about
// 300 clocks each however few the columns are: 35 us for 5120 x 5120 and one token.
// With at most 16 tokens a block needs only 16 of TMEM's 512 columns, so here
//   - a hand-off is 8 blocks (128 columns, four buffers: two of 16 blocks
//     leave the hand-off's latency open);
//   - a tile is 128, 64 or 32 weight rows, the most that still gives the card one
//     wave (the MMA always takes 128: the rows beyond the tile's are whatever lies
//     behind it in shared memory, and their results are not read);
//   - a stage is two hand-offs' 512 codes (one's 256 for tiles of 128 rows), brought by four
//     tensor copies: rows and tokens as three-dimensional boxes of 128-byte columns,
//     swizzled as the MMA reads them, and the blocks' scales of both.
//   warps 0..3  epilogue, a TMEM lane quarter each (a tile of 32 rows needs one): the
//               sums of 4 or 8 blocks at a time, the folds on packed pairs of tokens, of
//               which only those in use are read
//   warp 4      TMA producer;  warp 5  TMEM allocator and MMA issuer
// Every wait is bounded.
//
// Bound: HBM, 1.125 bytes a weight, where the tiles fill the card (34816 x 5120, one
// token: 35.6 us, 5.6 TB/s, 84% of the measured copy rate); a narrow projection is
// bound by the pace of one tile's stages, about 0.6 us per 512 codes, most of it the
// hand-offs (5120 x 5120: 12.4 us; 5120 x 17408: 28.2 us, 53%).  The roles that issue
// to the tensor core and the copy engine run as whole warps with one elected lane:
// descriptors in uniform registers, 47 clocks a product less.  (Measured and left:
// sums on CUDA cores in fp16 pairs, 11.8 us for 5120 x 5120 and one token but 66 us
// for 34816 x 5120 and five; mma.m16n8k16 on widened codes, 16 rows a warp, 15-17 us
// and 42-50 us, 47-66 instructions per 512 bytes of weights where this takes about 4.)

// poll without sleeping: the waits here are short and on the critical path
#ifndef H32_WAIT_SLEEP
#define H32_WAIT_SLEEP 0
#endif

#include "h32_few.cuh"
#include "h32_epilogue.cuh"
#include "h32_tmap.cuh"

namespace h32 {
namespace {

__device__ uint32_t g_few_status;   // kStatusTimeout: a bounded wait gave up

constexpr int kGroup = 8;                         // blocks of a hand-off
constexpr int kBufs = 4;                          // hand-offs in TMEM
constexpr int kCols = 16;                         // TMEM columns of a block: the tokens
constexpr int kMaxStages = 12;
constexpr int kWarps = 6;
constexpr int kMaxSmem = 225 * 1024;
constexpr uint64_t kDrainPolls = 1ull << 22;

struct FewArgs {
    int32_t M, N, K, rows, tiles, stages;   // rows of a tile
    uint64_t wait_limit;
    EpiArgs fin;
};

// byte sizes of a stage's parts
struct Sizes {
    uint32_t a, b, sa, sb;
    __host__ __device__ Sizes(int rows, int tokens, int xb, int blocks)
        : a(rows * blocks * 32), b(tokens * blocks * 32 * (xb / 4)), sa(rows * blocks * 4),
          sb(blocks * 16 * 4) {}
    __host__ __device__ uint32_t stage() const { return a + b + sa + sb; }
};

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const void *tmap, uint64_t *bar, int32_t x,
                                            int32_t y, int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// 2 PT consecutive columns of the warp's 32 lanes
template <int PT>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[2 * PT]) {
    if constexpr (PT == 1) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];"
                     : "=r"(r[0]), "=r"(r[1])
                     : "r"(taddr));
    } else if constexpr (PT == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                       "=r"(r[7])
                     : "r"(taddr));
    } else {
        tmem_ld_x16(taddr, r);
    }
}

// XB: activation bits; PT: pairs of tokens folded (2 PT >= M); kStageBlocks: blocks of a
// stage, 16 or 8
template <int XB, int PT, int kStageBlocks>
__global__ void __launch_bounds__(kWarps * 32, 1)
    few_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb,
               const FewArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_sfull[kBufs], s_sempty[kBufs], s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    constexpr int kStageCodes = 32 * kStageBlocks;
    constexpr int kCols128 = kStageCodes / 128;   // 128-byte columns of a stage's weights
    // tokens copied: 8 (the MMA then reads the next column's as tokens 8 .. 15, whose
    // results nobody reads) or 16
    constexpr int kTokens = PT <= 4 ? 8 : 16;
    const Sizes z(a.rows, kTokens, XB, kStageBlocks);
    const int S = a.stages;
    uint8_t *s_a = smem, *s_b = s_a + S * z.a, *s_sa = s_b + S * z.b, *s_sb = s_sa + S * z.sa;
    // (the broadcast tells the compiler that a warp's branch is uniform: the MMA's
    // descriptors then stay in uniform registers)
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int epi_warps = a.rows / 32;
    const int nb = a.K / 32, nst = (a.K + kStageCodes - 1) / kStageCodes;
    const uint64_t lim = a.wait_limit;
    volatile int *abort = &s_abort;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], epi_warps);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&s_sfull[i], 1);
            mbar_init(&s_sempty[i], epi_warps);
        }
        mbar_init(&s_drain, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();
    if (warp == 5) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    auto give_up = [&]() {
        s_abort = 1;
        atomicOr(&g_few_status, kStatusTimeout);
    };

    if (warp == 4) {
        // ------------------------------------------------------------ TMA
        const bool leader = elect_one();
        if (leader) {
            prefetch_tmap(&map_a);
            prefetch_tmap(&map_b);
            prefetch_tmap(&map_sa);
            prefetch_tmap(&map_sb);
        }
        int s = 0, fed = 0;   // the stage; stages fed so far, at most S
        uint32_t ph = 1;      // (the first round's waits pass at once)
        bool ok = true;
        for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
            for (int st = 0; st < nst; ++st) {
                if (!warp_wait_or_look(&s_empty[s], ph, lim, abort)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    mbar_arrive_expect_tx(&s_full[s], z.stage());
                    tma_load_3d(s_a + s * z.a, &map_a, &s_full[s], 0, t * a.rows, kCols128 * st);
                    tma_load_3d(s_b + s * z.b, &map_b, &s_full[s], 0, 0, kCols128 * (XB / 4) * st);
                    tma_load_2d(s_sa + s * z.sa, &map_sa, &s_full[s], kStageBlocks * st, t * a.rows);
                    tma_load_2d(s_sb + s * z.sb, &map_sb, &s_full[s], 0, kStageBlocks * st);
                }
                __syncwarp();
                if (fed < S) ++fed;
                if (++s == S) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
        if (leader) {
            if (!ok) give_up();
            // leave only when the copies under way have landed (at once unless a wait
            // gave up): each fed stage's last phase
            for (int i = 0; i < fed; ++i) {
                if (--s < 0) {
                    s = S - 1;
                    ph ^= 1;
                }
                mbar_wait_bounded(&s_full[s], ph ^ 1, kDrainPolls, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------------ MMA
        {
            const bool leader = elect_one();
            const uint32_t idesc = idesc_e4m3_f32(128, kCols);
            const uint64_t da0 = smem_desc_sw128(smem_u32(s_a)), db0 = smem_desc_sw128(smem_u32(s_b));
            const uint32_t a_step = z.a >> 4, b_step = z.b >> 4, a_col = a.rows * 128 >> 4;
            int s = 0, gb = 0;
            uint32_t ph = 0, gph = 1;
            bool ok = true;
            for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
                for (int st = 0; st < nst; ++st) {
                    if (!warp_wait_or_look(&s_full[s], ph, lim, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t da = da0 + s * a_step, db = db0 + s * b_step;
                    const int n = nb - st * kStageBlocks;   // blocks left: a multiple of 4
#pragma unroll
                    for (int j0 = 0; j0 < kStageBlocks; j0 += kGroup) {
                        if (j0 < n) {
                            if (!warp_wait_or_look(&s_sempty[gb], gph, lim, abort)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                            if (leader) {
#pragma unroll
                                for (int i = 0; i < kGroup; ++i) {
                                    const int j = j0 + i;
                                    if ((j & ~3) < n) {
                                        const uint64_t daj = da + (j >> 2) * a_col + (j & 3) * 2;
                                        const uint32_t slot = tmem + (gb * kGroup + i) * kCols;
                                        if constexpr (XB == 4) {
                                            mma_f8f6f4(slot, daj, db + (((j >> 2) * kTokens * 128 + (j & 3) * 32) >> 4),
                                                       idesc, 0);
                                        } else {
                                            // the 16 h, then the l, into one sum
                                            const uint64_t dbj = db + (((j >> 1) * kTokens * 128 + (j & 1) * 64) >> 4);
                                            mma_f8f6f4(slot, daj, dbj, idesc, 0);
                                            mma_f8f6f4(slot, daj, dbj + (32 >> 4), idesc, 1);
                                        }
                                    }
                                }
                                mma_commit(&s_sfull[gb]);
                            }
                            __syncwarp();
                            if (++gb == kBufs) {
                                gb = 0;
                                gph ^= 1;
                            }
                        }
                    }
                    if (!ok) break;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            if (leader) {
                if (!ok) give_up();
                mma_commit(&s_drain);
                mbar_wait_bounded(&s_drain, 0, kDrainPolls, nullptr);
            }
            __syncwarp();
        }
    } else if (warp < epi_warps) {
        // ------------------------------------------------------- epilogue
        // kBatch blocks' sums a load (measured: loads of the next batch under way while
        // one is folded made every case 30-80% slower)
        constexpr int kBatch = PT == 1 ? 8 : 4;
        static_assert(kGroup % kBatch == 0 && kStageBlocks % kGroup == 0, "batches within hand-offs");
        const int row = warp * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
        const EpiArgs &f = a.fin;
        int s = 0, gb = 0;
        uint32_t sph = 0, gph = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
            uint64_t acc[PT];
#pragma unroll
            for (int p = 0; p < PT; ++p) acc[p] = 0ull;
            for (int st = 0; st < nst && ok; ++st) {
                if (!warp_wait_or_look(&s_full[s], sph, lim, abort)) {
                    ok = false;
                    break;
                }
                const float *dw = reinterpret_cast<const float *>(s_sa + s * z.sa) + row * kStageBlocks;
                const float *dx = reinterpret_cast<const float *>(s_sb + s * z.sb);
                const int n = nb - st * kStageBlocks;   // blocks left: a multiple of 4
#pragma unroll
                for (int j0 = 0; j0 < kStageBlocks; j0 += kBatch) {
                    if (j0 < n) {
                        if (j0 % kGroup == 0) {
                            if (!warp_wait_or_look(&s_sfull[gb], gph, lim, abort)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
                        }
                        const uint32_t tcol = tmem + lane_addr + (gb * kGroup + j0 % kGroup) * kCols;
                        uint32_t v[kBatch][2 * PT];
#pragma unroll
                        for (int j = 0; j < kBatch; ++j) tmem_ld<PT>(tcol + j * kCols, v[j]);
                        tmem_ld_wait();
                        if (j0 % kGroup == kGroup - kBatch || j0 + kBatch >= n) {
                            // the hand-off's sums are in registers
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&s_sempty[gb]);
                            if (++gb == kBufs) {
                                gb = 0;
                                gph ^= 1;
                            }
                        }
#pragma unroll
                        for (int q = 0; q < kBatch; q += 4) {
                            if (q == 0 || j0 + q < n) {
                                const float4 d = *reinterpret_cast<const float4 *>(dw + j0 + q);
                                const float ds[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const uint32_t w = __float_as_uint(ds[j]);
                                    const uint64_t w2 = pair_of(w, w);
                                    const uint64_t *x = reinterpret_cast<const uint64_t *>(dx + (j0 + q + j) * 16);
#pragma unroll
                                    for (int p = 0; p < PT; ++p)
                                        acc[p] = fma_f32x2(mul_f32x2(w2, x[p]),
                                                           pair_of(v[q + j][2 * p], v[q + j][2 * p + 1]), acc[p]);
                                }
                            }
                        }
                    }
                }
                // (the products that read the stage are done: their sums were waited for)
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[s]);
                if (++s == S) {
                    s = 0;
                    sph ^= 1;
                }
            }
            if (!ok) break;
            // bias, activation, residual
            const int n = t * a.rows + row;
            const bool in = n < a.N;
            const float bias = (f.bias && in) ? __ldg(f.bias + n) : 0.0f;
            float y[2 * PT];
#pragma unroll
            for (int p = 0; p < PT; ++p) {
                y[2 * p] = __uint_as_float(static_cast<uint32_t>(acc[p]));
                y[2 * p + 1] = __uint_as_float(static_cast<uint32_t>(acc[p] >> 32));
            }
            if (f.bias) {
#pragma unroll
                for (int m = 0; m < 2 * PT; ++m) y[m] = __fadd_rn(y[m], bias);
            }
            if (f.act == H32_EPI_SWIGLU) {
                // gate and up rows are adjacent lanes
#pragma unroll
                for (int m = 0; m < 2 * PT; ++m) y[m] = swiglu(y[m], __shfl_xor_sync(0xFFFFFFFFu, y[m], 1));
                if (in && !(lane & 1)) finish_columns<2 * PT>(f, y, 0, 0, a.M, n >> 1);
            } else {
#pragma unroll
                for (int m = 0; m < 2 * PT; ++m) y[m] = activate(y[m], f.act);
                if (in) finish_columns<2 * PT>(f, y, 0, 0, a.M, n);
            }
        }
        if (!ok && lane == 0) give_up();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// rows of `row_bytes` as [row_bytes / 128][rows][128 bytes], boxes of `box_rows` rows
// and `box_cols` 128-byte columns, 128B-swizzled
bool code_map(CUtensorMap *map, const void *base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows,
              uint32_t box_cols) {
    const cuuint64_t dims[3] = {128, rows, row_bytes / 128}, strides[2] = {row_bytes, 128};
    const cuuint32_t box[3] = {128, box_rows, box_cols}, estr[3] = {1, 1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box,
                     estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool scale_map(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer, uint32_t box_inner,
               uint32_t box_outer) {
    const cuuint64_t dims[2] = {inner, outer}, strides[1] = {inner * 4};
    const cuuint32_t box[2] = {box_inner, box_outer}, estr[2] = {1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), dims, strides, box,
                     estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int XB, int PT, int kStageBlocks>
h32_status launch_few_kernel(const CUtensorMap *maps, const FewArgs &a, int grid, int smem,
                             cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(few_kernel<XB, PT, kStageBlocks>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess)
        e = launch_pdl(few_kernel<XB, PT, kStageBlocks>, dim3(grid), dim3(kWarps * 32), smem, s, maps[0],
                       maps[1], maps[2], maps[3], a);
    return launch_status(e != cudaSuccess ? e : cudaGetLastError());
}

template <int XB, int PT>
h32_status launch_few_pairs(const CUtensorMap *maps, const FewArgs &a, int blocks, int grid, int smem,
                            cudaStream_t s) {
    return blocks == 16 ? launch_few_kernel<XB, PT, 16>(maps, a, grid, smem, s)
                        : launch_few_kernel<XB, PT, 8>(maps, a, grid, smem, s);
}

}  // namespace

h32_status launch_few(int xbits, const uint8_t *wp, const float *wsc, int64_t ldws,
                      const uint8_t *xw, const float *xdt, int64_t ldxd, int64_t M, int64_t N,
                      int64_t K, const EpiArgs &fin, int sms, cudaStream_t s) {
    FewArgs a{};
    a.M = static_cast<int32_t>(M);
    a.N = static_cast<int32_t>(N);
    a.K = static_cast<int32_t>(K);
    // the widest tile that still is one wave of at least half the SMs
    a.rows = N > 128 * sms / 2 ? 128 : N > 64 * sms / 2 ? 64 : 32;
    a.tiles = static_cast<int32_t>((N + a.rows - 1) / a.rows);
    a.wait_limit = wait_limit();
    a.fin = fin;
    // longer stages for the narrow tiles, whose pace the barriers between the warps set;
    // of 128 rows more short ones fit
    const int blocks = a.rows == 128 ? 8 : 16;
    const uint32_t tokens = M <= 8 ? 8 : 16;
    const Sizes z(a.rows, tokens, xbits, blocks);
    // (the MMA reads 128 rows from every column of a stage's weights: what lies behind
    // the last one, at most 12 KB, is the tokens' and the scales' stages)
    const int fit = (kMaxSmem - 1024) / static_cast<int>(z.stage());
    a.stages = fit < kMaxStages ? fit : kMaxStages;
    const int smem = a.stages * static_cast<int>(z.stage()) + 1024;
    if (!tensor_map_encoder()) {
        note_error("cuTensorMapEncodeTiled is not available from the driver");
        return H32_ERR_CUDA;
    }
    const uint64_t xrow = K * (xbits / 4);
    CUtensorMap maps[4];
    if (!code_map(&maps[0], wp, K, N, a.rows, blocks / 4) ||
        !code_map(&maps[1], xw, xrow, M, tokens, blocks / 4 * (xbits / 4)) ||
        !scale_map(&maps[2], wsc, ldws, N, blocks, a.rows) ||
        !scale_map(&maps[3], xdt, ldxd, K / 32, 16, blocks)) {
        note_error("cuTensorMapEncodeTiled rejected a tensor map of the few-token product");
        return H32_ERR_CUDA;
    }
    const int grid = a.tiles < sms ? a.tiles : sms;
    if (xbits == 4) {
        if (M <= 2) return launch_few_pairs<4, 1>(maps, a, blocks, grid, smem, s);
        if (M <= 8) return launch_few_pairs<4, 4>(maps, a, blocks, grid, smem, s);
        return launch_few_pairs<4, 8>(maps, a, blocks, grid, smem, s);
    }
    if (M <= 2) return launch_few_pairs<8, 1>(maps, a, blocks, grid, smem, s);
    if (M <= 8) return launch_few_pairs<8, 4>(maps, a, blocks, grid, smem, s);
    return launch_few_pairs<8, 8>(maps, a, blocks, grid, smem, s);
}

__device__ uint32_t g_few_status_taken;
__global__ void take_g_few_status() { g_few_status_taken = atomicExch(&g_few_status, 0u); }

h32_status few_read_and_clear_status(cudaStream_t s) {
    bool ok = false;
    const uint32_t v = take_status(take_g_few_status, g_few_status_taken, s, &ok);
    if (!ok) return H32_ERR_CUDA;
    return (v & kStatusTimeout) ? H32_ERR_TIMEOUT : H32_OK;
}

}  // namespace h32
