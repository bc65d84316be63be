// Products of e4m3 codes with a scale for each block of 128 (sm_103a):
//   y[m][n] = sum over b of fl(dx[b][m] dw[n / 128][b]) S_b,
//   S_b = the sum over block b's 128 codes of xq[m][k] wq[n][k], in fp32 by the tensor core,
// folded in block order by one fp32 fma each, and rounded once to y's type.
//
// One block is one 128-byte K step: four tcgen05.mma (kind::f8f6f4, K = 32) give S for a
// tile in TMEM, the epilogue warps read it back and fold it into registers while the
// tensor core does the next one.
//
// rows_kernel, for a few tokens (or few tiles of a long K): weight rows on the TMEM lanes, NC tokens as
//   its columns.
//   A tile is 128 weight rows (one block of scales: d_w is uniform) x NC tokens; with few
//   tiles a cluster of CTAs shares its K steps out and adds up through shared memory.
//   warps 0..3  epilogue, a lane quarter each
//   warp 4      TMA producer: per K step the rows' and the tokens' codes and the tokens' scales
//   warp 5      TMEM allocator and MMA issuer
//   Bound: HBM, a byte a weight (131072 x 5120, one token: 108 us, 6.2 TB/s, 91% of the measured
//   copy rate); a narrow projection by launch and the steps' latency (5120 x 5120, 7 tokens:
//   9.4 us).
//
// lanes_kernel, for more: tokens on the lanes, so that a scale is one number a thread and K
//   step; 128 tokens and one CTA, or 256 and a pair (cta_group::2), x 64, 128 or 256 weight rows.
//   warps 0..7  epilogue: a lane quarter and half of the columns each
//   warp 8      TMA producer
//   warp 9      TMEM allocator; in the first CTA MMA issuer
//   Bound: of the 420 to 480 ns of a pair's K step (256 x 256 x 128; the clock depends on the power
//   the codes draw) the tensor core needs 270; the rest is the way from its last product to the
//   epilogue and back, which two buffers of 256 columns (all of TMEM) do not hide.  4096 x 34816 x
//   5120: 508 to 525 us, 2780 to 2870 TFLOP/s (back to back for more than half a second 563 to 575).
//   (Measured and left, in an earlier form: four buffers of 128 columns, 913 us for 555, as four
//   dependent products of 128 columns take 350 clocks instead of 256; 16 epilogue warps, scales
//   multiplied ahead of their step, scalar folds, and loads of sums two at a time, each 5 to 100%
//   slower; arrivals across the pair with release, twice the time; the outputs' stores are 5% of it,
//   the first weight scales of a tile under 1%.)
// Every wait is bounded.
#include "h32_f8.cuh"

#include "h32_epilogue.cuh"
#include "h32_f8_plan.h"

namespace h32 {
namespace {

__device__ uint32_t g_f8_status;   // kStatusTimeout, kStatusGuard

constexpr int kMaxStages = 12;
constexpr int kRowsWarps = 6;
// lanes_kernel: two epilogue warps for each quarter of the lanes, and a warpgroup of the roles
// that issue.  Of 12 warps with 168 registers at launch the epilogue's two warpgroups take over
// what that one does not need.  (The shares and the unrolling of the K steps are those that
// leave every instance without spills: a few spilled words cost it 12 to 30%.)
constexpr int kPairWarps = 12, kPairRegs = 168;
constexpr __host__ __device__ int issue_regs(int ctas) { return ctas == 2 ? 104 : 120; }
constexpr __host__ __device__ int epilogue_regs(int ctas) { return ctas == 2 ? 200 : 192; }
static_assert(128 * issue_regs(1) + 256 * epilogue_regs(1) <= kPairWarps * 32 * kPairRegs &&
                  128 * issue_regs(2) + 256 * epilogue_regs(2) <= kPairWarps * 32 * kPairRegs,
              "registers handed over");
constexpr int kMaxSmem = 225 * 1024;
constexpr uint64_t kDrainPolls = 1ull << 22;

struct F8Args {
    int32_t M, N, K;         // token rows, weight rows (of an expert), reduction length
    int32_t E;               // experts; 1 and off null: all rows
    int32_t stages;          // rows_kernel
    int32_t cluster;         // rows_kernel: CTAs of a tile
    uint8_t *ws;             // lanes_kernel: partial sums and flags of split tiles, or null
    const int32_t *off;      // [E + 1] or null
    const float *wd;         // [E][ceil(N / 128)][ceil(K / 128)]
    const float *xd;         // [ceil(K / 128)][ldxd]
    int64_t ldxd;
    void *y;
    int64_t ldy;
    uint8_t y_bf16, y_vec;   // y_vec: every row of y starts on 16 bytes
    uint64_t wait_limit;
};

// The groups of token rows: their offsets and the first tile of each, tiles numbered
// group-major, then by weight tile, then by chunk of tokens.  A group's chunks start at
// its first row rounded down to a multiple of 4 (the scales' copies start on 16 bytes);
// the rows of a chunk outside the group are computed and not stored.
struct Groups {
    int *off, *first;   // [E + 1] each
    static constexpr __host__ __device__ size_t bytes(int E) { return (2 * size_t(E + 1) * 4 + 1023) / 1024 * 1024; }
    __device__ int chunks(int e, int cols) const {
        const int lo = off[e], hi = off[e + 1];
        return hi > lo ? (hi - (lo & ~3) + cols - 1) / cols : 0;
    }
};

struct Tile {
    int e, n0, g0, clo, chi;   // expert, first weight row in it, first token row, its columns in use
};

__device__ __forceinline__ Tile tile_of(int t, const Groups &g, int E, int cols, int rows) {
    int lo = 0, hi = E;   // the last group whose first tile is <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.first[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    Tile r;
    r.e = lo;
    const int local = t - g.first[lo], chunks = g.chunks(lo, cols), wt = local / chunks;
    r.n0 = wt * rows;
    r.g0 = (g.off[lo] & ~3) + (local - wt * chunks) * cols;
    r.clo = max(0, g.off[lo] - r.g0);
    r.chi = min(cols, g.off[lo + 1] - r.g0);
    return r;
}

// Reads and checks the offsets (0 = off[0] <= ... <= off[E] = M) and numbers the tiles.
// Every thread of the CTA calls it; returns the number of tiles, -1 where the offsets
// are none.
__device__ int load_groups(const Groups &g, const F8Args &a, int cols, int weight_tiles, int *s_word) {
    const int tid = threadIdx.x, E = a.E;
    if (tid == 0) *s_word = 0;
    for (int i = tid; i <= E; i += blockDim.x) g.off[i] = a.off ? a.off[i] : i * a.M;
    __syncthreads();
    for (int i = tid; i <= E; i += blockDim.x) {
        const int v = g.off[i];
        if ((i == 0 && v != 0) || (i == E && v != a.M) || (i < E && g.off[i + 1] < v)) *s_word = 1;
    }
    __syncthreads();
    const bool bad = *s_word != 0;
    if (tid < 32 && !bad) {
        const int per = (E + 31) / 32, e0 = tid * per;
        int sum = 0;
        for (int i = e0; i < min(e0 + per, E); ++i) sum += weight_tiles * g.chunks(i, cols);
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (tid >= o) incl += v;
        }
        int run = incl - sum;
        for (int i = e0; i < min(e0 + per, E); ++i) {
            g.first[i] = run;
            run += weight_tiles * g.chunks(i, cols);
        }
        if (tid == 31) g.first[E] = incl;
    }
    __syncthreads();
    return bad ? -1 : g.first[E];
}

__device__ __forceinline__ void store_y(const F8Args &a, int64_t m, int n, float v) {
    if (a.y_bf16) static_cast<__nv_bfloat16 *>(a.y)[m * a.ldy + n] = __float2bfloat16_rn(v);
    else static_cast<float *>(a.y)[m * a.ldy + n] = v;
}

// A warp's 32 x 32 outputs (lane = token row m0 + lane, columns n ..), turned around in its
// 4 KB of shared memory so that each store covers whole 128-byte lines: a lane's own row
// a store made the tile's end twice as long.  16-byte pieces, piece p of row r at
// p ^ (r & 7): no bank conflicts either way.  Rows outside [lo, hi) of the tile (r0: the
// warp's first) and columns behind N are left out.  bf16: `fill` 0 stages the left half
// of a line, 1 the right one and stores (`last`: stores what there is).
__device__ __forceinline__ void stage_row(uint8_t *buf, int lane, bool bf16, int fill, const uint64_t (&acc)[16]) {
    const auto value = [&](int i) {
        return __uint_as_float(static_cast<uint32_t>(i & 1 ? acc[i / 2] >> 32 : acc[i / 2]));
    };
    uint4 *row = reinterpret_cast<uint4 *>(buf + lane * 128);
    if (bf16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(value(8 * q + 2 * i), value(8 * q + 2 * i + 1));
                w[i] = reinterpret_cast<const uint32_t &>(b);
            }
            row[(4 * fill + q) ^ (lane & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
            row[q ^ (lane & 7)] = make_uint4(__float_as_uint(value(4 * q)), __float_as_uint(value(4 * q + 1)),
                                             __float_as_uint(value(4 * q + 2)), __float_as_uint(value(4 * q + 3)));
    }
}
// the staged lines: `bytes` of each (64 or 128), from column n on
__device__ __forceinline__ void store_lines(const F8Args &a, const uint8_t *buf, int lane, int64_t m0, int r0, int lo,
                                            int hi, int n, int bytes) {
    const int es = a.y_bf16 ? 2 : 4;
    uint8_t *y = static_cast<uint8_t *>(a.y) + (m0 * a.ldy + n) * es;
    if (a.y_vec && n + bytes / es <= a.N) {
        const int p = lane & 7;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3);
            if (r0 + r >= lo && r0 + r < hi && 16 * p < bytes)
                *reinterpret_cast<uint4 *>(y + r * a.ldy * es + 16 * p) =
                    *reinterpret_cast<const uint4 *>(buf + r * 128 + ((p ^ (r & 7)) << 4));
        }
    } else {
        // rows that start anywhere (N odd), or the last columns: a value a lane, a row of 32 or
        // 64 columns a store (330 x 36226 x 96 fp32: 26 us, row by row without unrolling 69)
        const int cols = min(bytes / es, a.N - n);
        const int at = lane * es, rest = at & 15;
#pragma unroll 4
        for (int r = 0; r < 32; ++r) {
            const bool in = r0 + r >= lo && r0 + r < hi;
            const uint8_t *v = buf + r * 128 + rest;
            if (es == 4) {
                if (in && lane < cols)
                    reinterpret_cast<uint32_t *>(y)[lane] = *reinterpret_cast<const uint32_t *>(v + (((at >> 4) ^ (r & 7)) << 4));
            } else {
                if (in && lane < cols)
                    reinterpret_cast<uint16_t *>(y)[lane] = *reinterpret_cast<const uint16_t *>(v + (((at >> 4) ^ (r & 7)) << 4));
                if (in && lane + 32 < cols)
                    reinterpret_cast<uint16_t *>(y)[lane + 32] =
                        *reinterpret_cast<const uint16_t *>(v + (((at >> 4) + 4 ^ (r & 7)) << 4));
            }
            y += a.ldy * es;
        }
    }
}

// ----------------------------------------------------------------------------
// weight rows on the lanes
// ----------------------------------------------------------------------------
// the position and phase of a role that walks a ring of barriers
struct Ring {
    int i = 0;
    uint32_t ph;
    __device__ explicit Ring(uint32_t phase) : ph(phase) {}
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            ph ^= 1;
        }
    }
};

// With fewer tiles than SMs the K steps of a tile are dealt to the CTAs of a cluster
// (consecutive shares), and each CTA takes a slice of its columns at the end: the others'
// partial sums come to its shared memory and are added in the order of the shares.
template <int NC>
struct Rows {
    static constexpr int kBufs = 8;                           // sums in TMEM
    static constexpr uint32_t kTmem = kBufs * NC;
    static constexpr uint32_t kA = 128 * 128, kB = NC * 128;  // bytes of a stage's parts
    static constexpr uint32_t kS = NC * 4 < 128 ? 128 : NC * 4;
    static constexpr uint32_t kStage = kA + kB + kS;
    // the partial sums that a CTA gets: [share][column][row]
    static __host__ __device__ uint32_t parts(int cluster) { return (cluster - 1) * (NC / cluster) * 512; }
};

template <int NC>
__global__ void __launch_bounds__(kRowsWarps * 32, kRowsPerSm)
    rows_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                const __grid_constant__ CUtensorMap map_s, const F8Args a) {
    using C = Rows<NC>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // s_full: a stage's copies; s_empty: its products are done and its scales read; s_sum: a K
    // step's sums are in TMEM; s_free: they are in registers; s_part: the other CTAs' partial
    // sums are here
    __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages], s_sum[C::kBufs], s_free[C::kBufs], s_part, s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_word;
    __shared__ volatile int s_abort;
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int S = a.stages, cluster = a.cluster;
    const int slice = NC / cluster, slice_bits = 31 - __clz(slice);   // columns of a CTA: a power of 2
    const uint32_t rank = cluster > 1 ? cluster_rank() : 0;
    uint8_t *s_a = smem, *s_b = s_a + S * C::kA, *s_s = s_b + S * C::kB;
    float *s_parts = reinterpret_cast<float *>(s_s + S * C::kS);
    int *s_table = reinterpret_cast<int *>(s_s + S * C::kS + C::parts(cluster));
    const Groups g{s_table, s_table + a.E + 1};
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int nb = (a.K + 127) / 128, nt = (a.N + 127) / 128;
    // this CTA's K steps
    const int kb0 = nb * static_cast<int>(rank) / cluster, steps = nb * (static_cast<int>(rank) + 1) / cluster - kb0;
    const int first = blockIdx.x / cluster, stride = gridDim.x / cluster;
    const uint64_t lim = a.wait_limit;
    volatile int *abort = &s_abort;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 4);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(&s_sum[i], 1);
            mbar_init(&s_free[i], 4);
        }
        mbar_init(&s_part, cluster > 1 ? 4 * (cluster - 1) : 1);
        mbar_init(&s_drain, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if (warp == 5) {
        tmem_alloc(&s_tmem, C::kTmem);
        tmem_relinquish();
    }
    if (cluster > 1) cluster_sync();   // every CTA runs, and its barriers are there
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    int total = load_groups(g, a, NC, nt, &s_word);
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    if (total < 0) {
        if (threadIdx.x == 0) atomicOr(&g_f8_status, kStatusGuard);
        total = 0;
    }
    auto give_up = [&]() {
        s_abort = 1;
        atomicOr(&g_f8_status, kStatusTimeout);
    };

    if (warp == 4) {
        // ------------------------------------------------------------ TMA
        const bool leader = elect_one();
        if (leader) {
            prefetch_tmap(&map_w);
            prefetch_tmap(&map_x);
            prefetch_tmap(&map_s);
        }
        Ring st(1);   // (the first round's waits pass at once)
        int fed = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += stride) {
            const Tile ti = tile_of(t, g, a.E, NC, 128);
            for (int i = 0; i < steps; ++i) {
                if (!warp_wait_or_look(&s_empty[st.i], st.ph, lim, abort)) {
                    ok = false;
                    break;
                }
                if (leader) {
                    const int kb = kb0 + i;
                    mbar_arrive_expect_tx(&s_full[st.i], C::kA + C::kB + NC * 4);
                    tma_load_2d(s_a + st.i * C::kA, &map_w, &s_full[st.i], kb * 128, ti.e * a.N + ti.n0);
                    tma_load_2d(s_b + st.i * C::kB, &map_x, &s_full[st.i], kb * 128, ti.g0);
                    tma_load_2d(s_s + st.i * C::kS, &map_s, &s_full[st.i], ti.g0, kb);
                }
                __syncwarp();
                if (fed < S) ++fed;
                st.next(S);
            }
        }
        if (leader) {
            if (!ok) give_up();
            // leave only when the copies under way have landed (at once unless a wait
            // gave up): each fed stage's last phase
            for (int i = 0; i < fed; ++i) {
                if (--st.i < 0) {
                    st.i = S - 1;
                    st.ph ^= 1;
                }
                mbar_wait_bounded(&s_full[st.i], st.ph ^ 1, kDrainPolls, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 5) {
        // ------------------------------------------------------------ MMA
        const bool leader = elect_one();
        const uint32_t idesc = idesc_e4m3_f32(128, NC);
        const uint64_t da0 = smem_desc_sw128(smem_u32(s_a)), db0 = smem_desc_sw128(smem_u32(s_b));
        Ring st(0), bf(1);
        bool ok = true;
        for (int t = first; t < total && ok; t += stride) {
            for (int i = 0; i < steps; ++i) {
                if (!warp_wait_or_look(&s_full[st.i], st.ph, lim, abort) ||
                    !warp_wait_or_look(&s_free[bf.i], bf.ph, lim, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (leader) {
                    // (columns behind K are zeros in both operands)
                    const uint64_t da = da0 + st.i * (C::kA >> 4), db = db0 + st.i * (C::kB >> 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f8f6f4(tmem + bf.i * NC, da + 2 * j, db + 2 * j, idesc, j > 0);
                    mma_commit(&s_sum[bf.i]);
                }
                __syncwarp();
                st.next(S);
                bf.next(C::kBufs);
            }
        }
        if (leader) {
            if (!ok) give_up();
            mma_commit(&s_drain);
            mbar_wait_bounded(&s_drain, 0, kDrainPolls, nullptr);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------- epilogue
        const int row = warp * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
        Ring st(0), bf(0);
        bool ok = true;
        for (int t = first; t < total && ok; t += stride) {
            const Tile ti = tile_of(t, g, a.E, NC, 128);
            uint64_t acc[NC / 2];
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
            // the tile's weight scales, a lane's share of 32 steps ahead
            const float *wd = a.wd + (int64_t(ti.e) * nt + ti.n0 / 128) * nb + kb0;
            float dw_next = lane < steps ? __ldg(wd + lane) : 0.0f, dw_lane = 0.0f;
            for (int i = 0; i < steps; ++i) {
                if ((i & 31) == 0) {
                    dw_lane = dw_next;
                    dw_next = i + 32 + lane < steps ? __ldg(wd + i + 32 + lane) : 0.0f;
                }
                const float dw = __shfl_sync(0xFFFFFFFFu, dw_lane, i & 31);
                // (the stage's scales; its codes' sums follow)
                if (!warp_wait_or_look(&s_full[st.i], st.ph, lim, abort) ||
                    !warp_wait_or_look(&s_sum[bf.i], bf.ph, lim, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float *dx = reinterpret_cast<const float *>(s_s + st.i * C::kS);
                const uint32_t col = tmem + lane_addr + bf.i * NC;
                if constexpr (NC == 16) {
                    uint32_t v[16];
                    tmem_ld_x16(col, v);
                    tmem_ld_wait();
                    fold16(acc, dw, dx, v);
                } else {
                    uint32_t v[32];
                    tmem_ld_x32(col, v);
                    tmem_wait_for(v);
                    fold16(acc, dw, dx, reinterpret_cast<const uint32_t(&)[16]>(v[0]));
                    fold16(acc + 8, dw, dx + 16, reinterpret_cast<const uint32_t(&)[16]>(v[16]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s_free[bf.i]);
                    mbar_arrive(&s_empty[st.i]);
                }
                st.next(S);
                bf.next(C::kBufs);
            }
            if (!ok) break;
            const int n = ti.n0 + row;
            const auto value = [&](int c) {
                return __uint_as_float(static_cast<uint32_t>(c & 1 ? acc[c / 2] >> 32 : acc[c / 2]));
            };
            if (cluster == 1) {
#pragma unroll
                for (int c = 0; c < NC; ++c)
                    if (n < a.N && c >= ti.clo && c < ti.chi) store_y(a, ti.g0 + c, n, value(c));
                continue;
            }
            // (one tile a cluster.)  The other slices over, share p's sums of slice q to slot p
            // (p < q) or p - 1 (p > q) of CTA q; then this CTA's added up
            int share = static_cast<int>(rank);
            asm volatile("" : "+r"(share));   // (the addresses are made here, not kept over the steps)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const int q = c >> slice_bits;
                if (q != share)
                    peer_store(peer_smem(s_parts + ((share < q ? share : share - 1) * slice + (c & (slice - 1))) * 128 + row, q),
                               value(c));
            }
            __syncwarp();
            if (lane < cluster && lane != share) peer_arrive_release(peer_smem(&s_part, lane));
            if (!warp_wait_cluster(&s_part, 0, lim, abort)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (c >> slice_bits == share) {
                    const float *slot = s_parts + (c & (slice - 1)) * 128 + row;
                    float y = share == 0 ? value(c) : slot[0];
                    for (int p = 1; p < cluster; ++p)
                        y = __fadd_rn(y, p == share ? value(c) : slot[(p < share ? p : p - 1) * slice * 128]);
                    if (n < a.N && c >= ti.clo && c < ti.chi) store_y(a, ti.g0 + c, n, y);
                }
            }
        }
        if (!ok && lane == 0) give_up();
    }
    tc_fence_before();
    if (cluster > 1) cluster_sync();   // nothing of any CTA reaches into another any more
    else __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// ----------------------------------------------------------------------------
// token rows on the lanes, 128 to each of a tile's one or two CTAs
// ----------------------------------------------------------------------------
template <int kChunks, int kCtas>
struct Lanes {
    static constexpr int kBn = 64 * kChunks;             // weight rows of a tile
    static constexpr uint32_t kA = 128 * 128, kB = kBn / kCtas * 128;   // a CTA's codes of a stage
    static constexpr uint32_t kRest = Groups::bytes(kMaxExperts) + 1024 + 8 * 4096;
    static constexpr int kFit = (kMaxSmem - kRest) / (kA + kB);
    static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
    static constexpr uint32_t kSmem = kStages * (kA + kB) + kRest;
};

// A pair's work, as (tile, K steps): whole tiles in turn, or (kSplit) an equal run of all tiles'
// steps, last piece first.  A tile may be in several pairs' runs: the pair with its last steps
// adds the others' partial sums, all of pairs before it, to its own in those pairs' order.  They come
// from those pairs' first pieces, and it needs them for its last one.
template <bool kSplit, int kCtas>
struct Walk {
    int t, k0, k1;   // the piece: steps [k0, k1) of tile t
    // the first step of pair p's run, of `all` steps
    static __device__ __forceinline__ int64_t run(int64_t all, int p) { return all * p / (gridDim.x / kCtas); }
    __device__ __forceinline__ Walk(int total, int nb) {
        const int pair = blockIdx.x / kCtas;
        if constexpr (kSplit) {
            const int64_t all = int64_t(total) * nb, end = run(all, pair + 1);
            left = static_cast<int>(end - run(all, pair));
            t = static_cast<int>((end - 1) / nb) + 1;
            k0 = 0;
            last = static_cast<int>(end - int64_t(t - 1) * nb);
        } else {
            t = pair - static_cast<int>(gridDim.x / kCtas);
        }
    }
    __device__ __forceinline__ bool next(int total, int nb) {
        if constexpr (kSplit) {
            if (left == 0) return false;
            --t;
            k1 = last;
            last = nb;
            k0 = max(0, k1 - left);
            left -= k1 - k0;
            return true;
        }
        t += gridDim.x / kCtas;
        k0 = 0;
        k1 = nb;
        return t < total;
    }

private:
    int left, last;   // steps of the run still to come, and where the next piece ends
};

// Partial sums of a pair: a CTA's 8 epilogue warps, 32 pieces of 16 bytes a lane.  Behind all of
// them a flag for each warp, set when its sums are written.
struct Partials {
    static constexpr size_t kPair = 2 * 8 * 32 * 32 * 16;
    static __host__ __device__ size_t flags(int pairs) { return size_t(pairs) * 16 * 4; }
    static __host__ __device__ size_t bytes(int pairs) { return pairs * kPair + flags(pairs); }
    uint8_t *ws;
    int pairs, warp;   // the warp's place in its pair, 0 .. 15
    // piece i, four sums (volatile: one after another, not all held at once)
    __device__ __forceinline__ uint8_t *piece(int pair, int i) const {
        return ws + pair * kPair + ((warp * 32 + i) * 32 + (threadIdx.x & 31)) * 16;
    }
    __device__ __forceinline__ void put(int pair, int i, uint64_t lo, uint64_t hi) const {
        asm volatile("st.global.cg.v2.b64 [%0], {%1, %2};" ::"l"(piece(pair, i)), "l"(lo), "l"(hi) : "memory");
    }
    __device__ __forceinline__ void get(int pair, int i, uint64_t &lo, uint64_t &hi) const {
        asm volatile("ld.global.cg.v2.b64 {%0, %1}, [%2];" : "=l"(lo), "=l"(hi) : "l"(piece(pair, i)) : "memory");
    }
    __device__ uint32_t *flag(int pair) const {
        return reinterpret_cast<uint32_t *>(ws + pairs * kPair) + pair * 16 + warp;
    }
    __device__ void publish(int pair) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            __threadfence();
            asm volatile("st.release.gpu.global.u32 [%0], 1;" ::"l"(flag(pair)) : "memory");
        }
        __syncwarp();
    }
    __device__ bool wait(int pair, uint64_t limit, volatile int *abort) const {
        bool ok = false;
        if ((threadIdx.x & 31) == 0)
            for (uint64_t i = 0; i < limit && !ok; ++i) {
                uint32_t v;
                asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag(pair)) : "memory");
                ok = v != 0;
                if (!ok && *abort) break;
            }
        __syncwarp();   // (the other lanes' loads of the sums come after lane 0's acquire)
        return __shfl_sync(0xFFFFFFFFu, ok, 0);
    }
};

// kChunks: 32-column chunks of an epilogue warp (a tile has 64 kChunks weight rows).  (Compiled in, as every
// branch taken in the loop over the K steps costs about as much as a wait.)
template <int kCtas>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (kCtas == 2) mma_pair_f8f6f4(d, a, b, idesc, accumulate);
    else mma_f8f6f4(d, a, b, idesc, accumulate);
}
template <int kCtas>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (kCtas == 2) mma_commit_pair(bar);
    else mma_commit(bar);
}

// a box of codes to this CTA's shared memory; of a pair's it completes on CTA 0's barrier
template <int kCtas>
__device__ __forceinline__ void copy_codes(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
    if constexpr (kCtas == 2) tma_load_2d_pair(dst, map, peer_smem(bar, 0), x, y);
    else tma_load_2d(dst, map, bar, x, y);
}
// (a pair's come from both CTAs)
template <int kCtas>
__device__ __forceinline__ bool wait_codes(uint64_t *bar, uint32_t parity, uint64_t limit, volatile int *abort) {
    if constexpr (kCtas == 2) return warp_wait_or_look_cluster(bar, parity, limit, abort);
    else return warp_wait_or_look(bar, parity, limit, abort);
}
// Waits until what is under way to the stages has landed, `mine` and `peer` stages being fed by
// this CTA, which announced a stage's copies, and by the other (without one: the same).  They
// differ by a stage ring at most, as neither goes round without the products of both; what only one
// of them fed, of `bytes`, is made up for.
__device__ __forceinline__ void drain_codes(uint64_t *full, int stages, uint32_t mine, uint32_t peer, uint32_t bytes = 0) {
    const uint32_t least = min(mine, peer), most = max(mine, peer);
#pragma unroll 1
    for (uint32_t k = least; k != most; ++k) {
        if (mine > peer) mbar_complete_tx(&full[k % stages], bytes);
        else mbar_arrive_expect_tx(&full[k % stages], bytes);
    }
#pragma unroll 1
    for (uint32_t k = most > uint32_t(stages) ? most - stages : 0; k != most; ++k)
        mbar_wait_bounded(&full[k % stages], k / stages & 1, kDrainPolls, nullptr);
}

template <int kChunks, bool kSplit, int kCtas>
__global__ void __launch_bounds__(kPairWarps * 32, 1)
    lanes_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const F8Args a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // s_full (in CTA 0): both CTAs' copies of a stage; s_empty: the products have read the stage;
    // s_sum: a K step's sums are in TMEM; s_free (in CTA 0): both CTAs' epilogues have them in
    // registers
    using C = Lanes<kChunks, kCtas>;
    constexpr int S = C::kStages;
    constexpr uint32_t b_bytes = C::kB;
    __shared__ uint64_t s_full[S], s_empty[S], s_sum[2], s_free[2], s_drain;
    __shared__ uint32_t s_fed[2];   // in CTA 0: stages that each CTA's copies went to
    __shared__ uint32_t s_tmem;
    __shared__ int s_word;
    __shared__ volatile int s_abort;
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *s_a = smem, *s_b = s_a + S * C::kA, *s_y = s_b + S * b_bytes;   // (s_y: 4 KB an epilogue warp)
    int *s_table = reinterpret_cast<int *>(s_y + 8 * 4096);
    const Groups g{s_table, s_table + a.E + 1};
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = kCtas == 2 ? cluster_rank() : 0;
    const int nb = (a.K + 127) / 128, nt = (a.N + C::kBn - 1) / C::kBn;
    const uint64_t lim = a.wait_limit;
    volatile int *abort = &s_abort;
    if (threadIdx.x == 0) {
#pragma unroll 1
        for (int i = 0; i < S; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_sum[i], 1);
            mbar_init(&s_free[i], 8 * kCtas);
        }
        mbar_init(&s_drain, 1);
        s_abort = 0;
        fence_barrier_init();
    }
    if constexpr (kCtas == 2) {
        cluster_sync();   // both CTAs run, and their barriers are there
        if (warp == 9) tmem_alloc_pair(&s_tmem, 512);
    } else if (warp == 9) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();
    tc_fence_before();
    int total = load_groups(g, a, 128 * kCtas, nt, &s_word);
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    if (total < 0) {
        if (threadIdx.x == 0) atomicOr(&g_f8_status, kStatusGuard);
        total = 0;
    }
    auto give_up = [&]() {
        s_abort = 1;
        atomicOr(&g_f8_status, kStatusTimeout);
    };
    // (a pair gives up together, and neither CTA waits for the other in vain)
    auto tell_peer = [&]() {
        if constexpr (kCtas == 2)
            if (s_abort) peer_store(peer_smem(const_cast<int *>(&s_abort), cluster_rank() ^ 1), 1u);
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(issue_regs(kCtas)));
        if (warp == 8) {
            // ------------------------------------------------------------ TMA
            const bool leader = elect_one();
            if (leader) {
                prefetch_tmap(&map_w);
                prefetch_tmap(&map_x);
            }
            Ring st(1);   // (the first round's waits pass at once)
            uint32_t fed = 0;
            bool ok = true;
            Walk<kSplit, kCtas> work(total, nb);
            while (ok && work.next(total, nb)) {
                const Tile ti = tile_of(work.t, g, a.E, 128 * kCtas, C::kBn);
                const int x_row = ti.g0 + 128 * rank, w_row = ti.e * a.N + ti.n0 + C::kBn / kCtas * rank;
#pragma unroll 1
                for (int kb = kSplit ? work.k0 : 0; kb < (kSplit ? work.k1 : nb); ++kb) {
                    if (!warp_wait_or_look(&s_empty[st.i], st.ph, lim, abort)) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        if (rank == 0) mbar_arrive_expect_tx(&s_full[st.i], kCtas * (C::kA + b_bytes));
                        copy_codes<kCtas>(s_a + st.i * C::kA, &map_x, &s_full[st.i], kb * 128, x_row);
                        copy_codes<kCtas>(s_b + st.i * b_bytes, &map_w, &s_full[st.i], kb * 128, w_row);
                    }
                    __syncwarp();
                    ++fed;
                    st.next(S);
                }
            }
            if (leader) {
                if (!ok) give_up();
                // leave only when the last products have read the stages (their arrivals come from
                // CTA 0) and the copies under way have landed
#pragma unroll 1
                for (int i = 0; i < S && ok; ++i) {
                    ok = mbar_wait_bounded(&s_empty[st.i], st.ph, kDrainPolls, abort);
                    st.next(S);
                }
                tell_peer();
                if constexpr (kCtas == 2) {
                    // (what is left of a pair's codes: below, once both CTAs are here)
                    peer_store(peer_smem(&s_fed[rank], 0), fed);
                    mbar_wait_bounded(&s_drain, 0, kDrainPolls, nullptr);   // CTA 0's last arrival
                } else {
                    drain_codes(s_full, S, fed, fed);
                }
            }
            __syncwarp();
        } else if (warp == 9 && rank == 0) {
            // ------------------------------------------------------------ MMA
            const bool leader = elect_one();
            const uint32_t idesc = idesc_e4m3_f32(128 * kCtas, C::kBn);
            const uint64_t da0 = smem_desc_sw128(smem_u32(s_a)), db0 = smem_desc_sw128(smem_u32(s_b));
            Ring st(0), bf(1);
            bool ok = true;
            Walk<kSplit, kCtas> work(total, nb);
            while (ok && work.next(total, nb)) {
#pragma unroll 1
                for (int kb = kSplit ? work.k0 : 0; kb < (kSplit ? work.k1 : nb); ++kb) {
                    if (!wait_codes<kCtas>(&s_full[st.i], st.ph, lim, abort) ||
                        !warp_wait_or_look(&s_free[bf.i], bf.ph, lim, abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (leader) {
                        // (columns behind K are zeros in both operands)
                        const uint64_t da = da0 + st.i * (C::kA >> 4), db = db0 + st.i * (b_bytes >> 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma<kCtas>(tmem + bf.i * 256, da + 2 * j, db + 2 * j, idesc, j > 0);
                        commit<kCtas>(&s_empty[st.i]);
                        commit<kCtas>(&s_sum[bf.i]);
                    }
                    __syncwarp();
                    st.next(S);
                    bf.next(2);
                }
            }
            if (leader) {
                if (!ok) give_up();
                commit<kCtas>(&s_drain);
                mbar_wait_bounded(&s_drain, 0, kDrainPolls, nullptr);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(epilogue_regs(kCtas)));
        // ------------------------------------------------------- epilogue
        // warp w: lanes of its quarter, half w / 4 of the columns in chunks of 32
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint8_t *buf = s_y + warp * 4096;
        const uint32_t free0 = peer_smem(&s_free[0], 0), free1 = peer_smem(&s_free[1], 0);
        Ring bf(0);
        bool ok = true;
        Walk<kSplit, kCtas> work(total, nb);
        while (ok && work.next(total, nb)) {
            const Tile ti = tile_of(work.t, g, a.E, 128 * kCtas, C::kBn);
            uint64_t acc[kChunks][16];
#pragma unroll
            for (int j = 0; j < kChunks; ++j)
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[j][i] = 0ull;
            // the weight scales of the warp's columns: they lie in one block of 128
            const float *wd = a.wd + (int64_t(ti.e) * ((a.N + 127) / 128) + min(ti.n0 + 32 * kChunks * half, a.N - 1) / 128) * nb;
            const int k0 = kSplit ? work.k0 : 0, k1 = kSplit ? work.k1 : nb;
            // the scales of the lane's token (behind the last one: any) and of the columns, a step ahead
            // (the tokens' through shared memory, with barriers for their arrival and their being
            // read: 4096 x 34816 x 5120 581 us, now 515; loaded two steps ahead 523)
            const float *xd = a.xd + k0 * a.ldxd + min(ti.g0 + 128 * static_cast<int>(rank) + row, a.M - 1);
            float dw = __ldg(wd + k0), dx = __ldg(xd);
#pragma unroll 4
            for (int kb = k0; kb < k1; ++kb) {
                const uint32_t sc = __float_as_uint(__fmul_rn(dx, dw));
                const uint64_t s2 = pair_of(sc, sc);
                xd += a.ldxd;
                if (kb + 1 < k1) {
                    dw = __ldg(wd + kb + 1);
                    dx = __ldg(xd);
                }
                if (!warp_wait_or_look(&s_sum[bf.i], bf.ph, lim, abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t col = tmem + lane_addr + bf.i * 256 + 32 * kChunks * half;
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
                    uint32_t v[32];
                    tmem_ld_x32(col + 32 * j, v);
                    tmem_wait_for(v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[j][i] = fma_f32x2(s2, pair_of(v[2 * i], v[2 * i + 1]), acc[j][i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) peer_arrive(bf.i ? free1 : free0);
                bf.next(2);
            }
            if (!ok) break;
            if (kSplit && (work.k1 < nb || work.k0 > 0)) {
                // (the addresses are made here, not kept over the steps)
                Partials parts{a.ws, static_cast<int>(gridDim.x / 2), static_cast<int>(rank) * 8 + warp};
                asm volatile("" : "+l"(parts.ws), "+r"(parts.pairs), "+r"(parts.warp));
                const int pair = blockIdx.x / 2;
                if (work.k1 < nb) {
                    // the tile's later steps are another pair's: it gets the sums so far
#pragma unroll
                    for (int i = 0; i < 8 * kChunks; ++i) parts.put(pair, i, acc[i / 8][2 * (i % 8)], acc[i / 8][2 * (i % 8) + 1]);
                    parts.publish(pair);
                    continue;
                }
                const int64_t all = int64_t(total) * nb;
                int q0 = pair;   // the first pair with steps of the tile
                while (q0 > 0 && Walk<kSplit, kCtas>::run(all, q0) > int64_t(work.t) * nb) --q0;
                for (int q = q0; q < pair && ok; ++q) {
                    ok = parts.wait(q, lim, abort);
                    if (ok) {
#pragma unroll
                        for (int j = 0; j < kChunks; ++j) {
                            uint64_t part[16];   // (a chunk's loads under way together)
#pragma unroll
                            for (int i = 0; i < 8; ++i) parts.get(q, 8 * j + i, part[2 * i], part[2 * i + 1]);
#pragma unroll
                            for (int i = 0; i < 16; ++i) acc[j][i] = add_f32x2(acc[j][i], part[i]);
                        }
                    }
                }
                if (!ok) break;
            }
            const int r0 = 128 * rank + (warp & 3) * 32;   // the warp's first row of the tile
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                const int n = ti.n0 + 32 * (half * kChunks + j);
                if (n < a.N) {
                    const bool right = a.y_bf16 && (j & 1);
                    __syncwarp();   // (the lines before are read)
                    stage_row(buf, lane, a.y_bf16, right, acc[j]);
                    if (!a.y_bf16 || right || j + 1 == kChunks || n + 32 >= a.N) {
                        __syncwarp();
                        store_lines(a, buf, lane, ti.g0 + r0, r0, ti.clo, ti.chi, right ? n - 32 : n,
                                    a.y_bf16 && !right ? 64 : 128);
                    }
                }
            }
        }
        if (!ok && lane == 0) give_up();
    }
    __syncwarp();
    if (lane == 0) tell_peer();
    tc_fence_before();
    __syncwarp();
    if constexpr (kCtas == 2) {
        cluster_sync();   // nothing of either CTA reaches into the other any more, but copies:
        if (s_abort) {    // (of both or neither) a wait gave up, some may be under way
            // (the rank read anew: kept for this over the steps it cost spills)
            if (cluster_rank() == 0 && warp == 8 && lane == 0)
                drain_codes(s_full, S, s_fed[0], s_fed[1], C::kA + b_bytes);
            __syncwarp();
            cluster_sync();
        }
    } else {
        __syncthreads();
    }
    if (warp == 9) {
        tc_fence_after();
        if constexpr (kCtas == 2) tmem_dealloc_pair(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

// Clears the runs' flags.  The product may start at once: its setup runs meanwhile, and its
// own wait is for the end of this kernel, which comes after everything before it in the stream.
// (333 x 5120 x 17408: 46.8 us, with a memset 48.5.)
__global__ void __launch_bounds__(256) clear_flags(uint4 *flags, int n) {
    pdl_trigger();
    pdl_wait();
    for (int i = threadIdx.x; i < n; i += blockDim.x) flags[i] = make_uint4(0, 0, 0, 0);
}

// one launch in clusters of `cluster` CTAs, overlapping the tail of the stream's last kernel
template <auto kKernel, typename... Args>
h32_status launch_clusters(int grid, int threads, size_t smem, int cluster, cudaStream_t s, const Args &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = allow_smem<kKernel>(kMaxSmem);
    if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kKernel, args...);
    return launch_status(e != cudaSuccess ? e : cudaGetLastError());
}

template <int NC>
h32_status launch_rows(const uint8_t *wq, const uint8_t *xq, F8Args a, int64_t tiles, int cluster, int sms,
                       cudaStream_t s) {
    using C = Rows<NC>;
    const int nb = (a.K + 127) / 128;
    a.cluster = cluster;
    const bool two = tiles * a.cluster > sms && a.cluster > 1;
    const size_t rest = Groups::bytes(a.E) + 1024 + C::parts(a.cluster);
    const int fit = static_cast<int>(((two ? kMaxSmem / 2 : kMaxSmem) - rest) / C::kStage);
    a.stages = fit < kMaxStages ? fit : kMaxStages;
    CUtensorMap maps[3];
    if (!code_map(&maps[0], wq, a.K, int64_t(a.E) * a.N, 128) || !code_map(&maps[1], xq, a.K, a.M, NC) ||
        !scale_map(&maps[2], a.xd, a.ldxd, nb, NC)) {
        note_error("cuTensorMapEncodeTiled rejected a tensor map of the 8-bit product");
        return H32_ERR_CUDA;
    }
    const int grid = a.cluster > 1 ? static_cast<int>(tiles * a.cluster) : static_cast<int>(tiles < sms ? tiles : sms);
    return launch_clusters<rows_kernel<NC>>(grid, kRowsWarps * 32, a.stages * C::kStage + rest, a.cluster, s, maps[0], maps[1],
                                            maps[2], a);
}

template <int kChunks, int kCtas, bool kSplit = false>
h32_status launch_lanes(const uint8_t *wq, const uint8_t *xq, const F8Args &a, int64_t tiles, int sms, cudaStream_t s) {
    using C = Lanes<kChunks, kCtas>;
    CUtensorMap maps[2];
    if (!code_map(&maps[0], wq, a.K, int64_t(a.E) * a.N, C::kBn / kCtas) || !code_map(&maps[1], xq, a.K, a.M, 128)) {
        note_error("cuTensorMapEncodeTiled rejected a tensor map of the 8-bit product");
        return H32_ERR_CUDA;
    }
    const int units = static_cast<int>(tiles < sms / kCtas ? tiles : sms / kCtas);
    // the epilogue's setmaxnreg.inc waits until the pool holds its registers: never launch
    // with fewer registers a thread than the hand-over assumes
    int regs = 0;
    const cudaError_t e = kernel_regs<lanes_kernel<kChunks, kSplit, kCtas>>(&regs);
    if (e != cudaSuccess) return launch_status(e);
    if (regs < kPairRegs) {
        note_error("8-bit product compiled with fewer registers than its warpgroups hand over");
        return H32_ERR_CUDA;
    }
    return launch_clusters<lanes_kernel<kChunks, kSplit, kCtas>>(kCtas * units, kPairWarps * 32, C::kSmem, kCtas, s, maps[0], maps[1],
                                                                a);
}

h32_status run_f8_gemm(const uint8_t *wq, const float *wd, int32_t E, const uint8_t *xq, const float *xd,
                       int64_t ldxd, const int32_t *off, int64_t M, int64_t N, int64_t K, void *y,
                       h32_in_dtype y_dt, int64_t ldy, void *ws, size_t ws_bytes, void *stream) {
    if (E < 1 || E > kMaxExperts || !f8_sizes_fit(M, N, K, E) || ldxd < M || ldxd % 4 != 0 || ldxd > 0xFFFFFFFFll ||
        ldy < N || (y_dt != H32_IN_F32 && y_dt != H32_IN_BF16))
        return H32_ERR_INVALID_ARG;
    if (M == 0) return H32_OK;
    if (!wq || !wd || !xq || !xd || !y) return H32_ERR_INVALID_ARG;
    if (!aligned16(wq) || !aligned16(wd) || !aligned16(xq) || !aligned16(xd) || !aligned16(y) || !aligned16(ws) ||
        (off && reinterpret_cast<uintptr_t>(off) % 4 != 0))
        return H32_ERR_ALIGNMENT;
    int sms = 0;
    H32_TRY(check_device(&sms));
    if (!tensor_map_encoder()) {
        note_error("cuTensorMapEncodeTiled is not available from the driver");
        return H32_ERR_CUDA;
    }
    F8Args a{};
    a.M = static_cast<int32_t>(M);
    a.N = static_cast<int32_t>(N);
    a.K = static_cast<int32_t>(K);
    a.E = E;
    a.off = off;
    a.wd = wd;
    a.xd = xd;
    a.ldxd = ldxd;
    a.y = y;
    a.ldy = ldy;
    a.y_bf16 = y_dt == H32_IN_BF16;
    a.y_vec = ldy * (a.y_bf16 ? 2 : 4) % 16 == 0;
    a.wait_limit = wait_limit();
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const F8Plan plan = plan_f8(M, N, K, E, off != nullptr, sms);
    if (plan.columns == 16) return launch_rows<16>(wq, xq, a, plan.tiles, plan.cluster, sms, s);
    if (plan.columns == 32) return launch_rows<32>(wq, xq, a, plan.tiles, plan.cluster, sms, s);
    if (plan.runs > 0 && ws) {
        if (ws_bytes < Partials::bytes(plan.runs)) return H32_ERR_INVALID_ARG;
        a.ws = static_cast<uint8_t *>(ws);
        const size_t flags = Partials::flags(plan.runs);
        const cudaError_t e = launch_pdl(clear_flags, dim3(1), dim3(256), 0, s,
                                         reinterpret_cast<uint4 *>(a.ws + Partials::bytes(plan.runs) - flags),
                                         static_cast<int>(flags / 16));
        if (e != cudaSuccess) return launch_status(e);
        return launch_lanes<4, 2, true>(wq, xq, a, plan.runs, sms, s);
    }
    if (plan.ctas == 1) {
        if (plan.bn == 256) return launch_lanes<4, 1>(wq, xq, a, plan.tiles, sms, s);
        if (plan.bn == 128) return launch_lanes<2, 1>(wq, xq, a, plan.tiles, sms, s);
        return launch_lanes<1, 1>(wq, xq, a, plan.tiles, sms, s);
    }
    if (plan.bn == 256) return launch_lanes<4, 2>(wq, xq, a, plan.tiles, sms, s);
    if (plan.bn == 128) return launch_lanes<2, 2>(wq, xq, a, plan.tiles, sms, s);
    return launch_lanes<1, 2>(wq, xq, a, plan.tiles, sms, s);
}

}  // namespace

__device__ uint32_t g_f8_status_taken;
__global__ void take_g_f8_status() { g_f8_status_taken = atomicExch(&g_f8_status, 0u); }

h32_status f8_read_and_clear_status(cudaStream_t s) {
    bool ok = false;
    const uint32_t v = take_status(take_g_f8_status, g_f8_status_taken, s, &ok);
    if (!ok) return H32_ERR_CUDA;
    if (v & kStatusTimeout) return H32_ERR_TIMEOUT;
    return (v & kStatusGuard) ? H32_ERR_DEVICE_GUARD : H32_OK;
}

}  // namespace h32

extern "C" h32_status h32_f8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t *bytes) {
    using namespace h32;
    if (!bytes || !f8_sizes_fit(M, N, K, 1)) return H32_ERR_INVALID_ARG;
    int sms = 0;
    H32_TRY(check_device(&sms));
    const int runs = M > 0 ? plan_f8(M, N, K, 1, false, sms).runs : 0;
    *bytes = runs > 0 ? Partials::bytes(runs) : 0;
    return H32_OK;
}

extern "C" h32_status h32_f8_gemm(const uint8_t *wq, const float *wd, const uint8_t *xq, const float *xd,
                                  int64_t ldxd, int64_t M, int64_t N, int64_t K, void *y, h32_in_dtype y_dt,
                                  int64_t ldy, void *workspace, size_t workspace_bytes, void *stream) {
    return h32::run_f8_gemm(wq, wd, 1, xq, xd, ldxd, nullptr, M, N, K, y, y_dt, ldy, workspace, workspace_bytes,
                            stream);
}

extern "C" h32_status h32_f8_gemm_experts(const uint8_t *wq, const float *wd, int32_t E, const uint8_t *xq,
                                          const float *xd, int64_t ldxd, const int32_t *expert_off, int64_t R,
                                          int64_t N, int64_t K, void *y, h32_in_dtype y_dt, int64_t ldy,
                                          void *stream) {
    if (!expert_off) return H32_ERR_INVALID_ARG;
    return h32::run_f8_gemm(wq, wd, E, xq, xd, ldxd, expert_off, R, N, K, y, y_dt, ldy, nullptr, 0, stream);
}
