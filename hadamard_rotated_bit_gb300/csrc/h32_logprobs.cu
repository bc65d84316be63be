// Log probabilities behind the output head (sm_103a): per row of logits the log softmax at
// given tokens, the entropy, and the k most probable tokens.
//
//   m = max l,  S = sum e^(l - m),  W = sum e^(l - m) (l - m)
//   log p(i) = (l_i - m) - log S,   H = log S - W / S
//
// One pass over the logits.  Each thread keeps m, S and W of what it has read (all fp32,
// rescaled when m grows, summed by steps and runs of steps) and, for the k most probable tokens, the
// largest value of each of its chunks (16 fp32 or 32 bf16 values, more where a CTA takes over 16
// steps).  The k-th largest of the 64 maxima of groups of lanes bounds the k best from below, so only
// chunks that reach it, hardly more than k, are read again (from L2) for their values above it, and
// of those the k largest are found by counting, for each, the larger ones.  Nothing in the pass
// itself depends on the values: buffers filled as candidates come cost 30 to 80% more time there.
// Rows where too many values reach the bound (ties, mostly) are read again by warps that keep sorted
// lists.
//
// A row is one CTA's, or with few rows a cluster's: its CTAs take consecutive parts and
// leave their results in the first one's shared memory.
// Bound: HBM, one read of the logits, and next to it instruction issue (2048 x 131072 fp32, top 8:
// 161 us, 99% of the measured copy rate; 4096 x 131072 bf16, top 8: 184 us, 86%); one row: about 9 us
// of steps that wait for one another.
#include "h32_common.cuh"
#include "h32_epilogue.cuh"

#include <float.h>

namespace h32 {
namespace {

constexpr int kMaxTop = 32, kMaxCluster = 8;
constexpr int kVecs = 4;             // 16-byte loads of a thread's step
constexpr int kSlots = 16;           // chunks of a thread (32: 45 KB a CTA, f32 rows 10-40% slower)
constexpr int kRun = 16;             // steps whose sums a thread adds up plainly
constexpr int kMaxChunks = 256, kMaxKeys = 512;   // chunks read again, keys ranked
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kFar = -200.0f;      // e^kFar is 0 in fp32

struct LogprobArgs {
    const void *logits;
    int64_t V, ldl;
    const int32_t *targets;   // [T][n]
    int32_t n, top;
    float *logprob, *entropy, *top_logprob;
    int32_t *top_id;
};

// what a part of a row leaves: the running maximum, sums and best keys
struct Part {
    float m, S, W;
    uint64_t best[kMaxTop];
};

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// pairs of floats in a 64-bit register
__device__ __forceinline__ uint64_t pair(float a, float b) {
    return static_cast<uint64_t>(__float_as_uint(b)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ float low(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p)); }
__device__ __forceinline__ float high(uint64_t p) { return __uint_as_float(static_cast<uint32_t>(p >> 32)); }
// the larger one; NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// floats as integers of the same order (-0 as +0)
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
// the number below (none of the keys is ordered(-0) as it stands)
__device__ __forceinline__ float below(uint32_t o) { return value_of(o == 0x80000000u ? o - 2 : o - 1); }
// 0 is no key: the numbers above -inf have ordered() > 0
__device__ __forceinline__ uint64_t key_of(float v, uint32_t i) {
    return static_cast<uint64_t>(ordered(v)) << 32 | (0xFFFFFFFFu - i);
}
__device__ __forceinline__ uint32_t index_of(uint64_t key) { return 0xFFFFFFFFu - static_cast<uint32_t>(key); }

// one compare-exchange with the lane `o` apart; `large`: this lane keeps the larger
template <typename T>
__device__ __forceinline__ T exchange(T v, int o, bool large) {
    const T w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return (v > w) == large ? v : w;
}
// the warp's 32 values, largest in lane 0
template <typename T>
__device__ __forceinline__ T sort_warp(T v, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int o = size >> 1; o > 0; o >>= 1) v = exchange(v, o, ((lane & o) == 0) == ((lane & size) == 0));
    return v;
}
// the 32 largest of two sorted lists, sorted
__device__ __forceinline__ uint64_t merge_sorted(uint64_t a, uint64_t b, int lane) {
    b = __shfl_xor_sync(0xFFFFFFFFu, b, 31);
    uint64_t v = a > b ? a : b;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = exchange(v, o, (lane & o) == 0);
    return v;
}

// (m, S, W) joined with another part's
__device__ __forceinline__ void join(float &m, float &S, float &W, float m2, float S2, float W2) {
    const float top = fmaxf(m, m2);
    const float da = fmaxf(m - top, kFar), db = fmaxf(m2 - top, kFar);
    const float fa = exp2_fast(da * kLog2e), fb = exp2_fast(db * kLog2e);
    W = fa * fmaf(S, da, W) + fb * fmaf(S2, db, W2);
    S = fa * S + fb * S2;
    m = top;
}

// sum += part, `rest` what the roundings left over (to be added)
__device__ __forceinline__ void add_compensated(float &sum, float &rest, float part) {
    const float y = __fadd_rn(part, rest), t = __fadd_rn(sum, y);
    rest = __fsub_rn(y, __fsub_rn(t, sum));
    sum = t;
}

template <bool kBf16>
struct Vec {
    static constexpr int kN = kBf16 ? 8 : 4;
    uint4 u;
    __device__ __forceinline__ float operator[](int i) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        if constexpr (kBf16) return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        else return __uint_as_float(w[i]);
    }
};

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if constexpr (kBf16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
    else return static_cast<const float *>(p)[i];
}

// A warp's k best of what it is given: a sorted list, a key a lane, and a buffer of values
// above its k-th, merged 32 at a time.
struct List {
    uint64_t key = 0;
    float bound;           // values at or below it are not among the k
    int pending = 0;
    uint64_t *buf;         // [64], the warp's
    int k, lane;

    __device__ __forceinline__ void push(bool p, float v, uint32_t i) {
        const uint32_t mask = __ballot_sync(0xFFFFFFFFu, p);
        if (mask == 0) return;
        if (p) buf[pending + __popc(mask & ((1u << lane) - 1))] = key_of(v, i);
        pending += __popc(mask);
        __syncwarp();
        if (pending >= 32) {
            key = merge_sorted(key, sort_warp(buf[lane], lane), lane);
            const uint64_t rest = buf[32 + lane];
            __syncwarp();
            buf[lane] = rest;
            pending -= 32;
            __syncwarp();
        }
    }
    // once a run of ascending indices is pushed: the k-th of the list is a bound
    __device__ __forceinline__ void raise() {
        const uint32_t kth = static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, key, k - 1) >> 32);
        if (kth != 0) bound = fmaxf(bound, value_of(kth));
    }
    // what is left, as one sorted list
    __device__ __forceinline__ uint64_t finish() {
        return merge_sorted(key, sort_warp(lane < pending ? buf[lane] : 0, lane), lane);
    }
};

// the `top` largest of n different keys, in order, by counting the larger ones of each;
// keys [n .. n + 3] are 0
template <int kThreads>
__device__ __forceinline__ void rank_keys(const uint64_t *keys, int n, int top, uint64_t *best) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t mine = keys[i];
        int above = 0;
#pragma unroll 2
        for (int j = 0; j < n; j += 4) {
            const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(keys + j);
            const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(keys + j + 2);
            above += (p.x > mine) + (p.y > mine) + (q.x > mine) + (q.y > mine);
        }
        if (above < top) best[above] = mine;   // (0, no key: above all that are)
    }
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// `n` bytes (a multiple of 8) of this CTA's shared memory to the first CTA's
template <int kThreads>
__device__ __forceinline__ void to_first(void *dst, const void *src, int bytes) {
    uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst)), r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(d));
    for (int i = threadIdx.x; i < bytes / 8; i += kThreads)
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(r + 8 * i), "l"(static_cast<const uint64_t *>(src)[i])
                     : "memory");
}

template <bool kBf16, int kThreads>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
    using V4 = Vec<kBf16>;
    constexpr int kWarps = kThreads / 32, kGroup = kThreads / 64;   // threads of a group
    constexpr int kN = V4::kN;
    __shared__ __align__(16) float s_chunk[kSlots][kThreads];   // largest values of the chunks
    // keys and the warps' lists behind the pass; in it, for each thread, m, S, W and what the
    // roundings of S and W left over (no memory of their own: the pass is faster with more L1)
    __shared__ __align__(16) uint64_t s_pool[kMaxKeys + 4 + kWarps * 64];
    static_assert(sizeof(s_pool) >= 5 * kThreads * sizeof(float), "a thread's sums of runs");
    uint64_t *s_all = s_pool, *s_buf = s_pool + kMaxKeys + 4;
    float(*s_run)[kThreads] = reinterpret_cast<float(*)[kThreads]>(s_pool);
    __shared__ uint64_t s_best[kMaxTop];
    __shared__ uint32_t s_list[kMaxChunks];
    __shared__ Part s_part[kMaxCluster];
    __shared__ __align__(16) float s_group[64];
    __shared__ float s_m[kWarps], s_S[kWarps], s_W[kWarps], s_bound;
    __shared__ int s_count[2], s_chunks, s_keys;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t c = cluster_size(), rank = cluster_rank();
    const int64_t row = blockIdx.x / c;
    if (tid == 0) s_chunks = s_keys = 0;
    if (tid < kMaxTop) s_part[rank].best[tid] = s_best[tid] = 0;
    pdl_wait();
    pdl_trigger();

    constexpr int kSize = kBf16 ? 2 : 4;
    const uint8_t *l = static_cast<const uint8_t *>(a.logits) + row * a.ldl * kSize;
    // the row as values up to its first 16-byte boundary, whole 16-byte vectors, the rest
    const int64_t skew = (16 - (reinterpret_cast<uintptr_t>(l) & 15)) & 15;
    const int64_t head = min(a.V, skew / kSize), nvec = (a.V - head) / kN, tail = head + nvec * kN;
    const uint4 *body = reinterpret_cast<const uint4 *>(l + head * kSize);
    // this CTA's vectors: steps of kThreads x kVecs, dealt to the cluster in order
    const int64_t steps = (nvec + kThreads * kVecs - 1) / (kThreads * kVecs);
    const int64_t step0 = steps * rank / c, step1 = steps * (rank + 1) / c;
    const int64_t per_slot = (step1 - step0 + kSlots - 1) / kSlots;   // steps of a chunk

    float m = -FLT_MAX, S = 0.0f, W = 0.0f;
    // The sums of even and odd places.  Of S a step's terms are added up by themselves first, the
    // steps' sums plainly for kRun steps, and the runs' with compensation: terms below half a step
    // of the sum, the floor under a likely token, would all be lost if they were added to it one by
    // one (131071 of e^-17 next to 1: 1e-5 of log p).  W has no such 1, its terms are added as they
    // come.  (512 x 100003 fp32 36.2 us, one by one 37.4, every step with compensation 40.9;
    // 4096 x 131072 bf16, top 8: 184, 178 and 184.)
    uint64_t S2 = 0, W2 = 0;
    const auto end_run = [&](bool first) {
        float run_s = low(S2) + high(S2), run_w = low(W2) + high(W2), rest_s = 0.0f, rest_w = 0.0f;
        if (!first) {
            // (m is no lower than the runs' before)
            const float dm = fmaxf(s_run[0][tid] - m, kFar), f = exp2_fast(dm * kLog2e);
            float all_s = s_run[1][tid], all_w = s_run[2][tid];
            rest_s = s_run[3][tid], rest_w = s_run[4][tid];
            all_w = f * fmaf(all_s, dm, all_w);
            rest_w = f * fmaf(rest_s, dm, rest_w);
            all_s *= f;
            rest_s *= f;
            add_compensated(all_s, rest_s, run_s);
            add_compensated(all_w, rest_w, run_w);
            run_s = all_s;
            run_w = all_w;
        }
        s_run[0][tid] = m;
        s_run[1][tid] = run_s;
        s_run[2][tid] = run_w;
        s_run[3][tid] = rest_s;
        s_run[4][tid] = rest_w;
        S2 = W2 = 0;
    };
    // values read as what changes nothing: -inf
    constexpr uint32_t kNone = kBf16 ? 0xFF80FF80u : 0xFF800000u;
    auto load = [&](int64_t step, V4 (&v)[kVecs]) {
        const int64_t at = (step * kWarps + warp) * (32 * kVecs) + lane;
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
            v[u].u = step < step1 && at + 32 * u < nvec ? __ldcs(body + at + 32 * u)
                                                        : make_uint4(kNone, kNone, kNone, kNone);
    };
    V4 next[kVecs];
    load(step0, next);
    float chunk = -INFINITY;
    float *slot = &s_chunk[0][tid];
    int in_slot = 0, slots = 0, in_run = 0, runs = 0;
    for (int64_t step = step0; step < step1; ++step) {
        V4 v[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u) v[u] = next[u];
        load(step + 1, next);
        float cm = v[0][0];
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int i = 0; i < kN; ++i) cm = fmaxf(cm, v[u][i]);
        // (what was summed so far, under the new maximum)
        const float top = fmaxf(m, cm);
        const float dm = fmaxf(m - top, kFar), f = exp2_fast(dm * kLog2e);
        W2 = mul_f32x2(pair(f, f), fma_f32x2(S2, pair(dm, dm), W2));
        S2 = mul_f32x2(S2, pair(f, f));
        m = top;
        const uint64_t less = pair(-m, -m);
        uint64_t s[kVecs];
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
#pragma unroll
            for (int i = 0; i < kN; i += 2) {
                // (-inf and far values: e = 0, and 0 times a finite d)
                const uint64_t x = add_f32x2(pair(v[u][i], v[u][i + 1]), less);
                const uint64_t d = pair(max_nan(low(x), kFar), max_nan(high(x), kFar));
                const uint64_t t = mul_f32x2(d, pair(kLog2e, kLog2e));
                const uint64_t e = pair(exp2_fast(low(t)), exp2_fast(high(t)));
                s[u] = i == 0 ? e : add_f32x2(s[u], e);
                W2 = fma_f32x2(e, d, W2);
            }
        static_assert(kVecs == 4, "vectors of a step");
        S2 = add_f32x2(S2, add_f32x2(add_f32x2(s[0], s[1]), add_f32x2(s[2], s[3])));
        if (++in_run == kRun && step + 1 < step1) {
            end_run(runs++ == 0);
            in_run = 0;
        }
        chunk = fmaxf(chunk, cm);
        if (++in_slot == per_slot || step + 1 == step1) {
            *slot = chunk;
            slot += kThreads;
            chunk = -INFINITY;
            in_slot = 0;
            ++slots;
        }
    }
    const float m_body = m;
    if (runs > 0) {
        end_run(false);
        S = s_run[1][tid] + s_run[3][tid];
        W = s_run[2][tid] + s_run[4][tid];
    } else {
        S = low(S2) + high(S2);
        W = low(W2) + high(W2);
    }
    // the values before and behind the vectors: fewer than 16, a lane each
    float extra = -INFINITY;
    const int64_t extra_at = lane < 16 ? lane : tail + (lane - 16);
    if (rank == 0 && warp == 0) {
        if (lane < 16 ? lane < head : extra_at < a.V) extra = load_logit<kBf16>(l, extra_at);
        join(m, S, W, fmaxf(extra, -FLT_MAX), extra > -INFINITY ? 1.0f : extra == extra ? 0.0f : extra, 0.0f);
    }
    // the warp's sums, then the CTA's
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        join(m, S, W, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, S, o),
             __shfl_xor_sync(0xFFFFFFFFu, W, o));
    if (lane == 0) {
        s_m[warp] = m;
        s_S[warp] = S;
        s_W[warp] = W;
    }
    if (a.top > 0) {
        float g = m_body;
#pragma unroll
        for (int o = 1; o < kGroup; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xFFFFFFFFu, g, o));
        if (lane % kGroup == 0) s_group[tid / kGroup] = g;
    }
    __syncthreads();
    if (warp == 0) {
        if (a.top > 0) {
            // the bound: the k-th largest of the groups' maxima (k <= 32 of 64)
            const float g0 = s_group[lane], g1 = s_group[32 + lane];
            int n0 = 0, n1 = 0;
#pragma unroll 4
            for (int i = 0; i < 64; ++i) {
                const float o = s_group[i];
                n0 += o > g0 || (o == g0 && i < lane);
                n1 += o > g1 || (o == g1 && i < 32 + lane);
            }
            if (n0 == a.top - 1) s_bound = g0;
            if (n1 == a.top - 1) s_bound = g1;
        }
        m = s_m[0], S = s_S[0], W = s_W[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) join(m, S, W, s_m[w], s_S[w], s_W[w]);
        if (lane == 0) {
            s_part[rank].m = m;
            s_part[rank].S = S;
            s_part[rank].W = W;
        }
    }
    if (a.top > 0) {
        __syncthreads();
        // (at least the lowest number: -inf is no candidate)
        const float bound = s_bound;
        if (m_body >= bound)
            for (int i = 0; i < slots; ++i)
                if (s_chunk[i][tid] >= bound) {
                    const int at = atomicAdd(&s_chunks, 1);
                    if (at < kMaxChunks) s_list[at] = static_cast<uint32_t>(i) << 16 | tid;
                }
        __syncthreads();
        const auto keep = [&](bool p, float v, uint32_t i) {
            const uint32_t mask = __ballot_sync(0xFFFFFFFFu, p);
            if (mask == 0) return;
            int at = 0;
            if (lane == 0) at = atomicAdd(&s_keys, __popc(mask));
            at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(mask & ((1u << lane) - 1));
            if (p && at < kMaxKeys) s_all[at] = key_of(v, i);
        };
        const int chunks = s_chunks;
        for (int i = warp; i < min(chunks, kMaxChunks); i += kWarps) {
            const uint32_t e = s_list[i];
            const int64_t first = step0 + (e >> 16) * per_slot, last = min(first + per_slot, step1);
            const int t = e & 0xFFFF;
            for (int64_t step = first; step < last; ++step)
#pragma unroll
                for (int j = 0; j < kVecs * kN; j += 32) {
                    const int u = (j + lane) / kN;
                    const int64_t vec = (step * kWarps + (t >> 5)) * (32 * kVecs) + 32 * u + (t & 31);
                    const bool in = u < kVecs && vec < nvec;
                    const int64_t at = head + vec * kN + lane % kN;
                    const float v = in ? load_logit<kBf16>(l, at) : -INFINITY;
                    keep(v >= bound && v > -INFINITY, v, static_cast<uint32_t>(at));
                }
        }
        if (warp == 0 && rank == 0) keep(extra >= bound && extra > -INFINITY, extra, static_cast<uint32_t>(extra_at));
        __syncthreads();
        int keys = s_keys;
        if (chunks > kMaxChunks || keys > kMaxKeys) {
            // too many: this CTA's values once more, each warp keeping its best, in ascending
            // order of their indices (equal values behind the k-th are not better)
            List list;
            list.bound = below(ordered(bound));
            list.buf = s_buf + 64 * warp;
            list.k = a.top;
            list.lane = lane;
            for (int64_t step = step0; step < step1; ++step) {
                V4 v[kVecs];
                load(step, v);
                const uint32_t i0 = static_cast<uint32_t>(head + ((step * kWarps + warp) * (32 * kVecs) + lane) * kN);
#pragma unroll
                for (int u = 0; u < kVecs; ++u)
#pragma unroll
                    for (int i = 0; i < kN; ++i)
                        list.push(v[u][i] > list.bound && v[u][i] > -INFINITY, v[u][i], i0 + u * 32 * kN + i);
                list.raise();
            }
            if (warp == 0 && rank == 0)   // (out of order: equal values pass, and the keys decide)
                list.push(extra >= list.bound && extra > -INFINITY, extra, static_cast<uint32_t>(extra_at));
            s_all[tid] = list.finish();
            keys = kThreads;
            __syncthreads();
        }
        if (tid < 4) s_all[keys + tid] = 0;
        __syncthreads();
        rank_keys<kThreads>(s_all, keys, a.top, s_part[rank].best);
    }
    if (c > 1) {
        cluster_sync();   // (every CTA of the cluster runs, and its part is in its shared memory)
        if (rank != 0) to_first<kThreads>(&s_part[rank], &s_part[rank], sizeof(Part));
        cluster_sync();
        if (rank != 0) return;
        if (a.top > 0) {
            const int n = static_cast<int>(c) * a.top;
            for (int i = tid; i < n + 4; i += kThreads) s_all[i] = i < n ? s_part[i / a.top].best[i % a.top] : 0;
            __syncthreads();
            rank_keys<kThreads>(s_all, n, a.top, s_best);
        }
    }
    __syncthreads();
    // the row's
    m = s_part[0].m, S = s_part[0].S, W = s_part[0].W;
    for (uint32_t r = 1; r < c; ++r) join(m, S, W, s_part[r].m, s_part[r].S, s_part[r].W);
    if (m == INFINITY) {
        // +inf logits share the probability (the limit of the softmax): count them
        if (threadIdx.x < 2) s_count[threadIdx.x] = 0;
        __syncthreads();
        int inf = 0, nan = 0;
        for (int64_t i = threadIdx.x; i < a.V; i += kThreads) {
            const float v = load_logit<kBf16>(l, i);
            inf += v == INFINITY;
            nan |= v != v;
        }
        atomicAdd(&s_count[0], inf);
        atomicOr(&s_count[1], nan);
        __syncthreads();
        S = s_count[1] ? NAN : static_cast<float>(s_count[0]);
        W = 0.0f;
    }
    // (S - 1 is exact where S is near 1, but S itself is rounded: next to a certain token log p
    // is good to some 2^-24, not relative to itself.)  An empty row (S = 0): log S is not used
    const float log_s = log1pf(S - 1.0f);
    auto logprob_of = [&](float v) {
        if (S != S) return S;
        if (v == -INFINITY || S == 0.0f) return -INFINITY;
        if (m == INFINITY) return v == INFINITY ? -log_s : -INFINITY;
        return v == v ? (v - m) - log_s : v;
    };
    if (threadIdx.x == 0 && a.entropy) a.entropy[row] = S != S ? S : S == 0.0f ? 0.0f : log_s - W / S;
    for (int i = threadIdx.x; i < a.n; i += kThreads) {
        const int32_t t = a.targets[row * a.n + i];
        a.logprob[row * a.n + i] = t < 0 ? 0.0f : t >= a.V ? NAN : logprob_of(load_logit<kBf16>(l, t));
    }
    if (warp == 0 && a.top > 0) {
        const uint64_t key = c > 1 ? s_best[lane] : s_part[0].best[lane];
        const int found = min(a.top, __popc(__ballot_sync(0xFFFFFFFFu, key != 0)));
        int32_t *ids = a.top_id + row * a.top;
        float *lps = a.top_logprob + row * a.top;
        if (lane < found) {
            ids[lane] = static_cast<int32_t>(index_of(key));
            lps[lane] = logprob_of(value_of(static_cast<uint32_t>(key >> 32)));
        }
        // fewer numbers above -inf than asked for: the first -inf, then the first NaN
        int have = found;
        for (int pass = 0; pass < 2 && have < a.top; ++pass)
            for (int64_t i0 = 0; i0 < a.V && have < a.top; i0 += 32) {
                const float v = i0 + lane < a.V ? load_logit<kBf16>(l, i0 + lane) : 0.0f;
                const bool p = pass == 0 ? v == -INFINITY : v != v;
                const uint32_t mask = __ballot_sync(0xFFFFFFFFu, p);
                const int at = have + __popc(mask & ((1u << lane) - 1));
                if (p && at < a.top) {
                    ids[at] = static_cast<int32_t>(i0 + lane);
                    lps[at] = logprob_of(v);
                }
                have += __popc(mask);
            }
    }
}

}  // namespace
}  // namespace h32

extern "C" h32_status h32_token_logprobs(const void *logits, h32_in_dtype dt, int64_t T, int64_t V, int64_t ldl,
                                         const int32_t *targets, int32_t n, int32_t top, float *logprob,
                                         float *entropy, int32_t *top_id, float *top_logprob, void *stream) {
    using namespace h32;
    if (T < 0 || V <= 0 || V > 0x7FFFFFFFll || ldl < V || (dt != H32_IN_F32 && dt != H32_IN_BF16) || n < 0 ||
        top < 0 || top > kMaxTop || top > V || T > 0x7FFFFFFFll / kMaxCluster)
        return H32_ERR_INVALID_ARG;
    if (T == 0) return H32_OK;
    if (!logits || (n > 0 && (!targets || !logprob)) || (top > 0 && (!top_id || !top_logprob)))
        return H32_ERR_INVALID_ARG;
    const auto off4 = [](const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; };
    if (reinterpret_cast<uintptr_t>(logits) % (dt == H32_IN_BF16 ? 2 : 4) != 0 || off4(targets) || off4(logprob) ||
        off4(entropy) || off4(top_id) || off4(top_logprob))
        return H32_ERR_ALIGNMENT;
    int sms = 0;
    H32_TRY(check_device(&sms));
    // CTAs of a row.  With few rows up to 8, as long as each has a step and they are no more than
    // 1.6 an SM, or 2 with at least 16 steps each: beyond, the steps behind the pass and the cluster's
    // meeting cost more than the shorter pass gives (131072 bf16: 76 rows 10.0 us by twos, 15.7
    // by eights; 150 rows 11.2 by one, 17.0 by fours, but fp32 15.8 by twos and 20.8 by one).  Long
    // rows go by twos as long as all of them run at once, five CTAs an SM (131072 fp32 by one and by
    // twos: 160 rows 26.8 and 20.4 us, 240 28.7 and 27.0, 300 30.7 and 29.1, 380 33.9 and 33.1, 400 40.1
    // and 50.9; bf16 160 rows 21.6 and 17.4, 300 23.7 and 20.6, 380 30.4 and 30.0, 400 30.4 and
    // 31.0; rows of 8 steps, 65536 bf16, 420 18.1 and 22.9, 160 the same).
    const int64_t steps = V / (256 * kVecs * (dt == H32_IN_BF16 ? 8 : 4));
    int c = 1;
    while (c < kMaxCluster && 2 * c <= steps &&
           (T * 2 * c * 5 <= 8 * int64_t(sms) || (T * 2 * c <= 2 * int64_t(sms) && steps >= 32 * c)))
        c *= 2;
    if (c == 1 && steps >= 16 && 2 * T <= 5 * int64_t(sms)) c = 2;
    // Many rows: what follows the pass is steps that wait for one another, so more rows at once in
    // CTAs of 128 threads (4096 rows, with 128 and 256 threads: 1000 fp32 24 and 33 us, 11472 bf16 37
    // and 52, 32768 bf16 61 and 70, 65536 bf16 101 and 107, 131072 bf16 and 65536 fp32, 256 KB, equal;
    // beyond, 90000 fp32 275 and 226), unless they are too few to fill the SMs (700 x 50000 fp32 46 and
    // 26) or, of 48 KB or more, between half a wave of such CTAs and one, which then all end together
    // (32768 fp32: 1064 rows 26 and 32 us, but 1250 36 and 34, 1500 46 and 36, 2048 50 and 51; 131072
    // bf16 1500 rows 81 and 74).
    const int64_t bytes = V * (dt == H32_IN_BF16 ? 2 : 4);
    const bool half = c == 1 && T >= 7 * int64_t(sms) && bytes <= 256 * 1024 &&
                      (bytes < 48 * 1024 || T <= 8 * int64_t(sms) || T >= 12 * int64_t(sms));
    const LogprobArgs a{logits, V, ldl, targets, n, top, logprob, entropy, top_logprob, top_id};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(T * c));
    cfg.blockDim = dim3(half ? 128 : 256);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(c);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const auto kernel = dt == H32_IN_BF16 ? half ? logprobs_kernel<true, 128> : logprobs_kernel<true, 256>
                        : half            ? logprobs_kernel<false, 128>
                                          : logprobs_kernel<false, 256>;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return launch_status(e != cudaSuccess ? e : cudaGetLastError());
}
