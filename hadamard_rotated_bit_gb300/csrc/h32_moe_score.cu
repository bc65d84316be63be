// Routing by scores (sm_103a): h32_moe_route_scored.
//
// Per token: scores s_e = softmax or sigmoid of the logits, keys s_e + bias_e, the
// topk_group groups of experts with the largest sums of their group_top best
// keys, the k experts of largest key in those groups, their weights from the
// scores alone, and the (token, choice) rows grouped by expert as by
// h32_moe_route.
//
// The order of keys is exact.  Without a bias (and with groups by their best key)
// it is the order of the logits.  Else it is that of the keys' values in double:
// keys are computed in fp32 with a bound on their error, and where two keys whose
// order matters are nearer than their bounds (a few tokens in a thousand on random
// sigmoid keys, fewer with the softmax) the keys in question are taken again in
// double, one a lane.
//
// route_token: one warp per token.  Lane i holds `per` consecutive experts, so a
// lower lane holds lower ids and, with `per` dividing a group's size, a group is a
// run of whole lanes.  Keys become unsigned integers of the same order; each lane
// keeps its two largest, and a round of the selection is one warp-wide integer
// maximum, one ballot (ties: the lowest lane) and the winner's step to its next.
//
// Grouping: a block counts its chunk of tokens per expert while it routes them,
// and a second kernel places the rows of one chunk a block: an expert's rows start
// at the counts of lower experts and of its own in earlier chunks, and a choice's
// rank within the chunk is a population count over the expert's bitmap of tokens.
// Up to 64 tokens one block does both, in one launch.
//
// Bound: instruction issue.  The data are 4 bytes a logit (16.8 MB for 16384 tokens
// x 256 experts, 2.5 us at the copy rate); measured, sigmoid with a bias, 8 groups by
// their two best, top 8: routing 28.8 us (22 without groups), grouping 9.7.  1024 x
// 128, softmax with a bias: 7.2 and 6.3 us.  One token: 6.3 us, one launch (grouping
// by a block an expert, as h32_moe_route: 16384 x 256 290 us altogether).
#include <float.h>

#include "h32_common.cuh"
#include "h32_moe.cuh"

namespace h32 {
namespace {

constexpr int kSoloTokens = 64;       // tokens one block routes and groups in one launch
constexpr int kPlaceThreads = 1024;
static_assert(kPlaceThreads >= kMaxE, "a thread an expert");
constexpr int kPassTokens = 512;      // tokens whose bitmaps are in shared memory at once

struct ScoreArgs {
    const float *logits, *bias;
    int64_t ldl;
    int32_t T, E, k, n_group, topk_group, group_top, per;
    int32_t sigmoid, renorm, vec, lanes;   // lanes: a group's lanes where `per` divides its size, else 0
    float scale;
    int32_t *topk_id;
    float *topk_w;
    int32_t chunk;                         // tokens a block
};

// A key as an unsigned integer of the same order: 0 = not a candidate, 1 = NaN,
// then -inf < ... < +inf (-0 and +0 equal).
__device__ __forceinline__ uint32_t ordered(float key) {
    const uint32_t u = __float_as_uint(__fadd_rn(key, 0.0f));
    const uint32_t o = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
    return isnan(key) ? 1u : o;
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
    return __uint_as_float((u >> 31) ? u & 0x7FFFFFFFu : ~u);
}

// What a token's scores need beside the logit: for the softmax the largest
// logit that is a number and 1 / sum exp(l - max).
template <typename F>
struct Norm {
    F lmax, inv;
};

// score of a logit, to a few ulps; a NaN or -inf logit scores 0
__device__ __forceinline__ float score_of(float l, const Norm<float> &n, bool sigmoid) {
    if (isnan(l) || l == -INFINITY) return 0.0f;
    if (sigmoid) return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-l)));
    if (n.lmax == INFINITY) return l == INFINITY ? n.inv : 0.0f;
    return __fmul_rn(expf(__fsub_rn(l, n.lmax)), n.inv);
}
__device__ __forceinline__ double score_of(double l, const Norm<double> &n, bool sigmoid) {
    if (isnan(l) || l == -static_cast<double>(INFINITY)) return 0.0;
    if (sigmoid) return 1.0 / (1.0 + exp(-l));
    if (isinf(n.lmax)) return isinf(l) ? n.inv : 0.0;
    return exp(l - n.lmax) * n.inv;
}

// key: score + bias, a -inf logit masks its expert (key -inf), a NaN logit or
// bias ranks below it (key NaN)
template <typename F>
__device__ __forceinline__ F key_of(float l, F s, float b) {
    if (isnan(l)) return static_cast<F>(NAN);
    if (l == -INFINITY) return static_cast<F>(isnan(b) ? NAN : -INFINITY);
    return s + static_cast<F>(b);
}

template <typename F>
__device__ __forceinline__ F warp_max(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const F u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = u > v ? u : v;
    }
    return v;
}
template <typename F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// (a, b) with a >= b: the two largest of themselves and v
template <typename F>
__device__ __forceinline__ void insert2(F &a, F &b, F v) {
    if (v > a) {
        b = a;
        a = v;
    } else if (v > b) {
        b = v;
    }
}

// sum of a group's best keys, those above -inf (a the best, b the second)
template <typename F>
__device__ __forceinline__ F group_score(F a, F b, int top) {
    const F none = -static_cast<F>(INFINITY);
    return (top == 1 || b == none) ? a : a + b;
}

__device__ __forceinline__ uint64_t ordered(double key) {
    if (isnan(key)) return 1ull;
    const uint64_t u = static_cast<uint64_t>(__double_as_longlong(key + 0.0));
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

__device__ __forceinline__ double from_ordered(uint64_t u) {
    return __longlong_as_double(static_cast<long long>((u >> 63) ? u & 0x7FFFFFFFFFFFFFFFull : ~u));
}

// The token decided in double altogether: lane j returns choice j's expert.  For
// groups that are not whole lanes and too near, or more near keys than lanes; rare.  The card's
// double rate is low, so every key is computed once and kept.
template <int NPER>
__device__ __noinline__ int route_exact(const ScoreArgs &a, const float *row) {
    const int lane = threadIdx.x & 31;
    const bool sg = a.sigmoid != 0;
    const double none = -static_cast<double>(INFINITY);
    const int e0 = lane * a.per;
    double kd[NPER];
    Norm<double> nm{none, 1.0};
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        kd[i] = (i < a.per && e0 + i < a.E) ? static_cast<double>(row[e0 + i]) : none;
        if (kd[i] > nm.lmax) nm.lmax = kd[i];   // false for NaN
    }
    if (!sg) {
        nm.lmax = warp_max(nm.lmax);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NPER; ++i) sum += score_of(kd[i], nm, false);
        sum = warp_sum(sum);
        nm.inv = sum > 0.0 ? 1.0 / sum : 0.0;
    }
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const int e = e0 + i;
        const bool in = i < a.per && e < a.E;
        kd[i] = key_of<double>(in ? row[e] : -INFINITY, score_of(kd[i], nm, sg),
                               (in && a.bias) ? a.bias[e] : 0.0f);
    }
    uint32_t groups = 0xFFFFFFFFu;   // the groups chosen, one bit each
    const int size = a.E / a.n_group;
    if (a.n_group > 1) {
        // the two best keys of every group, compared as integers of the same order
        const uint64_t floor = ordered(none);
        uint64_t g1 = floor, g2 = floor;   // lane g: group g's
        for (int g = 0; g < a.n_group; ++g) {
            uint64_t b1 = floor, b2 = floor;
#pragma unroll
            for (int i = 0; i < NPER; ++i) {
                const int e = e0 + i;
                if (i < a.per && e >= g * size && e < (g + 1) * size) insert2(b1, b2, ordered(kd[i]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t c1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
                const uint64_t c2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
                insert2(b1, b2, c1);
                insert2(b1, b2, c2);
            }
            if (lane == g) {
                g1 = b1;
                g2 = b2;
            }
        }
        const double mine = group_score(from_ordered(g1), from_ordered(g2), a.group_top);
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const double o = __shfl_sync(0xFFFFFFFFu, mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        groups = __ballot_sync(0xFFFFFFFFu, lane < a.n_group && rank < a.topk_group);
    }
    uint64_t key[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const int e = e0 + i;
        const bool in = i < a.per && e < a.E && ((groups >> min(e / size, 31)) & 1u);
        key[i] = in ? ordered(kd[i]) : 0ull;
    }
    int my = -1;
    for (int j = 0; j < a.k; ++j) {
        uint64_t best = 0ull;
        int at = 0;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t bh = static_cast<uint32_t>(best >> 32), bl = static_cast<uint32_t>(best);
        const uint32_t mh = __reduce_max_sync(0xFFFFFFFFu, bh);
        const uint32_t ml = __reduce_max_sync(0xFFFFFFFFu, bh == mh ? bl : 0u);
        const int w = __ffs(__ballot_sync(0xFFFFFFFFu, bh == mh && bl == ml)) - 1;
        const int id = __shfl_sync(0xFFFFFFFFu, e0 + at, w);
        if (lane == j) my = id;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (lane == w && i == at) key[i] = 0ull;
    }
    return my;
}

// The double normaliser of the token's softmax scores.
template <int NPER>
__device__ __forceinline__ Norm<double> exact_norm(const ScoreArgs &a, const float *row) {
    const int e0 = (threadIdx.x & 31) * a.per;
    Norm<double> nm{-static_cast<double>(INFINITY), 1.0};
    double v[NPER];
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        v[i] = (i < a.per && e0 + i < a.E) ? static_cast<double>(row[e0 + i])
                                           : -static_cast<double>(INFINITY);
        if (v[i] > nm.lmax) nm.lmax = v[i];   // false for NaN
    }
    nm.lmax = warp_max(nm.lmax);
    const bool inf = isinf(nm.lmax);
    double sum = 0.0;
    // (no branches: the exps run side by side; terms below exp(-700) add nothing)
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const double e = exp(fmax(v[i] - nm.lmax, -700.0));
        const bool none = !(v[i] > -static_cast<double>(INFINITY));   // or NaN
        sum += none ? 0.0 : inf ? (v[i] == nm.lmax ? 1.0 : 0.0) : e;
    }
    sum = warp_sum(sum);
    nm.inv = sum > 0.0 ? 1.0 / sum : 0.0;
    return nm;
}

// Groups whose scores are too near, a group being whole lanes (ScoreArgs::lanes):
// bit i of `cand` marks the lane's experts that may be among their group's best,
// one or two in most lanes; their keys in double, the groups' scores and order.
// Returns whether the lane's group stays.
template <int NPER>
__device__ __noinline__ bool exact_groups(const ScoreArgs &a, const float *row, uint32_t cand) {
    const int lane = threadIdx.x & 31, e0 = lane * a.per;
    const bool sg = a.sigmoid != 0;
    const double none = -static_cast<double>(INFINITY);
    Norm<double> nm{none, 1.0};
    if (!sg) nm = exact_norm<NPER>(a, row);
    uint64_t b1 = ordered(none), b2 = b1;
    while (__any_sync(0xFFFFFFFFu, cand != 0u)) {
        if (cand) {
            const int e = e0 + __ffs(cand) - 1;
            cand &= cand - 1u;
            const float l = row[e];
            insert2(b1, b2, ordered(key_of<double>(l, score_of(static_cast<double>(l), nm, sg),
                                                   a.bias ? a.bias[e] : 0.0f)));
        }
    }
    const uint64_t m1 = b1, m2 = b2;
    const int first = lane - lane % a.lanes, me = lane - first;
    for (int j = 1; j < a.lanes; ++j) {
        const int from = (first + (me + j >= a.lanes ? me + j - a.lanes : me + j)) & 31;
        const uint64_t c1 = __shfl_sync(0xFFFFFFFFu, m1, from);
        const uint64_t c2 = __shfl_sync(0xFFFFFFFFu, m2, from);
        insert2(b1, b2, c1);
        insert2(b1, b2, c2);
    }
    const double mine = group_score(from_ordered(b1), from_ordered(b2), a.group_top);
    const int my_group = lane / a.lanes;
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
        const double o = __shfl_sync(0xFFFFFFFFu, mine, g * a.lanes);
        rank += o > mine || (o == mine && g < my_group);
    }
    return my_group < a.n_group && rank < a.topk_group;
}

// A token whose nearest keys are among its first c (sorted, c <= 32; lane j holds
// candidate j's expert and logit): those keys alone in double, one a lane, and
// their order.  Lane j returns choice j's expert.  (Without a bias too: logits that
// differ may have one score, and then the lower id is first.)
template <int NPER>
__device__ __noinline__ int route_refine(const ScoreArgs &a, const float *row, int c, int id) {
    const int lane = threadIdx.x & 31;
    const bool sg = a.sigmoid != 0, in = lane < c;
    const float l = in ? row[id] : -INFINITY;
    Norm<double> nm{-static_cast<double>(INFINITY), 1.0};
    if (!sg) nm = exact_norm<NPER>(a, row);
    const double key = key_of<double>(l, score_of(static_cast<double>(l), nm, sg),
                                      (in && a.bias) ? a.bias[id] : 0.0f);
    const uint64_t mine = in ? ordered(key) : 0ull;
    int rank = 0;
    for (int j = 0; j < c; ++j) {
        const uint64_t o = __shfl_sync(0xFFFFFFFFu, mine, j);
        const int oid = __shfl_sync(0xFFFFFFFFu, id, j);
        rank += o > mine || (o == mine && oid < id);
    }
    int my = -1;
    for (int j = 0; j < a.k; ++j) {
        const int from = __ffs(__ballot_sync(0xFFFFFFFFu, in && rank == j)) - 1;
        const int e = __shfl_sync(0xFFFFFFFFu, id, from);
        if (lane == j) my = e;
    }
    return my;
}

// 1 / (1 + exp(-l)) by the fast units (its error is in the bounds below); results
// below 2^-126 come out as 0
__device__ __forceinline__ float fast_sigmoid(float l) {
    float e, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(l, -1.4426950408889634f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(__fadd_rn(1.0f, e)));
    return s;
}

// Routes the warp's token: writes its choices and weights; lane j returns choice
// j's expert (lanes >= k: -1).  kLogit: the keys are ordered as the logits.
template <int NPER, bool kLogit>
__device__ __forceinline__ int route_token(const ScoreArgs &a, int64_t t) {
    const int lane = threadIdx.x & 31;
    const float *row = a.logits + t * a.ldl;
    const bool sg = a.sigmoid != 0;
    const int e0 = lane * a.per;
    const float none = -INFINITY;
    float l[NPER];
    if (NPER % 4 == 0 && a.vec) {   // per == NPER, everything on 16-byte boundaries
#pragma unroll
        for (int i = 0; i + 3 < NPER; i += 4) {
            float4 f = make_float4(none, none, none, none);
            if (e0 + i < a.E) f = *reinterpret_cast<const float4 *>(row + e0 + i);
            l[i] = f.x;
            l[i + 1] = f.y;
            l[i + 2] = f.z;
            l[i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPER; ++i) l[i] = (i < a.per && e0 + i < a.E) ? row[e0 + i] : none;
    }
    Norm<float> nm{none, 1.0f};
    if (!sg && (!kLogit || !a.renorm)) {
#pragma unroll
        for (int i = 0; i < NPER; ++i) nm.lmax = fmaxf(nm.lmax, l[i]);   // skips NaN
        nm.lmax = warp_max(nm.lmax);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NPER; ++i) sum += score_of(l[i], nm, false);
        sum = warp_sum(sum);
        nm.inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    }
    uint32_t key[NPER];
    float bias[NPER];
    if (!kLogit && a.bias) {
        if (NPER % 4 == 0 && a.vec) {
#pragma unroll
            for (int i = 0; i + 3 < NPER; i += 4) {
                float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (e0 + i < a.E) f = *reinterpret_cast<const float4 *>(a.bias + e0 + i);
                bias[i] = f.x;
                bias[i + 1] = f.y;
                bias[i + 2] = f.z;
                bias[i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                bias[i] = (i < a.per && e0 + i < a.E) ? a.bias[e0 + i] : 0.0f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPER; ++i) bias[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const bool in = i < a.per && e0 + i < a.E;
        float k = l[i];
        if constexpr (!kLogit) {
            // a NaN logit gives a NaN score and key; a -inf logit masks its expert
            k = sg ? fast_sigmoid(k) : isnan(k) ? k : score_of(k, nm, false);
            k = __fadd_rn(k, bias[i]);
            if (l[i] == none && !isnan(k)) k = none;
        }
        key[i] = in ? ordered(k) : 0u;
    }
    // the lane's two largest keys after (kl, il) in decreasing order (0: none), the
    // lower id first among equals
    uint32_t k1 = 0u, k2 = 0u;
    int i1 = 0, i2 = 0;
    auto scan = [&](uint32_t kl, int il) {
        k1 = k2 = 0u;
#pragma unroll
        for (int i = 0; i < NPER; ++i) {
            const uint32_t v = (key[i] < kl || (key[i] == kl && i > il)) ? key[i] : 0u;
            if (v > k1) {
                k2 = k1;
                i2 = i1;
                k1 = v;
                i1 = i;
            } else if (v > k2) {
                k2 = v;
                i2 = i;
            }
        }
    };
    scan(0xFFFFFFFFu, -1);
    // Bounds on the fp32 errors of keys, in units of u = 2^-23 (kLogit: none needed).
    // Scores: the fast sigmoid is within (2 + 1.2 |l|) (1 - s) + 2.5 relative, at most
    // 5 absolute; a softmax score within 2.5 + 1.7 d relative (expf, the rounding of
    // d = lmax - l) and what all share, the sum of up to 1024 terms (38).  With a bias
    // that is absolute: 5, or 40 smax, and the key's rounding adds |key|.  Without one
    // what all share leaves the order alone: (8 + 2 d) s, d = -ln(s / smax) >= |l|, d.
    const float u = 0x1p-23f, tiny = 0x1p-124f;   // tiny: below the fast units' range
    const float cap = a.bias ? (sg ? 5.0f : 40.0f * nm.inv) * u : 0.0f;
    auto err_of = [&](float k) {
        if (a.bias) return cap + fabsf(k) * u;
        const float d = k > 0.0f ? fmaxf(0.0f, -__logf(sg ? k : __fdividef(k, nm.inv))) : 104.0f;
        return fabsf(k) * (8.0f + 2.0f * d) * u + tiny;
    };
    bool near = false, alive = true;   // alive: the lane's experts may be chosen
    if (a.n_group > 1) {
        const int size = a.E / a.n_group;
        float mine = none, err = 0.0f;   // the group's score and its bound
        float f1 = none, f2 = none;      // its two best keys
        auto finish = [&](uint32_t b1, uint32_t b2) {
            f1 = from_ordered(b1);
            f2 = from_ordered(b2);
            mine = group_score(f1, f2, a.group_top);
            if constexpr (!kLogit) {
                // (a sum below fp32's range is a score all the same, unlike no key at all)
                if (f1 > none) mine = fmaxf(mine, -FLT_MAX);
                if (f1 > none) err = err_of(f1);
                if (a.group_top == 2 && f2 > none) err += err_of(f2) + fabsf(mine) * u;
            }
        };
        const uint32_t floor = 0x007FFFFFu;   // -inf: NaN and absent keys count as that
        int my_group;                          // the group this lane's score is of (n_group: none)
        if (a.lanes) {
            // a group is `lanes` whole lanes: all groups at once
            uint32_t b1 = max(k1, floor), b2 = max(k2, floor);
            auto merge = [&](uint32_t c1, uint32_t c2) {
                b2 = max(min(b1, c1), max(b2, c2));
                b1 = max(b1, c1);
            };
            if ((a.lanes & (a.lanes - 1)) == 0) {
                for (int o = 1; o < a.lanes; o <<= 1) {
                    const uint32_t c1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
                    const uint32_t c2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
                    merge(c1, c2);
                }
            } else {
                const uint32_t m1 = b1, m2 = b2;
                const int first = lane - lane % a.lanes, me = lane - first;
                for (int j = 1; j < a.lanes; ++j) {
                    const int from = first + (me + j >= a.lanes ? me + j - a.lanes : me + j);
                    const uint32_t c1 = __shfl_sync(0xFFFFFFFFu, m1, from & 31);
                    const uint32_t c2 = __shfl_sync(0xFFFFFFFFu, m2, from & 31);
                    merge(c1, c2);
                }
            }
            finish(b1, b2);
            my_group = min(lane / a.lanes, a.n_group);
        } else {
            uint32_t s1 = floor, s2 = floor;
            for (int g = 0; g < a.n_group; ++g) {
                uint32_t b1 = floor, b2 = floor;
#pragma unroll
                for (int i = 0; i < NPER; ++i) {
                    const int e = e0 + i;
                    const uint32_t v = (e >= g * size && e < (g + 1) * size) ? max(key[i], floor) : floor;
                    b2 = max(min(b1, v), b2);
                    b1 = max(b1, v);
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint32_t c1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
                    const uint32_t c2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
                    b2 = max(min(b1, c1), max(b2, c2));
                    b1 = max(b1, c1);
                }
                if (lane == g) {
                    s1 = b1;
                    s2 = b2;
                }
            }
            finish(s1, s2);
            my_group = min(lane, a.n_group);
        }
        const int step = a.lanes ? a.lanes : 1;
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const float o = __shfl_sync(0xFFFFFFFFu, mine, g * step);
            rank += o > mine || (o == mine && g < my_group);
        }
        const bool have = my_group < a.n_group;
        bool stays = have && rank < a.topk_group;
        if constexpr (!kLogit) {
            const int in_at = __ffs(__ballot_sync(0xFFFFFFFFu, have && rank == a.topk_group - 1)) - 1;
            const int out_at = __ffs(__ballot_sync(0xFFFFFFFFu, have && rank == a.topk_group)) - 1;
            const float in = __shfl_sync(0xFFFFFFFFu, mine, in_at);
            const float out = __shfl_sync(0xFFFFFFFFu, mine, out_at);
            const float worst = __uint_as_float(
                __reduce_max_sync(0xFFFFFFFFu, have ? __float_as_uint(err) : 0u));
            // (both -inf: no key in either; they go by id)
            near = out > none && !(in - out > 2.0f * worst);
            if (a.lanes && near) {
                // an expert may be among its group's best when its key is within the
                // errors of the last of them
                const float last = a.group_top == 2 ? f2 : f1;
                const float cut = last > none ? last - 4.0f * err_of(last) : none;
                uint32_t cand = 0u;
#pragma unroll
                for (int i = 0; i < NPER; ++i)
                    if (have && key[i] > 0x007FFFFFu && !(from_ordered(key[i]) < cut)) cand |= 1u << i;
                stays = exact_groups<NPER>(a, row, cand);
                near = false;
            }
        }
        if (a.lanes) {
            alive = stays;
            if (!stays) k1 = k2 = 0u;   // never scanned again: it wins no round
        } else {
            const uint32_t groups = __ballot_sync(0xFFFFFFFFu, stays);
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                if (!((groups >> min((e0 + i) / size, 31)) & 1u)) key[i] = 0u;
            scan(0xFFFFFFFFu, -1);
        }
    }
    // k rounds; then the best key left out
    int my = -1;
    uint32_t my_u = 0u;
    auto take = [&](int j) {   // the best key that is left, to lane j
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, k1);
        const int w = __ffs(__ballot_sync(0xFFFFFFFFu, k1 == m)) - 1;
        const int id = __shfl_sync(0xFFFFFFFFu, e0 + i1, w);
        if (lane == j) {
            my = id;
            my_u = m;
        }
        if (lane == w) {
            if (k2) {
                k1 = k2;
                i1 = i2;
                k2 = 0u;
            } else {
                scan(k1, i1);
            }
        }
        return m;
    };
    for (int j = 0; j < a.k; ++j) take(j);
    float ml = lane < a.k ? row[my] : 0.0f;
    if constexpr (!kLogit) {
        // choice j against the one after it, the last against the best left out; both
        // finite: above -inf and below +inf as ordered integers
        const uint32_t next_u = __reduce_max_sync(0xFFFFFFFFu, k1);
        uint32_t ou = __shfl_down_sync(0xFFFFFFFFu, my_u, 1);
        if (lane == a.k - 1) ou = next_u;
        bool unclear = false;
        if (lane < a.k && ou > 0x007FFFFFu && my_u < 0xFF800000u) {
            const float ka = from_ordered(my_u), kb = from_ordered(ou);
            unclear = !(ka - kb > err_of(ka) + err_of(kb));
        }
        const uint32_t unclears = __ballot_sync(0xFFFFFFFFu, unclear);
        bool tie = false;
        if (unclears) {
            // whether key ka (logit la, bias ba) is at least kb for certain: they are the
            // same key, or further apart than their errors
            auto apart = [&](float ka, float la, float ba, float kb, float lb, float bb) {
                float err = err_of(ka) + err_of(kb);
                if (a.bias && !sg) {
                    // what the softmax's scores share weighs only by their difference, the
                    // rest by its own d
                    const float sa = score_of(la, nm, false), sb = score_of(lb, nm, false);
                    err = fminf(err, u * (40.0f * fabsf(sa - sb) + sa * (3.0f + 1.7f * (nm.lmax - la)) +
                                          sb * (3.0f + 1.7f * (nm.lmax - lb)) + fabsf(ka) + fabsf(kb)) + tiny);
                }
                return (ka == kb && la == lb && ba == bb) || ka - kb > err;
            };
            const float mb = (lane < a.k && a.bias) ? a.bias[my] : 0.0f;
            const float ol = __shfl_down_sync(0xFFFFFFFFu, ml, 1);
            const float ob = __shfl_down_sync(0xFFFFFFFFu, mb, 1);
            if (unclear && lane < a.k - 1) tie = !apart(from_ordered(my_u), ml, mb, from_ordered(ou), ol, ob);
            // The last choice: below it by err_of's bounds, which do not depend on the pair,
            // the best key left out speaks for all of them.  Else every key left out within
            // the errors is held against the last choice by itself: one that is apart (its
            // scores share what they err by, or it is the very same key) says nothing of the
            // others.
            if ((unclears >> (a.k - 1)) & 1u) {
                const uint32_t last_u = __shfl_sync(0xFFFFFFFFu, my_u, a.k - 1);
                const float last = from_ordered(last_u), cut = last - 4.0f * err_of(last);
                const int last_id = __shfl_sync(0xFFFFFFFFu, my, a.k - 1);
                const float last_l = __shfl_sync(0xFFFFFFFFu, ml, a.k - 1);
                const float last_b = __shfl_sync(0xFFFFFFFFu, mb, a.k - 1);
                uint32_t cand = 0u;   // the lane's keys left out that are not below `cut`
#pragma unroll
                for (int i = 0; i < NPER; ++i)
                    if (alive && key[i] > 0x007FFFFFu && !(from_ordered(key[i]) < cut) &&
                        (key[i] < last_u || (key[i] == last_u && e0 + i > last_id)))
                        cand |= 1u << i;
                while (cand) {
                    const int at = __ffs(cand) - 1;
                    cand &= cand - 1u;
                    uint32_t v = 0u;
#pragma unroll
                    for (int i = 0; i < NPER; ++i)
                        if (i == at) v = key[i];
                    tie |= !apart(last, last_l, last_b, from_ordered(v), row[e0 + at],
                                  a.bias ? a.bias[e0 + at] : 0.0f);
                }
            }
        }
        if (__any_sync(0xFFFFFFFFu, near)) {
            my = route_exact<NPER>(a, row);
            if (lane < a.k) ml = row[my];
        } else if (__any_sync(0xFFFFFFFFu, tie)) {
            // more candidates until one is clearly below the ones before it
            uint32_t last = __shfl_sync(0xFFFFFFFFu, my_u, a.k - 1);
            int c = a.k;
            bool clear = false;
            for (; c <= 32; ++c) {
                const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, k1);
                const float ka = from_ordered(last), kb = from_ordered(m);
                clear = m <= 0x007FFFFFu || ka - kb > err_of(ka) + err_of(kb);
                if (clear || c == 32) break;
                last = take(c);
            }
            my = clear ? route_refine<NPER>(a, row, c, my) : route_exact<NPER>(a, row);
            if (lane < a.k) ml = row[my];
        }
    }
    // weights, from the scores alone
    float w;
    if (a.renorm) {
        // ratios of scores: for the softmax (and for sigmoids so far below 1 that they
        // are exp(l) to fp32) exp(l - the largest chosen logit), which cannot underflow
        // together; else the sigmoids times 2^64, those far below 1 as (exp(l / 2) 2^32)^2,
        // so that none vanishes before its ratio does
        const bool num = lane < a.k && !isnan(ml);
        const float lc = warp_max(num ? ml : none);
        float x = 0.0f;
        if (num && ml > none) {
            if (sg && lc > -40.0f) {
                const bool far = ml <= -40.0f;
                const float e = expf(far ? 0.5f * ml : -ml);
                const float r = far ? __fmul_rn(e, 0x1p32f) : __fdiv_rn(1.0f, __fadd_rn(1.0f, e));
                x = __fmul_rn(r, far ? r : 0x1p64f);
            } else if (lc == INFINITY) {
                x = ml == lc ? 1.0f : 0.0f;
            } else {
                x = expf(__fsub_rn(ml, lc));
            }
        }
        if (lc == none && lane < a.k) x = 1.0f;   // every choice masked: equal weights
        float s = 0.0f;
        for (int j = 0; j < a.k; ++j) s = __fadd_rn(s, __shfl_sync(0xFFFFFFFFu, x, j));
        w = __fdiv_rn(x, s);
    } else {
        w = lane < a.k ? score_of(ml, nm, sg) : 0.0f;
    }
    if (lane < a.k) {
        a.topk_id[t * a.k + lane] = my;
        a.topk_w[t * a.k + lane] = __fmul_rn(w, a.scale);
    }
    return lane < a.k ? my : -1;
}

// exclusive prefix over the block's threads in order, E <= blockDim.x values
// (threads >= E pass 0); s_warp: 32 ints
__device__ __forceinline__ int block_exclusive(int v, int *s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
    return before + x - v;
}

// Rows of the choices of tokens [t0, t1): s_start[e] = the first row of expert e's
// choices in this chunk, s_map[e][words] = the bitmap of the chunk's tokens that
// chose e.
__device__ __forceinline__ void place_chunk(const int32_t *topk_id, int t0, int t1, int k, int words,
                                            const int *s_start, const uint32_t *s_map,
                                            int32_t *row_idx, int32_t *row_of) {
    const int n = (t1 - t0) * k;
    for (int c = threadIdx.x; c < n; c += blockDim.x) {
        const int i = c / k, e = topk_id[static_cast<int64_t>(t0) * k + c];
        const uint32_t *map = s_map + e * words;
        int r = s_start[e] + __popc(map[i >> 5] & ((1u << (i & 31)) - 1u));
        for (int w = 0; w < (i >> 5); ++w) r += __popc(map[w]);
        row_of[static_cast<int64_t>(t0) * k + c] = r;
        row_idx[r] = t0 + i;
    }
}

// pitch of a row of counts: whole 16-byte groups
__host__ __device__ constexpr int count_pitch(int E) { return (E + 3) & ~3; }

// One block of `chunk` tokens: routes them and writes the chunk's counts per
// expert, counts[chunk][count_pitch(E)].
template <int NPER, bool kLogit>
__global__ void __launch_bounds__(1024) route_chunk_kernel(const ScoreArgs a, int32_t *counts) {
    __shared__ int s_count[kMaxE];
    pdl_wait();
    pdl_trigger();
    const int pitch = count_pitch(a.E);
    for (int e = threadIdx.x; e < pitch; e += blockDim.x) s_count[e] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * a.chunk, n = min(a.T - t0, a.chunk);
    for (int i = threadIdx.x >> 5; i < n; i += blockDim.x >> 5) {
        const int e = route_token<NPER, kLogit>(a, static_cast<int64_t>(t0) + i);
        if (e >= 0 && counts) atomicAdd(&s_count[e], 1);
    }
    if (!counts) return;
    __syncthreads();
    for (int e = threadIdx.x; e < pitch; e += blockDim.x)
        counts[static_cast<int64_t>(blockIdx.x) * pitch + e] = s_count[e];
}

// The whole call in one block, for few tokens.
template <int NPER, bool kLogit>
__global__ void __launch_bounds__(1024) route_solo_kernel(const ScoreArgs a, int32_t *expert_off,
                                                          int32_t *row_idx, int32_t *row_of) {
    constexpr int kWords = kSoloTokens / 32;
    __shared__ uint32_t s_map[kMaxE * kWords];
    __shared__ int s_start[kMaxE];
    __shared__ int s_warp[32];
    pdl_wait();
    pdl_trigger();
    for (int e = threadIdx.x; e < a.E * kWords; e += blockDim.x) s_map[e] = 0u;
    __syncthreads();
    for (int t = threadIdx.x >> 5; t < a.T; t += blockDim.x >> 5) {
        const int e = route_token<NPER, kLogit>(a, t);
        if (e >= 0) atomicOr(&s_map[e * kWords + (t >> 5)], 1u << (t & 31));
    }
    __syncthreads();
    // expert offsets, blockDim.x experts at a time
    int base = 0;
    for (int e0 = 0; e0 < a.E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int n = 0;
        if (e < a.E)
            for (int w = 0; w < kWords; ++w) n += __popc(s_map[e * kWords + w]);
        const int at = base + block_exclusive(n, s_warp);
        if (e < a.E) {
            s_start[e] = at;
            expert_off[e] = at;
            if (e == a.E - 1) expert_off[a.E] = at + n;
        }
        __syncthreads();
        for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) base += s_warp[w];
        __syncthreads();
    }
    place_chunk(a.topk_id, 0, a.T, a.k, kWords, s_start, s_map, row_idx, row_of);
}

// One block a chunk: where each expert's rows of the chunk start, then the rows, the
// bitmaps of up to kPassTokens tokens at a time.
__global__ void __launch_bounds__(kPlaceThreads)
    route_place_kernel(const int32_t *__restrict__ topk_id, const int32_t *__restrict__ counts, int T,
                       int E, int k, int chunk, int chunks, int32_t *__restrict__ expert_off,
                       int32_t *__restrict__ row_idx, int32_t *__restrict__ row_of) {
    extern __shared__ uint32_t s_map[];   // [E][words]
    __shared__ int s_before[kMaxE], s_all[kMaxE];
    __shared__ int s_warp[32];
    const int words = (min(chunk, kPassTokens) + 31) / 32;
    for (int e = threadIdx.x; e < E; e += kPlaceThreads) s_before[e] = s_all[e] = 0;
    for (int i = threadIdx.x; i < E * words; i += kPlaceThreads) s_map[i] = 0u;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const int t0 = blockIdx.x * chunk, t1 = t0 + min(T - t0, chunk);
    int p0 = t0, p1 = t0 + min(t1 - t0, kPassTokens);
    const int32_t *ids = topk_id + static_cast<int64_t>(t0) * k;
    const int n0 = (p1 - p0) * k;
    const int x0 = threadIdx.x < n0 ? ids[threadIdx.x] : 0;   // on its way during the counts
    // counts of earlier chunks and of all: four columns (experts) of the table per
    // thread, the rows shared out over the threads of a column
    const int quads = count_pitch(E) / 4, cols = min((quads + 31) & ~31, kPlaceThreads);
    const int segs = kPlaceThreads / cols, q = threadIdx.x % cols, seg = threadIdx.x / cols;
    if (q < quads && seg < segs) {
        int4 before = make_int4(0, 0, 0, 0), all = before;
        const int4 *table = reinterpret_cast<const int4 *>(counts) + q;
#pragma unroll 10
        for (int c = seg; c < chunks; c += segs) {
            const int4 n = table[static_cast<int64_t>(c) * quads];
            const int m = c < static_cast<int>(blockIdx.x) ? -1 : 0;
            all = make_int4(all.x + n.x, all.y + n.y, all.z + n.z, all.w + n.w);
            before = make_int4(before.x + (n.x & m), before.y + (n.y & m), before.z + (n.z & m),
                               before.w + (n.w & m));
        }
        auto add = [&](int i, int b, int t) {
            if (t) {   // (columns past E are 0)
                atomicAdd(&s_before[4 * q + i], b);
                atomicAdd(&s_all[4 * q + i], t);
            }
        };
        add(0, before.x, all.x);
        add(1, before.y, all.y);
        add(2, before.z, all.z);
        add(3, before.w, all.w);
    }
    auto fill = [&](const int32_t *id, int n, int first) {
        for (int c = threadIdx.x; c < n; c += kPlaceThreads) {
            const int i = c / k, x = c == static_cast<int>(threadIdx.x) ? first : id[c];
            atomicOr(&s_map[x * words + (i >> 5)], 1u << (i & 31));
        }
    };
    fill(ids, n0, x0);
    __syncthreads();
    const int x = threadIdx.x;
    const int tot = x < E ? s_all[x] : 0;
    const int at = block_exclusive(tot, s_warp);
    if (x < E) {
        s_before[x] += at;
        if (blockIdx.x == 0) {
            expert_off[x] = at;
            if (x == E - 1) expert_off[E] = at + tot;
        }
    }
    __syncthreads();
    for (;;) {
        place_chunk(topk_id, p0, p1, k, words, s_before, s_map, row_idx, row_of);
        if (p1 == t1) break;
        __syncthreads();
        if (x < E) {   // past this pass's rows
            for (int w = 0; w < words; ++w) {
                s_before[x] += __popc(s_map[x * words + w]);
                s_map[x * words + w] = 0u;
            }
        }
        __syncthreads();
        p0 = p1;
        p1 += min(t1 - p1, kPassTokens);
        ids = topk_id + static_cast<int64_t>(p0) * k;
        fill(ids, (p1 - p0) * k, threadIdx.x < (p1 - p0) * k ? ids[threadIdx.x] : 0);
        __syncthreads();
    }
}

// The chunks of a call with a workspace: as many as the card has SMs, twice that where
// they are longer than a pass (their table of counts stays small for any T).
struct Chunks {
    int64_t size, count;
};
inline Chunks route_chunks(int64_t T) {
    constexpr int64_t kSms = 152;
    int64_t size = (T + kSms - 1) / kSms;
    if (size < 8) size = 8;
    if (size > kPassTokens) size = (T + 2 * kSms - 1) / (2 * kSms);
    return Chunks{size, (T + size - 1) / size};
}

template <int NPER, bool kLogit>
cudaError_t launch_scored(const ScoreArgs &a, int32_t *counts, int64_t blocks, bool solo,
                          int32_t *expert_off, int32_t *row_idx, int32_t *row_of, cudaStream_t s) {
    const int warps = a.chunk < 32 ? a.chunk : 32;
    if (solo)   // (at least 8 warps: they share the offsets of the experts)
        return launch_pdl(route_solo_kernel<NPER, kLogit>, dim3(1), dim3((warps < 8 ? 8 : warps) * 32),
                          0, s, a, expert_off, row_idx, row_of);
    return launch_pdl(route_chunk_kernel<NPER, kLogit>, dim3(static_cast<unsigned>(blocks)),
                      dim3(warps * 32), 0, s, a, counts);
}

}  // namespace
}  // namespace h32

extern "C" h32_status h32_moe_route_scored_workspace_bytes(int64_t T, int32_t E, size_t *bytes) {
    using namespace h32;
    if (!bytes) return H32_ERR_INVALID_ARG;
    *bytes = 0;
    if (T < 0 || T > 0x7FFFFFFFll || E < 1 || E > kMaxE) return H32_ERR_INVALID_ARG;
    if (T > kSoloTokens) *bytes = static_cast<size_t>(route_chunks(T).count) * count_pitch(E) * 4;
    return H32_OK;
}

extern "C" h32_status h32_moe_route_scored(const float *logits, int64_t T, int32_t E, int64_t ldl,
                                           int32_t score, const float *bias, int32_t n_group,
                                           int32_t topk_group, int32_t group_top, int32_t k,
                                           int32_t renormalize, float scale, int32_t *topk_id,
                                           float *topk_w, int32_t *expert_off, int32_t *row_idx,
                                           int32_t *row_of, void *workspace,
                                           size_t workspace_bytes, void *stream) {
    using namespace h32;
    if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E || ldl < E || !expert_off)
        return H32_ERR_INVALID_ARG;
    if ((score != H32_SCORE_SOFTMAX && score != H32_SCORE_SIGMOID) || n_group < 1 ||
        n_group > 32 || E % n_group != 0 || topk_group < 1 || topk_group > n_group ||
        group_top < 1 || group_top > 2 || k > topk_group * (E / n_group) || !(scale > -INFINITY) ||
        !(scale < INFINITY))
        return H32_ERR_INVALID_ARG;
    if (T > 0x7FFFFFFFll || T * k > 0x7FFFFFFFll) return H32_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !topk_id || !topk_w || !row_idx || !row_of))
        return H32_ERR_INVALID_ARG;
    auto off4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    if (off4(logits) || off4(bias) || off4(expert_off) || (topk_id && !aligned16(topk_id)) ||
        off4(topk_w) || off4(row_idx) || off4(row_of))
        return H32_ERR_ALIGNMENT;
    const bool solo = T <= kSoloTokens;
    const Chunks ch = route_chunks(T);
    if (workspace && !solo) {
        if (workspace_bytes < static_cast<size_t>(ch.count) * count_pitch(E) * 4) return H32_ERR_INVALID_ARG;
        if (!aligned16(workspace)) return H32_ERR_ALIGNMENT;
    }
    H32_TRY(check_device(nullptr));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int t32 = static_cast<int>(T);
    if (T == 0)
        return launch_status(launch_route_group(topk_id, 0, E, k, expert_off, row_idx, row_of, s));
    ScoreArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.ldl = ldl;
    a.T = t32;
    a.E = E;
    a.k = k;
    a.n_group = topk_group == n_group ? 1 : n_group;   // all groups stay: no groups
    a.topk_group = topk_group;
    a.group_top = group_top;
    a.sigmoid = score == H32_SCORE_SIGMOID;
    a.renorm = renormalize != 0;
    a.scale = scale;
    a.topk_id = topk_id;
    a.topk_w = topk_w;
    a.chunk = static_cast<int32_t>(solo ? T : workspace ? ch.size : 8);
    const int64_t blocks = solo ? 1 : workspace ? ch.count : (T + 7) / 8;
    // experts a lane: the fewest, or the next divisor of a group's size, so that
    // groups are whole lanes
    const int fewest = (E + 31) / 32;
    a.per = fewest;
    if (a.n_group > 1) {
        const int size = E / a.n_group;
        for (int d = fewest; d <= 32 && d <= size; ++d)
            if (size % d == 0) {
                a.per = d;
                a.lanes = size / d;
                break;
            }
    }
    const bool v4 = E % 4 == 0 && ldl % 4 == 0 && aligned16(logits) && (!bias || aligned16(bias));
    const bool by_logit = !bias && (a.n_group == 1 || group_top == 1);
    int32_t *counts = solo ? nullptr : static_cast<int32_t *>(workspace);
    cudaError_t e;
#define H32_SCORED(N)                                                                             \
    do {                                                                                          \
        a.vec = v4 && (N) % 4 == 0 && a.per == (N);                                               \
        e = by_logit ? launch_scored<N, true>(a, counts, blocks, solo, expert_off, row_idx, row_of, s) \
                     : launch_scored<N, false>(a, counts, blocks, solo, expert_off, row_idx, row_of, s); \
    } while (0)
    if (a.per <= 1) H32_SCORED(1);
    else if (a.per <= 2) H32_SCORED(2);
    else if (a.per <= 4) H32_SCORED(4);
    else if (a.per <= 8) H32_SCORED(8);
    else if (a.per <= 16) H32_SCORED(16);
    else H32_SCORED(32);
#undef H32_SCORED
    if (e != cudaSuccess || solo) return launch_status(e != cudaSuccess ? e : cudaGetLastError());
    if (!workspace)
        return launch_status(launch_route_group(topk_id, t32, E, k, expert_off, row_idx, row_of, s));
    const int64_t pass = ch.size < kPassTokens ? ch.size : kPassTokens;
    const size_t smem = static_cast<size_t>(E) * ((pass + 31) / 32) * 4;
    if (smem > 32768) {   // above what a kernel may use beside its static arrays unasked
        e = cudaFuncSetAttribute(route_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 65536);
        if (e != cudaSuccess) return launch_status(e);
    }
    e = launch_pdl(route_place_kernel, dim3(static_cast<unsigned>(ch.count)), dim3(kPlaceThreads), smem,
                   s, topk_id, counts, t32, E, k, static_cast<int>(ch.size),
                   static_cast<int>(ch.count), expert_off, row_idx, row_of);
    return launch_status(e != cudaSuccess ? e : cudaGetLastError());
}
