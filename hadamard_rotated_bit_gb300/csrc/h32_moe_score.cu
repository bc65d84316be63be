// Routing by scores (sm_103a): h32_moe_route_scored.
//
// Per token: scores s_e = softmax or sigmoid of the logits, keys s_e + bias_e, the
// topk_group groups of experts with the largest sums of their group_top best
// keys, the k experts of largest key in those groups, their weights from the
// scores alone, and the (token, choice) rows grouped by expert as by
// h32_moe_route.  The order of keys is that of their values in double: keys are
// computed in fp32 with a bound on their error, and where two keys whose order
// matters are nearer than their bounds (about one token in a thousand on random
// logits) the token is decided again in double.
//
// One warp per token.  Lane i holds `per` consecutive experts, so a lower lane
// holds lower ids and, with `per` dividing a group's size, a group is a run of
// whole lanes.  Keys become unsigned integers of the same order; a round of the
// selection is one warp-wide integer maximum, one ballot (ties: the lowest
// lane) and the winner's rescan of its own keys.
//
// Bound: instruction issue.  The data are 4 bytes a logit (16.8 MB for 16384
// tokens x 256 experts, 2.5 us at the copy rate) against about 70 instructions a
// token and round.
#include "h32_common.cuh"
#include "h32_moe.cuh"

namespace h32 {
namespace {

constexpr int kScoreWarps = 8;   // tokens a block

struct ScoreArgs {
    const float *logits, *bias;
    int64_t ldl;
    int32_t T, E, k, n_group, topk_group, group_top, per;
    int32_t sigmoid, renorm, vec;
    float scale;
    int32_t *topk_id;
    float *topk_w;
};

// A key as an unsigned integer of the same order: 0 = not a candidate, 1 = NaN,
// then -inf < ... < +inf (-0 and +0 equal).
__device__ __forceinline__ uint32_t ordered(float key) {
    if (isnan(key)) return 1u;
    const uint32_t u = __float_as_uint(__fadd_rn(key, 0.0f));
    return (u >> 31) ? ~u : u | 0x80000000u;
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

// score of a logit; a NaN or -inf logit scores 0
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

// The token decided in double: lane j returns choice j's expert.  Slow (the
// card's double rate is low) and rare.
__device__ __noinline__ int route_exact(const ScoreArgs &a, const float *row) {
    const int lane = threadIdx.x & 31;
    const bool sg = a.sigmoid != 0;
    const double none = -static_cast<double>(INFINITY);
    const int e0 = lane * a.per, e1 = min(e0 + a.per, a.E);
    Norm<double> nm{none, 0.0};
    if (!sg) {
        for (int e = e0; e < e1; ++e) {
            const double l = row[e];
            if (l > nm.lmax) nm.lmax = l;   // false for NaN
        }
        nm.lmax = warp_max(nm.lmax);
        double sum = 0.0;
        nm.inv = 1.0;
        for (int e = e0; e < e1; ++e) sum += score_of(static_cast<double>(row[e]), nm, false);
        sum = warp_sum(sum);
        nm.inv = sum > 0.0 ? 1.0 / sum : 0.0;
    }
    auto key = [&](int e) {
        const float l = row[e];
        return key_of<double>(l, score_of(static_cast<double>(l), nm, sg),
                              a.bias ? a.bias[e] : 0.0f);
    };
    uint32_t groups = 0xFFFFFFFFu;   // the groups chosen, one bit each
    if (a.n_group > 1) {
        const int size = a.E / a.n_group;
        double mine = none;   // lane g: group g's score
        for (int g = 0; g < a.n_group; ++g) {
            double b1 = none, b2 = none;
            for (int e = max(e0, g * size); e < min(e1, (g + 1) * size); ++e) insert2(b1, b2, key(e));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const double c1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
                const double c2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
                insert2(b1, b2, c1);
                insert2(b1, b2, c2);
            }
            if (lane == g) mine = group_score(b1, b2, a.group_top);
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const double o = __shfl_sync(0xFFFFFFFFu, mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        groups = __ballot_sync(0xFFFFFFFFu, lane < a.n_group && rank < a.topk_group);
    }
    // k rounds: the best expert after the previous choice in (key, id) order
    double last = 0.0;
    int last_id = -1, my = -1;
    const int size = a.n_group > 1 ? a.E / a.n_group : a.E;
    auto before = [](double ka, int ia, double kb, int ib) {   // (ka, ia) ranks above (kb, ib)
        if (ib < 0) return ia >= 0;
        if (ia < 0) return false;
        const bool na = isnan(ka), nb = isnan(kb);
        if (na || nb) return na && nb ? ia < ib : nb;
        return ka > kb || (ka == kb && ia < ib);
    };
    for (int j = 0; j < a.k; ++j) {
        double bk = 0.0;
        int bi = -1;
        for (int e = e0; e < e1; ++e) {
            if (a.n_group > 1 && !((groups >> (e / size)) & 1u)) continue;
            const double ke = key(e);
            if (last_id >= 0 && !before(last, last_id, ke, e)) continue;
            if (before(ke, e, bk, bi)) {
                bk = ke;
                bi = e;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double ok = __shfl_xor_sync(0xFFFFFFFFu, bk, o);
            const int oi = __shfl_xor_sync(0xFFFFFFFFu, bi, o);
            if (before(ok, oi, bk, bi)) {
                bk = ok;
                bi = oi;
            }
        }
        last = bk;
        last_id = bi;
        if (lane == j) my = bi;
    }
    return my;
}

template <int NPER>
__global__ void __launch_bounds__(kScoreWarps * 32) route_scored_kernel(const ScoreArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kScoreWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const float *row = a.logits + t * a.ldl;
    const bool sg = a.sigmoid != 0;
    const int e0 = lane * a.per;
    float l[NPER];
    if (a.vec) {   // per == NPER, a multiple of 4, everything on 16-byte boundaries
#pragma unroll
        for (int i = 0; i < NPER; i += 4) {
            float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e0 + i < a.E) f = *reinterpret_cast<const float4 *>(row + e0 + i);
            l[i] = f.x;
            if (NPER > 1) l[i + (NPER > 1)] = f.y;
            if (NPER > 2) l[i + (NPER > 2) * 2] = f.z;
            if (NPER > 3) l[i + (NPER > 3) * 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            l[i] = (i < a.per && e0 + i < a.E) ? row[e0 + i] : -INFINITY;
    }
    Norm<float> nm{-INFINITY, 1.0f};
    if (!sg) {
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
#pragma unroll
    for (int i = 0; i < NPER; ++i) {
        const int e = e0 + i;
        const bool in = i < a.per && e < a.E;
        const float s = score_of(l[i], nm, sg);
        key[i] = in ? ordered(key_of<float>(l[i], s, (a.bias && in) ? a.bias[e] : 0.0f)) : 0u;
    }
    // Bounds on the fp32 errors, in units of 2^-23.  With a bias: a sigmoid is
    // within 4, a softmax score within (32 + |l - lmax|) s <= 32 smax (expf, the
    // difference's rounding, a sum of up to 1024 terms in trees), and the key's own
    // rounding adds |key|.  Without one the key is the score: a sigmoid is within 4 s,
    // and of a softmax score what all share (the sum) leaves their order alone and
    // the rest is within (5 + |l - lmax|) s, |l - lmax| <= 104 where it is not 0.
    const float u = 0x1p-23f, tiny = 0x1p-140f;   // tiny: subnormal results
    const float cap = a.bias ? (sg ? 4.0f : 32.0f * nm.inv) * u : 0.0f;
    const float rel = (a.bias ? 1.0f : sg ? 5.0f : 110.0f) * u;
    bool near = false;
    if (a.n_group > 1) {
        const int size = a.E / a.n_group;
        const float none = -INFINITY;
        float mine = none, err = 0.0f;   // lane g: group g's score and its bound
        for (int g = 0; g < a.n_group; ++g) {
            float b1 = none, b2 = none;
#pragma unroll
            for (int i = 0; i < NPER; ++i) {
                const int e = e0 + i;
                if (key[i] > 1u && e >= g * size && e < (g + 1) * size)
                    insert2(b1, b2, from_ordered(key[i]));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const float c1 = __shfl_xor_sync(0xFFFFFFFFu, b1, o);
                const float c2 = __shfl_xor_sync(0xFFFFFFFFu, b2, o);
                insert2(b1, b2, c1);
                insert2(b1, b2, c2);
            }
            if (lane == g) {
                mine = group_score(b1, b2, a.group_top);
                if (b1 > none) err = cap + fabsf(b1) * rel + tiny;
                if (a.group_top == 2 && b2 > none)
                    err += cap + fabsf(b2) * rel + fabsf(mine) * u + tiny;
            }
        }
        int rank = 0;
        for (int g = 0; g < a.n_group; ++g) {
            const float o = __shfl_sync(0xFFFFFFFFu, mine, g);
            rank += o > mine || (o == mine && g < lane);
        }
        const bool have = lane < a.n_group;
        const uint32_t groups = __ballot_sync(0xFFFFFFFFu, have && rank < a.topk_group);
        if (a.topk_group < a.n_group) {
            const int in_at = __ffs(__ballot_sync(0xFFFFFFFFu, have && rank == a.topk_group - 1)) - 1;
            const int out_at = __ffs(__ballot_sync(0xFFFFFFFFu, have && rank == a.topk_group)) - 1;
            const float in = __shfl_sync(0xFFFFFFFFu, mine, max(in_at, 0));
            const float out = __shfl_sync(0xFFFFFFFFu, mine, max(out_at, 0));
            const float worst = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(err)));
            // (both -inf: no key in either; they go by id)
            near = out > none && !(in - out > 2.0f * worst);
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                if (!((groups >> min((e0 + i) / size, 31)) & 1u)) key[i] = 0u;
        }
    }
    // k rounds, and one more for the best key left out
    uint32_t best = 0u, next_u = 0u;
    int at = 0, my = -1, next = -1;
    uint32_t my_u = 0u;
    auto rescan = [&]() {
        best = 0u;
#pragma unroll
        for (int i = 0; i < NPER; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
    };
    rescan();
    for (int j = 0; j <= a.k; ++j) {
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
        const int w = __ffs(__ballot_sync(0xFFFFFFFFu, best == m)) - 1;
        const int id = __shfl_sync(0xFFFFFFFFu, e0 + at, w);
        if (j == a.k) {
            next = m ? id : -1;
            next_u = m;
        } else if (lane == j) {
            my = id;
            my_u = m;
        }
        if (lane == w) {
#pragma unroll
            for (int i = 0; i < NPER; ++i)
                if (i == at) key[i] = 0u;
            rescan();
        }
    }
    // choice j against the one after it (the last against the best left out)
    float ml = 0.0f, mb = 0.0f;
    if (lane < a.k) {
        ml = row[my];
        mb = a.bias ? a.bias[my] : 0.0f;
    }
    {
        const float nl = next >= 0 ? row[next] : 0.0f;
        const float nb = (next >= 0 && a.bias) ? a.bias[next] : 0.0f;
        uint32_t ou = __shfl_down_sync(0xFFFFFFFFu, my_u, 1);
        float ol = __shfl_down_sync(0xFFFFFFFFu, ml, 1);
        float ob = __shfl_down_sync(0xFFFFFFFFu, mb, 1);
        const bool last = lane == a.k - 1;
        if (last) {
            ou = next_u;
            ol = nl;
            ob = nb;
        }
        // both finite (above -inf and below +inf as ordered integers)
        const uint32_t lo = 0x007FFFFFu, hi = 0xFF800000u;
        if (lane < a.k && ou > lo && my_u < hi) {
            const float ka = from_ordered(my_u), kb = from_ordered(ou);
            const float bound = 2.0f * cap + (fabsf(ka) + fabsf(kb)) * rel + tiny;
            const bool same = my_u == ou && ml == ol && mb == ob;
            near = near || (!same && !(ka - kb > bound));
        }
    }
    if (__any_sync(0xFFFFFFFFu, near)) {
        my = route_exact(a, row);
        if (lane < a.k) ml = row[my];
    }
    // weights, from the scores alone
    float w;
    if (a.renorm) {
        // ratios of scores: for the softmax (and for sigmoids so far below 1 that they
        // are exp(l) to fp32) exp(l - the largest chosen logit), which cannot underflow
        // together
        const bool num = lane < a.k && !isnan(ml);
        const float lc = warp_max(num ? ml : -INFINITY);
        float x = 0.0f;
        if (num && ml > -INFINITY) {
            if (sg && lc > -40.0f) x = score_of(ml, nm, true);
            else if (lc == INFINITY) x = ml == lc ? 1.0f : 0.0f;
            else x = expf(__fsub_rn(ml, lc));
        }
        if (lc == -INFINITY && lane < a.k) x = 1.0f;   // every choice masked: equal weights
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
}

}  // namespace
}  // namespace h32

extern "C" h32_status h32_moe_route_scored(const float *logits, int64_t T, int32_t E, int64_t ldl,
                                           int32_t score, const float *bias, int32_t n_group,
                                           int32_t topk_group, int32_t group_top, int32_t k,
                                           int32_t renormalize, float scale, int32_t *topk_id,
                                           float *topk_w, int32_t *expert_off, int32_t *row_idx,
                                           int32_t *row_of, void *stream) {
    using namespace h32;
    if (T < 0 || E < 1 || E > kMaxE || k < 1 || k > kMaxK || k > E || ldl < E || !expert_off)
        return H32_ERR_INVALID_ARG;
    if ((score != H32_SCORE_SOFTMAX && score != H32_SCORE_SIGMOID) || n_group < 1 ||
        n_group > 32 || E % n_group != 0 || topk_group < 1 || topk_group > n_group ||
        group_top < 1 || group_top > 2 || k > topk_group * (E / n_group) || !(scale > -INFINITY) ||
        !(scale < INFINITY))
        return H32_ERR_INVALID_ARG;
    if (T * k > 0x7FFFFFFFll) return H32_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !topk_id || !topk_w || !row_idx || !row_of))
        return H32_ERR_INVALID_ARG;
    auto off4 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; };
    if (off4(logits) || off4(bias) || off4(expert_off) || (topk_id && !aligned16(topk_id)) ||
        off4(topk_w) || off4(row_idx) || off4(row_of))
        return H32_ERR_ALIGNMENT;
    H32_TRY(check_device(nullptr));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T > 0) {
        ScoreArgs a{};
        a.logits = logits;
        a.bias = bias;
        a.ldl = ldl;
        a.T = static_cast<int32_t>(T);
        a.E = E;
        a.k = k;
        a.n_group = n_group;
        a.topk_group = topk_group;
        a.group_top = group_top;
        a.per = (E + 31) / 32;
        a.sigmoid = score == H32_SCORE_SIGMOID;
        a.renorm = renormalize != 0;
        a.scale = scale;
        a.topk_id = topk_id;
        a.topk_w = topk_w;
        const dim3 grid(static_cast<unsigned>((T + kScoreWarps - 1) / kScoreWarps));
        const dim3 block(kScoreWarps * 32);
        const bool v4 = E % 4 == 0 && ldl % 4 == 0 && aligned16(logits);
        cudaError_t e1;
#define H32_SCORED(N)                                                     \
    do {                                                                  \
        a.vec = v4 && (N) % 4 == 0 && a.per == (N);                       \
        e1 = launch_pdl(route_scored_kernel<N>, grid, block, 0, s, a);    \
    } while (0)
        if (a.per <= 1) H32_SCORED(1);
        else if (a.per <= 2) H32_SCORED(2);
        else if (a.per <= 4) H32_SCORED(4);
        else if (a.per <= 8) H32_SCORED(8);
        else if (a.per <= 16) H32_SCORED(16);
        else H32_SCORED(32);
#undef H32_SCORED
        if (e1 != cudaSuccess) return launch_status(e1);
    }
    const cudaError_t e2 = launch_route_group(topk_id, static_cast<int>(T), E, k, expert_off, row_idx,
                                              row_of, s);
    return launch_status(e2 != cudaSuccess ? e2 : cudaGetLastError());
}
