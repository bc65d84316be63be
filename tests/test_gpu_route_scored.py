"""GPU parity of h32_moe_route_scored against a float64 evaluation of its rule.

Ids, offsets and row maps are exact (near ties included: the rule orders keys by
their values in double).  Weights: relative to the exact value within
  - a score: expf within 2 ulp (4 half steps), the argument's rounding |l - lmax|
    half steps (at most 104, softmax), 1 + or the sum over E in trees (up to 37 adds
    of terms with 4 + |d| half steps each: below 37 + 4 + 104), one divide and one
    product: below 260 half steps of 2^-24;
  - renormalised: the exps of the choices (4 + |d| with |d| <= 104), their sum over
    k <= 32 (31 more), one divide, one product: below 260 as well;
floor 2^-126 * scale where a weight underflows."""
import numpy as np
import pytest

import oracle
from tests._gpu import np_of, torch_of

pytestmark = pytest.mark.gpu

TOL = 260 * 2.0 ** -24


@pytest.fixture(scope="module")
def h32():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hadamard_rotated_bit_gb300 as m
    from hadamard_rotated_bit_gb300 import _build
    _build.build()
    return m


def _check(h32, l, k, bias=None, pad=0, **kw):
    import torch
    T, E = l.shape
    if pad:
        wide = np.full((T, E + pad), 1e9, np.float32)
        wide[:, :E] = l
        lt = torch_of(wide)[:, :E]
    else:
        lt = torch_of(l)
    bt = None if bias is None else torch_of(np.asarray(bias, np.float32))
    ids, w, off, ridx, row_of = h32.h32_moe_route_scored(lt, k, bias=bt, **kw)
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    rid, rw, roff, rridx, rrow = oracle.moe_route_scored(l, k, bias=bias, **kw)
    assert np.array_equal(np_of(ids), rid)
    assert np.array_equal(np_of(off), roff)
    assert np.array_equal(np_of(ridx), rridx)
    assert np.array_equal(np_of(row_of), rrow)
    gw = np_of(w).astype(np.float64)
    floor = 2.0 ** -126 * abs(kw.get("scale", 1.0)) + 2.0 ** -149
    assert np.all(np.abs(gw - rw) <= TOL * np.abs(rw) + floor)


def _logits(T, E, seed, sigma=1.5):
    return (np.random.default_rng(seed).standard_normal((T, E)) * sigma).astype(np.float32)


CASES = [  # T, E, k, n_group, topk_group, group_top
    (1, 1, 1, 1, 1, 1), (1, 128, 8, 1, 1, 1), (7, 5, 5, 1, 1, 2), (33, 64, 6, 8, 3, 1),
    (40, 256, 8, 8, 4, 2), (65, 160, 6, 8, 3, 1), (9, 40, 4, 8, 2, 2), (20, 1000, 32, 5, 3, 2),
    (31, 1024, 32, 32, 31, 2), (17, 1022, 8, 2, 1, 2), (50, 33, 32, 1, 1, 1), (64, 32, 4, 32, 4, 1),
    (12, 36, 12, 4, 2, 2), (300, 37, 8, 1, 1, 1), (8, 512, 1, 16, 1, 1)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,G,tg,gt", CASES)
def test_matches_the_rule(h32, score, renorm, T, E, k, G, tg, gt):
    l = _logits(T, E, T * 31 + E)
    bias = 0.05 * np.random.default_rng(E).standard_normal(E)
    for b in (None, bias.astype(np.float32)):
        _check(h32, l, k, b, score=score, n_group=G, topk_group=tg, group_top=gt,
               renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("T,E,k,G,tg", [(77824, 33, 3, 1, 1), (77825, 40, 4, 8, 3), (190001, 20, 2, 1, 1)])
def test_long_batches(h32, T, E, k, G, tg):
    """Chunks of exactly one pass of tokens, and of more than one."""
    _check(h32, _logits(T, E, T), k, score="sigmoid", n_group=G, topk_group=tg)


def test_row_pitch(h32):
    l = _logits(19, 64, 3)
    for pad in (1, 4, 64):
        _check(h32, l, 5, pad=pad, score="sigmoid", n_group=4, topk_group=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_and_exact_ties(h32, score):
    """Logits one fp32 step apart, equal logits with equal and with different biases,
    biases that undo a difference of scores to the last bit, whole rows equal, scores
    that saturate or underflow in fp32, groups that tie."""
    r = np.random.default_rng(5)
    T, E = 48, 64
    l = _logits(T, E, 8, 0.5)
    for t in range(T):
        p = r.permutation(E)
        l[t, p[1]] = l[t, p[0]]
        l[t, p[2]] = np.nextafter(l[t, p[0]], np.float32(9))
        l[t, p[3]] = np.nextafter(l[t, p[0]], np.float32(-9))
    l[0] = 0.25
    l[1, ::2] = 20.0
    l[1, 1::2] = 25.0                       # sigmoids that round to 1
    l[2] = -120.0 + np.arange(E) * 0.01     # sigmoids that underflow
    l[3] = np.arange(E) * -3.0              # softmax scores that underflow
    l[4, 32:] = l[4, :32]                   # groups equal pairwise
    s0 = 1 / (1 + np.exp(-l[5].astype(np.float64)))
    cancel = (0.75 - s0).astype(np.float32)  # every key of row 5 near 0.75
    some = np.zeros(E, np.float32)
    some[::3] = 0.125
    for b in (None, np.zeros(E, np.float32), some, cancel):
        for G, tg, gt in ((1, 1, 1), (8, 3, 2), (2, 1, 1), (4, 2, 2)):
            for renorm in (True, False):
                _check(h32, l, 7, b, score=score, n_group=G, topk_group=tg, group_top=gt,
                       renormalize=renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_non_finite_logits(h32, score):
    """-inf (masked), NaN and +inf logits, masked whole groups and rows, fewer
    unmasked experts than choices, non-finite biases."""
    r = np.random.default_rng(9)
    T, E = 60, 48
    l = _logits(T, E, 10)
    for t in range(T):
        m = r.random(E)
        l[t, m < 0.3] = -np.inf
        l[t, (m >= 0.3) & (m < 0.35)] = np.nan
    l[0] = -np.inf
    l[1] = np.nan
    l[2, :5] = np.inf
    l[3, 12:] = -np.inf                     # one group of four left
    l[4] = -np.inf
    l[4, 20] = 0.5                          # one expert left
    l[5, ::2] = np.nan
    l[5, 1::2] = -np.inf
    bias = 0.1 * r.standard_normal(E)
    odd = bias.copy()
    odd[3], odd[4], odd[5] = np.nan, -np.inf, np.inf
    for b in (None, bias.astype(np.float32), odd.astype(np.float32)):
        for G, tg, gt in ((1, 1, 1), (4, 2, 2), (4, 1, 1), (12, 5, 2)):
            for renorm in (True, False):
                _check(h32, l, 4, b, score=score, n_group=G, topk_group=tg, group_top=gt,
                       renormalize=renorm)


@pytest.mark.parametrize("T,E,k", [(4096, 64, 2), (2500, 256, 8), (3001, 128, 8)])
def test_many_tokens(h32, T, E, k):
    _check(h32, _logits(T, E, T), k, 0.02 * np.random.default_rng(1).standard_normal(E).astype(np.float32),
           score="sigmoid", n_group=8, topk_group=4, group_top=2, scale=2.5)


@pytest.mark.parametrize("T", [63, 64, 65, 153, 609, 700])
def test_token_counts_around_the_launch_shapes(h32, T):
    """One block up to 64 tokens, chunks beyond; odd last chunks; every expert count
    of a lane; a shared row of choices (one expert with every token)."""
    for E, k, G, tg, gt in ((8, 8, 1, 1, 1), (1024, 2, 1, 1, 1), (72, 6, 8, 3, 2), (640, 9, 5, 2, 2)):
        l = _logits(T, E, T + E)
        l[:, 3] = 9.0
        _check(h32, l, k, None, n_group=G, topk_group=tg, group_top=gt)
        _check(h32, l, k, np.full(E, 0.25, np.float32), score="sigmoid", n_group=G, topk_group=tg,
               group_top=gt)


def test_long_chunks(h32):
    """Chunks of 512 tokens (bitmaps of 16 words an expert), more chunks than SMs."""
    _check_fast(h32, 90001, 1024, 2)
    _check_fast(h32, 78000, 16, 4)


def _check_fast(h32, T, E, k):
    l = _logits(T, E, 77)
    ids, w, off, ridx, row_of = (np_of(t) for t in h32.h32_moe_route_scored(torch_of(l), k))
    assert h32.h32_device_status() == 0
    rid = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    assert np.array_equal(ids, rid)
    tok = np.repeat(np.arange(T), k)
    order = np.lexsort((tok, rid.reshape(-1)))
    assert np.array_equal(ridx, tok[order])
    back = np.empty(T * k, np.int32)
    back[order] = np.arange(T * k)
    assert np.array_equal(row_of.reshape(-1), back)
    assert np.array_equal(off, np.concatenate(([0], np.cumsum(np.bincount(rid.reshape(-1), minlength=E)))))


def test_without_a_workspace(h32):
    """The library call with a null workspace groups the rows all the same."""
    import ctypes
    import torch
    T, E, k = 300, 96, 5
    l = torch_of(_logits(T, E, 6))
    want = h32.h32_moe_route_scored(l, k, score="sigmoid", renormalize=False)
    got = [torch.full_like(t, -3) for t in want]
    v = ctypes.c_void_p
    st = h32.lib().h32_moe_route_scored(
        v(l.data_ptr()), T, E, E, 1, v(0), 1, 1, 1, k, 0, 1.0, *(v(t.data_ptr()) for t in got), v(0), 0,
        v(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_softmax_without_bias_equals_the_plain_router(h32):
    """The same ids, offsets and row maps as h32_moe_route, weights within both bounds."""
    import torch
    l = torch_of(_logits(700, 128, 4))
    a = h32.h32_moe_route(l, 8)
    b = h32.h32_moe_route_scored(l, 8)
    for i in (0, 2, 3, 4):
        assert torch.equal(a[i], b[i])
    assert torch.all((a[1] - b[1]).abs() <= 2 * TOL * a[1])


def test_empty_given_outputs_stream_and_graph(h32):
    import torch
    E, k = 32, 4
    out = h32.h32_moe_route_scored(torch.empty((0, E), device="cuda"), k)
    torch.cuda.synchronize()
    assert out[0].shape == (0, k) and out[2].tolist() == [0] * (E + 1)
    T = 21
    i32 = dict(dtype=torch.int32, device="cuda")
    ids, w = torch.full((T + 2, k), -7, **i32), torch.full((T + 2, k), -7.0, device="cuda")
    off, ridx, rof = (torch.full((E + 3,), -7, **i32), torch.full((T * k + 5,), -7, **i32),
                      torch.full((T + 1, k), -7, **i32))
    l = torch_of(_logits(T, E, 2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h32.h32_moe_route_scored(l, k, score="sigmoid", topk_id=ids, topk_w=w, expert_off=off,
                             row_idx=ridx, row_of=rof, stream=s)
    s.synchronize()
    rid, rw, roff, rridx, rrow = oracle.moe_route_scored(np_of(l), k, score="sigmoid")
    assert np.array_equal(np_of(ids[:T]), rid) and np.array_equal(np_of(off[:E + 1]), roff)
    assert np.array_equal(np_of(ridx[:T * k]), rridx) and np.array_equal(np_of(rof[:T]), rrow)
    for t, n in ((ids, T), (w, T), (off, E + 1), (ridx, T * k), (rof, T)):
        assert torch.all(t[n:] == -7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = h32.h32_moe_route_scored(l, k, score="sigmoid")
    for seed in (5, 6):
        l.copy_(torch_of(_logits(T, E, seed)))
        g.replay()
        torch.cuda.synchronize()
        rid, rw, roff, rridx, rrow = oracle.moe_route_scored(np_of(l), k, score="sigmoid")
        assert np.array_equal(np_of(out[0]), rid) and np.array_equal(np_of(out[3]), rridx)
        assert np.array_equal(np_of(out[2]), roff) and np.array_equal(np_of(out[4]), rrow)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,tg", [(3, 1, 1, 1), (16, 3, 1, 1), (256, 8, 1, 1), (1024, 5, 1, 1), (64, 2, 4, 2)])
def test_duplicates_on_the_border_of_the_choice(h32, score, E, k, G, tg):
    """Two experts of the same logit and bias share the k-th key, and one of a higher id
    has a key one step above theirs, within fp32's errors: it is chosen, the duplicates
    go without (or the lower one takes the last place)."""
    r = np.random.default_rng(E + k)
    T = 200
    for bias in (np.zeros(E, np.float32), np.full(E, 0.125, np.float32)):
        l = (r.standard_normal((T, E)) * 0.5 - 8).astype(np.float32)
        for t in range(T):
            at = np.sort(r.permutation(E)[:3])
            top = np.float32(r.standard_normal() * 0.5)
            l[t, at[:2]] = top
            l[t, at[2]] = np.nextafter(top, np.float32(9))
            others = np.setdiff1d(r.permutation(E), at)[:k - 1]
            l[t, others] = top + 2 + 0.5 * np.arange(k - 1)
        _check(h32, l, k, bias, score=score, n_group=G, topk_group=tg, group_top=1)
        _check(h32, l, min(k + 1, E), bias, score=score, n_group=G, topk_group=tg, group_top=1)


def test_duplicates_and_a_bias_that_undoes_a_score(h32):
    """The duplicates' key is 0.5, a third key is 0.5 and a little in double but at most
    0.5 in fp32."""
    l = np.array([[0, 0, 0.1]], np.float32)
    bias = np.array([0, 0, 0.5 - 1 / (1 + np.exp(-np.float64(l[0, 2]))) + 6.7e-10], np.float32)
    assert bias[2] + 1 / (1 + np.exp(-np.float64(l[0, 2]))) > 0.5
    _check(h32, l, 1, bias, score="sigmoid")
    _check(h32, np.zeros((70, 200), np.float32), 9, np.zeros(200, np.float32), score="softmax")
    _check(h32, np.zeros((70, 200), np.float32), 9, np.full(200, -0.5, np.float32), score="sigmoid")


@pytest.mark.parametrize("E,k", [(5, 1), (40, 4), (256, 8)])
def test_small_scores_beside_a_large_one_that_the_bias_undoes(h32, E, k):
    """Softmax: two experts of negligible scores and biases 2e-8 and 1.9e-8 on the border,
    and one of a score near 0.4 whose bias leaves a little more than 2e-8 of it: in fp32
    its key may come out below both, and it is chosen all the same."""
    r = np.random.default_rng(E)
    T = 300
    bias = np.full(E, -1.0, np.float32)
    a, b, c = k - 1, k, E - 1
    bias[a], bias[b] = 2e-8, 1.9e-8
    bias[:k - 1] = 0.5                      # clear choices
    l = (r.standard_normal((T, E)) - 3).astype(np.float32)
    l[:, [a, b]] = -60 + r.standard_normal((T, 2))
    target = np.float64(3e-8)
    bias[c] = np.float32(-0.4)

    def key(row):
        e = np.exp(row.astype(np.float64) - row.max())
        return e[c] / e.sum() + np.float64(bias[c])

    for t in range(T):
        others = np.exp(np.delete(l[t].astype(np.float64), c)).sum()
        l[t, c] = np.log(others * (target - bias[c]) / (1 - target + bias[c]))
        while key(l[t]) < 2.2e-8:
            l[t, c] = np.nextafter(l[t, c], np.float32(9))
        assert 2.2e-8 <= key(l[t]) < 2e-7
    _check(h32, l, k, bias)
    assert (oracle.moe_route_scored(l, k, bias=bias)[0][:, -1] == c).all()
    for renorm in (True, False):
        _check(h32, l, k + 1, bias, renormalize=renorm)


@pytest.mark.parametrize("E,G,tg,k", [(16, 4, 2, 2), (16, 4, 2, 4), (36, 4, 3, 6), (256, 8, 4, 8), (12, 2, 1, 3)])
def test_scores_that_saturate_without_a_bias(h32, E, G, tg, k):
    """Groups by their two best keys, no bias: sigmoids of different large logits are all 1
    in double, softmax scores of different very low ones all 0, and the lower id is
    first; few such experts (decided one a lane) and many (decided altogether)."""
    r = np.random.default_rng(E + k)
    T = 60
    for many in (2, min(k + 1, E), E):
        l = (r.standard_normal((T, E)) * 0.5 - 3).astype(np.float32)
        for t in range(T):
            at = r.permutation(E)[:many]
            l[t, at] = 39 + 10 * r.random(many)
        _check(h32, l, k, None, score="sigmoid", n_group=G, topk_group=tg, group_top=2)
    l = np.full((1, E), -3, np.float32)
    l[0, 2], l[0, 3] = 39, 40
    assert oracle.moe_route_scored(l, 2, "sigmoid", n_group=G, topk_group=tg, group_top=2)[0].tolist() == [[2, 3]]
    _check(h32, l, 2, None, score="sigmoid", n_group=G, topk_group=tg, group_top=2)
    l = (-1000 * r.random((T, E)) - 1000).astype(np.float32)
    l[:, E // 2] = 0.0
    _check(h32, l, k, None, score="softmax", n_group=G, topk_group=tg, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_near_the_lowest_value(h32, score):
    """Experts switched off by biases near fp32's lowest value: sums of two such keys leave
    fp32's range, and still order their groups; groups of one key and of none beside."""
    low = np.finfo(np.float32).min
    r = np.random.default_rng(12)
    for E, G in ((4, 2), (48, 4), (40, 8), (64, 32)):
        size = E // G
        l = _logits(30, E, E)
        some = np.zeros(E, np.float32)
        some[::2] = low
        some[: size] = low
        scaled = (low * (0.8 + 0.2 * r.random(E))).astype(np.float32)
        high = (-low * (0.8 + 0.2 * r.random(E))).astype(np.float32)
        sums = np.array([np.sort(scaled[g * size:(g + 1) * size].astype(np.float64))[-2:].sum()
                         for g in range(G)])
        assert (sums < low).all() and np.unique(sums).size == G
        masked = l.copy()
        masked[:, size:2 * size] = -np.inf          # a group of no key
        masked[:, 1:size] = -np.inf                 # and one of a single key
        for b in (np.full(E, low, np.float32), some, scaled, high):
            for x in (l, masked):
                for tg in (1, G // 2, G - 1):
                    _check(h32, x, min(size, 4), b, score=score, n_group=G, topk_group=tg, group_top=2)


def test_ratios_of_sigmoids_far_apart(h32):
    """Renormalised weights of choices whose sigmoids are far below the others', down to
    where the weight itself leaves fp32's range: sigmoids that leave it sooner than
    their ratio to a small largest one, on both sides of where the evaluation turns."""
    r = np.random.default_rng(3)
    T, E = 400, 6
    for top in (60.0, 5.0, 0.0, -20.0, -39.9, -40.1, -70.0, -110.0):
        l = (top - 100 * r.random((T, E))).astype(np.float32)
        l[:, 2] = top
        l[0, 3:] = (-39.99, -40.0, -40.01)
        for bias in (None, (0.1 * r.standard_normal(E)).astype(np.float32)):
            _check(h32, l, E, bias, score="sigmoid", scale=2.5)
            _check(h32, l, 3, bias, score="sigmoid", n_group=3, topk_group=2, group_top=2)
