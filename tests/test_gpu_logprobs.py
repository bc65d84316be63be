"""GPU parity of h32_token_logprobs against a 64-bit evaluation: ids exactly, log
probabilities and entropies within a bound derived from the roundings."""
import numpy as np
import pytest

import oracle
from hadamard_rotated_bit_gb300 import workloads as wl
from tests._gpu import np_of, torch_bf16, torch_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF, NAN = np.inf, np.nan


@pytest.fixture(scope="module")
def h32():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hadamard_rotated_bit_gb300 as m
    from hadamard_rotated_bit_gb300 import _build
    _build.build()
    return m


def _logits(T, V, seed, bf16=False):
    """fp32 values (representable in bf16 with `bf16`) and the device tensor."""
    import torch
    r = np.random.default_rng(seed)
    l = (2.0 * r.standard_normal((T, V))).astype(np.float32)
    for t in range(T):
        at = r.integers(0, V, min(V, 6))
        l[t, at] = 8 + 3 * r.standard_normal(at.size)
    if bf16:
        bits = wl.f32_to_bf16_bits(l)
        return oracle.bf16_to_f32(bits), torch_bf16(bits)
    return l, torch_of(l)


def _compare(h32, l, t, targets, top, **kw):
    """A thread's sums are at most V / 256 + 32 terms in a row, then joined by fewer than 32
    steps: each rounding U of the sum, each exponential 4 U (argument, instruction) and
    U |l - m| (the argument's rounding, as e^d |d| <= 1 no more than U of the sum);
    log S and the subtractions a few U of their values."""
    import torch
    tt = None if targets is None else torch_of(targets)
    lp, ent, ids, tlp = h32.h32_token_logprobs(t, tt, top=top, **kw)
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    two = None if targets is None else targets.reshape(l.shape[0], -1)
    rlp, rent, rids, rtlp = oracle.token_logprobs(l, two, top)
    T, V = l.shape
    n = V / 256 + 32 + 32 + 8
    mean = np.zeros(T)   # sum p |l - m|
    for i in range(T):
        r = l[i].astype(np.float64)
        if np.isfinite(r.max()):
            e = np.exp(r - r.max())
            mean[i] = (e * np.where(e > 0, r.max() - r, 0)).sum() / e.sum() if np.isfinite(e.sum()) else 0

    def near(got, want, tol):
        got, want = np_of(got).reshape(want.shape).astype(np.float64), want
        assert np.array_equal(np.isnan(got), np.isnan(want))
        odd = ~np.isfinite(want)
        assert np.array_equal(got[odd], want[odd], equal_nan=True)
        err = np.abs(got[~odd] - want[~odd])
        assert (err <= np.broadcast_to(tol, want.shape)[~odd]).all(), err.max()

    fin = lambda a: np.where(np.isfinite(a), np.abs(a), 0)  # noqa: E731
    log_s = np.log(V)
    if targets is not None:
        assert lp.shape == targets.shape
        near(lp, rlp, U * (n + 4 * (2 * fin(rlp) + 2 * log_s)))
    near(ent, rent, U * (2 * n * (1 + mean) + 4 * log_s + 4 * mean))
    if top:
        assert np.array_equal(np_of(ids), rids)
        near(tlp, rtlp, U * (n + 4 * (2 * fin(rtlp) + 2 * log_s)))
    else:
        assert ids is None and tlp is None


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,V,n,top", [(1, 1, 1, 1), (1, 2, 0, 2), (3, 5, 1, 5), (2, 31, 2, 31), (2, 32, 1, 32), (5, 33, 1, 32),
                                       (1, 1000, 1, 20), (4, 1023, 3, 1), (3, 8191, 1, 7), (1, 40000, 1, 32),
                                       (2, 65537, 2, 20), (1, 131072, 5, 20), (9, 100003, 1, 5), (40, 20011, 1, 8),
                                       (700, 1999, 1, 3), (160, 9001, 4, 0)])
def test_random_rows(h32, T, V, n, top, bf16):
    l, t = _logits(T, V, T + V + n, bf16)
    targets = None
    if n:
        targets = np.random.default_rng(1).integers(0, V, (T, n)).astype(np.int32)
        targets[:, 0] = l.argmax(1)
        if T > 2:
            targets[T - 1], targets[0, -1], targets[1, 0] = -1, V, -100
        if n == 1 and T % 2:
            targets = targets[:, 0].copy()
    _compare(h32, l, t, targets, top)


def _odd_rows(V, bf16):
    """16 rows, masked, tied or not finite: values and device tensor."""
    low = float(np.float32(-3.3895314e38))   # bf16's lowest number
    l, _ = _logits(16, V, V, bf16)
    r = np.random.default_rng(0)
    l[0] = -INF                                   # nothing left
    l[1] = -INF
    l[1, V - 1] = -3.0                            # one token left, the last
    l[2, r.random(V) < 0.9] = -INF                # most masked
    l[3] = -INF
    l[3, r.integers(0, V, 7)] = 1.5               # fewer left than asked for
    l[4] = low                                    # a mask of the lowest number
    l[5] = low
    l[5, [2, 17]] = [0.5, -2.0]
    l[6, [1, 30]] = INF
    l[7, 11] = NAN
    l[8] = NAN
    l[9] = -INF
    l[9, [3, 9]] = NAN
    l[10, [4, 20]] = [INF, NAN]
    l[11] = 0.0                                   # all equal
    l[12] = -0.0
    l[12, ::2] = 0.0                              # equal zeros of either sign
    l[13] = 1e4 * l[13].clip(-1, 1)               # wide: one probability is 1
    l[14] = np.linspace(-10, 10, V)               # ascending: every value passes the bound
    l[15] = np.linspace(10, -10, V)
    t = torch_of(l)
    if bf16:
        bits = wl.f32_to_bf16_bits(l)
        t, l = torch_bf16(bits), oracle.bf16_to_f32(bits)
    return l, t


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [40, 3001, 70001])
def test_rows_that_are_masked_or_not_finite(h32, V, bf16):
    l, t = _odd_rows(V, bf16)
    targets = np.stack([np.full(16, 0), np.full(16, V - 1), np.full(16, 11), np.full(16, 3)], 1).astype(np.int32)
    for top in (1, 5, 32):
        _compare(h32, l, t, targets, top)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V,top", [(40, 32), (1999, 3), (3001, 20), (12270, 32)])
def test_many_rows(h32, V, top, bf16):
    """More rows than run at once: each still gets its own results, whatever the rows around it."""
    odd, todd = _odd_rows(V, bf16)
    l, t = _logits(1101, V, V, bf16)
    at = np.random.default_rng(V).permutation(1101)[:32]
    for i in range(2):
        l[at[16 * i:16 * i + 16]] = odd
        t[torch_of(at[16 * i:16 * i + 16].copy())] = todd
    targets = np.random.default_rng(2).integers(-1, V + 1, (1101, 2)).astype(np.int32)
    _compare(h32, l, t, targets, top)


@pytest.mark.parametrize("V", [2000, 50000])
def test_ties_go_to_the_lower_id(h32, V):
    """Few distinct values, so that ties straddle warps, steps and CTAs."""
    for seed, levels in ((0, 2), (1, 5), (2, 40)):
        l = np.random.default_rng(seed).integers(0, levels, (3, V)).astype(np.float32)
        l[1, : V - 40] = 0
        _compare(h32, l, torch_of(l), None, 32)


@pytest.mark.parametrize("bf16", [False, True])
def test_pitches_and_alignments(h32, bf16):
    """Rows that start on any multiple of their type's size."""
    l, _ = _logits(5, 4099, 3, bf16)
    for start in range(0, 9):
        for V in (4090, 17, 3):
            wide = np.full((5, 4099 + 6), NAN, np.float32)
            wide[:, start:start + V] = l[:, :V]
            t = (torch_bf16(wl.f32_to_bf16_bits(wide)) if bf16 else torch_of(wide))[:, start:start + V]
            _compare(h32, l[:, :V], t, np.zeros((5, 1), np.int32), 3)


def test_certain_tokens(h32):
    """log p next to 0 keeps its absolute accuracy, and is never above 0."""
    import torch
    l = np.zeros((3, 5000), np.float32)
    l[0, 7], l[1, 7], l[2, 7] = 20.0, 40.0, 200.0
    _compare(h32, l, torch_of(l), np.full(3, 7, np.int32), 2)
    lp = h32.h32_token_logprobs(torch_of(l), torch.full((3,), 7, dtype=torch.int32, device="cuda"))[0]
    assert bool((lp <= 0).all())


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [1, 200])
def test_a_certain_token_over_a_wide_floor(h32, T, bf16):
    """One likely token and 131071 others whose e^(l - max) = 4.1e-8 is below half a step of the
    sum next to 1: together they are 5.4e-3, however many of them one thread adds up (a CTA or
    more to a row).  The sum's roundings, of about 1 + 5.4e-3 each, do not grow with the row:
    within a step at most 4 of a vector's and 2 of the vectors' sums, 16 of a run's steps, 2 of
    the compensated sum of the runs, 2 of the two halves, then 5 joins of lanes, 7 of warps, 7 of
    CTAs and 1 of the values beside the vectors, one each as the part that is not scaled is the
    large one: 46.  An exponential's own error is 3 |d| + 4 = 55 U of 5.4e-3.
    W = 17 * 5.4e-3 comes of as many joins and, in a run, of at most 256 additions to partial
    sums that are half of the run's on average: 128 U more."""
    V, big, d = 131072, 12.0, 17.0
    l = np.full((T, V), big - d, np.float32)
    at = np.random.default_rng(T).integers(0, V, T)
    at[0] = 0
    l[np.arange(T), at] = big
    bits = wl.f32_to_bf16_bits(l)
    t = torch_bf16(bits) if bf16 else torch_of(l)
    other = (at + 1) % V
    lp, ent, ids, tlp = h32.h32_token_logprobs(t, torch_of(np.stack([at, other], 1).astype(np.int32)), top=2)
    rest = (V - 1) * np.exp(-d)
    log_s = np.log1p(rest)
    assert np.array_equal(np_of(ids), np.stack([at, np.where(at == 0, 1, 0)], 1))
    for got in (np_of(lp), np_of(tlp)):
        err = np.abs(got.astype(np.float64) - [-log_s, -d - log_s])
        print("log p off by, in U:", err.max(0) / U)
        assert (err <= [52 * U, (52 + 2 * d) * U]).all()
    err = np.abs(np_of(ent).astype(np.float64) - (log_s + d * rest / (1 + rest)))
    print("entropy off by, in U:", err.max() / U)
    assert (err <= 52 * (1 + 2 * d * rest) * U + (3 * d + 4 + 128) * d * rest * U).all()


@pytest.mark.parametrize("T,V,bf16", [(267, 65600, False), (300, 70001, False), (304, 131073, True), (305, 131073, True),
                                      (121, 131072, True), (122, 131072, True), (152, 70001, False), (153, 70001, False),
                                      (1063, 40000, False), (1064, 40000, False), (1064, 131072, True),
                                      (1064, 131080, True), (2100, 65536, False), (380, 70001, False), (381, 70001, False),
                                      (1217, 12500, False), (1824, 12500, False)])
def test_row_counts_around_the_choices_of_a_rows_ctas(h32, T, V, bf16):
    """How many CTAs a row is split over and how large they are depend on the number of rows."""
    import torch
    n, top = 7, 6
    l, base = _logits(n, V, T + V, bf16)
    odd = n - 1
    l[odd, : V - 3], base[odd, : V - 3] = -INF, -INF        # fewer left than asked for
    rows = np.random.default_rng(T).integers(0, n, T)
    rows[:n] = np.arange(n)
    targets = np.stack([l.argmax(1), np.full(n, V // 2), np.full(n, V - 1)], 1).astype(np.int32)
    at = torch_of(rows)
    got = h32.h32_token_logprobs(base[at], torch_of(targets)[at], top=top)
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    rlp, rent, rids, rtlp = oracle.token_logprobs(l, targets, top)
    lp, ent, ids, tlp = (np_of(g).astype(np.float64) for g in got)
    assert np.array_equal(ids, rids[rows])
    # at most 64 roundings of the sum and 4 more at each of a thread's rises of its maximum (a few
    # of its up to 64 steps), 3 |l - m| + 4 of an exponential (p |l - m| adds up to less than 3 here),
    # and of the values themselves: 400 U in all for values up to 20
    for g, want in ((lp, rlp[rows]), (ent, rent[rows]), (tlp, rtlp[rows])):
        odd = ~np.isfinite(want)
        assert np.array_equal(g[odd], want[odd], equal_nan=True)
        assert (np.abs(g[~odd] - want[~odd]) <= 400 * U * np.maximum(1, np.abs(want[~odd]) / 20)).all()


def test_given_outputs_streams_and_graphs(h32):
    import torch
    l, t = _logits(6, 30011, 5)
    targets = np.arange(6, dtype=np.int32)
    out = dict(logprob=torch.empty(6, device="cuda"), entropy=torch.full((8,), 9.0, device="cuda"),
               top_id=torch.full((7, 4), 9, dtype=torch.int32, device="cuda"), top_logprob=torch.full((7, 4), 9.0, device="cuda"))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    r = h32.h32_token_logprobs(t, torch_of(targets), top=4, stream=s, **out)
    torch.cuda.synchronize()
    assert r[0] is out["logprob"] and r[2] is out["top_id"]
    plain = h32.h32_token_logprobs(t, torch_of(targets), top=4)
    for a, b in zip(r, plain):
        assert torch.equal(a[:6], b)
    assert bool((out["entropy"][6:] == 9).all()) and bool((out["top_id"][6:] == 9).all())
    tt = torch_of(targets)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c = h32.h32_token_logprobs(t, tt, top=4)
    l2, t2 = _logits(6, 30011, 6)
    t.copy_(t2)
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(c, h32.h32_token_logprobs(t2, tt, top=4)):
        assert torch.equal(a, b)


def test_empty(h32):
    import torch
    lp, ent, ids, tlp = h32.h32_token_logprobs(torch.zeros((0, 50), device="cuda"),
                                               torch.zeros(0, dtype=torch.int32, device="cuda"), top=2)
    assert lp.shape == (0,) and ent.shape == (0,) and ids.shape == (0, 2) and tlp.shape == (0, 2)
    lp, ent, ids, tlp = h32.h32_token_logprobs(torch.zeros((3, 50), device="cuda"),
                                               torch.zeros((3, 0), dtype=torch.int32, device="cuda"))
    assert lp.shape == (3, 0) and ids is None and np.allclose(np_of(ent), np.log(50), rtol=1e-6)
