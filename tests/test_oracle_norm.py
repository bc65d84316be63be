"""Pins for the oracle's residual addition and root-mean-square norm, against
float64 and closed forms (the norm itself; its quantized output is the
quantizers', pinned on their own)."""
import numpy as np
import pytest

import oracle
from hadamard_rotated_bit_gb300 import workloads as wl

U = 2.0 ** -24   # half a step of fp32


@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (5, 1024), (2, 1056), (4, 5120), (2, 17408)])
def test_norm_against_float64(M, K):
    """n within the forward bound: an 8-term fma chain, one sum and two 5-level trees
    (and one more sum above 16384 values) keep the sum of squares (all positive)
    within 8 + 1 + 10 + 1 half steps, fl(1/K), its product and the sum with eps add
    3, the root halves them; the reciprocal root and two products add 3."""
    r = np.random.default_rng(M * K)
    x = (r.standard_normal((M, K)) * 3).astype(np.float32)
    res = (r.standard_normal((M, K)) * 2).astype(np.float32)
    w = (1 + 0.1 * r.standard_normal(K)).astype(np.float32)
    h, n = oracle.add_rms_norm(x, w, res, 1e-6)
    assert np.array_equal(h, x + res)
    h64 = h.astype(np.float64)
    want = h64 / np.sqrt((h64 ** 2).mean(1, keepdims=True) + np.float64(np.float32(1e-6))) * w
    bound = ((8 + 1 + 10 + 1 + 3) / 2 + 3) * U * (1 + 1e-4)
    assert np.all(np.abs(n - want) <= bound * np.abs(want))


def test_bf16_residual_is_rounded_before_the_norm():
    r = np.random.default_rng(1)
    x = r.standard_normal((4, 256)).astype(np.float32)
    res = wl.f32_to_bf16_bits(r.standard_normal((4, 256)).astype(np.float32))
    h, n = oracle.add_rms_norm(x, np.ones(256, np.float32), res)
    stored = wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(x + wl.bf16_bits_to_f32(res)))
    assert np.array_equal(h, stored) and not np.array_equal(h, x + wl.bf16_bits_to_f32(res))
    _, n2 = oracle.add_rms_norm(stored, np.ones(256, np.float32), None)
    assert np.array_equal(n, n2)


def test_closed_forms():
    one = np.ones(64, np.float32)
    # constant rows: mean square exact, r = 1/c
    h, n = oracle.add_rms_norm(np.full((1, 64), 4.0, np.float32), one, None, 1e-30)
    assert np.all(n == 1.0)
    # zero rows: n = 0 whatever r = 1/sqrt(eps) is
    _, n = oracle.add_rms_norm(np.zeros((1, 64), np.float32), one, None, 1e-30)
    assert np.all(n == 0.0)
    # a sum of squares above fp32's range: the row is scaled first
    big = np.full((1, 64), 2.0 ** 100, np.float32)
    big[0, 1] = -(2.0 ** 100)
    _, n = oracle.add_rms_norm(big, one, None, 1e-6)
    assert n[0, 0] == 1.0 and n[0, 1] == -1.0


def test_sum_order_is_the_stated_one():
    """Terms of a quarter step are lost one by one but kept when their piece, or
    their place's chain, is summed first."""
    x = np.zeros((1, 64), np.float32)
    x[0, 0] = 1.0
    x[0, 2:16:2] = 2.0 ** -13      # squares 2^-26 (a quarter step): lost in the chain of 1
    x[0, 1:16:2] = 2.0 ** -13      # the odd places' chain: 8 * 2^-26 = 2^-23, then joins
    x[0, 16:32] = 2.0 ** -13       # the next piece: 2^-22
    _, n = oracle.add_rms_norm(x, np.ones(64, np.float32), None, 1e-30)
    s = np.float32(1.0 + 2.0 ** -23 + 2.0 ** -22)
    r = np.float32(1 / np.sqrt(np.float64(s / np.float32(64))))
    assert n[0, 0] == r and s != 1
    # trees: 32 pieces a group, 32 groups, then in order
    K = 16384 + 32
    y = np.zeros((1, K), np.float32)
    y[0, 0] = 4096.0               # 2^24: a 1 joins a tree neighbour before it
    y[0, 16384] = y[0, 16384 + 16] = 1.0
    _, n = oracle.add_rms_norm(y, np.ones(K, np.float32), None, 1e-30)
    s = np.float32(2.0 ** 24 + 2.0)
    ms = s * (np.float32(1) / np.float32(K))
    assert n[0, 16384] == np.float32(1 / np.sqrt(np.float64(ms)))


@pytest.mark.parametrize("K", [32, 512, 5120, 17408])
def test_overflowing_rows_keep_their_eps(K):
    """Rows whose sum of squares leaves fp32's range, and rows whose mean square does with
    eps: the formula in float64, eps included, within the same bound."""
    r = np.random.default_rng(K)
    x = (r.choice((-1.0, 1.0), (4, K)) * (1 + r.random((4, K)))).astype(np.float32)
    x *= (2.0 ** np.array([57, 62, 64, 70]))[:, None].astype(np.float32)
    w = np.ones(K, np.float32)
    with np.errstate(over="ignore"):
        assert np.isinf((x.astype(np.float32) ** 2).sum(1)[2:]).all()
    for eps in (1e-6, 1.0, 1e30, 1e36, 1e38, 3.4028234e38):
        _, n = oracle.add_rms_norm(x, w, None, eps)
        x64 = x.astype(np.float64)
        want = x64 / np.sqrt((x64 ** 2).mean(1, keepdims=True) + np.float64(np.float32(eps)))
        bound = ((8 + 1 + 10 + 1 + 3) / 2 + 3) * U * (1 + 1e-4)
        assert np.all(np.abs(n - want) <= bound * np.abs(want))
