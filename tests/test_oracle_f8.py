"""Pins of the oracle's 8-bit floating-point codes, products and log probabilities:
independent evaluations and closed forms, no GPU."""
import numpy as np
import pytest
import torch

import oracle


def test_e4m3_values_and_rounding():
    v = oracle.e4m3_values()
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, want, equal_nan=True)
    r = np.random.default_rng(0)
    q = np.concatenate([r.standard_normal(20000) * 10.0 ** r.uniform(-4, 2.5, 20000),
                        (v[:126] + v[1:127]) / 2, -(v[:126] + v[1:127]) / 2, v[:127], [0.0, -0.0]])
    q = q[np.abs(q) <= 448].astype(np.float32)
    got = oracle.e4m3_round(q)
    want = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(got, want)
    assert list(oracle.e4m3_round([449.0, 1e30, -np.inf, np.nan])) == [126, 126, 254, 127]


def test_quantizers_by_hand():
    # amax 448 in each group: d = 1, the codes are the values; the second group is scaled by 2
    x = np.zeros((2, 160), np.float32)
    x[0, :4] = [448, -17, 18.999, 0.0029]
    x[0, 128:131] = [896, 3, -1]
    q, d = oracle.quantize_act_f8(x)
    assert d.tolist() == [[1.0, 2.0], [0.0, 0.0]]
    v = oracle.e4m3_values()[q]
    assert v[0, :4].tolist() == [448, -16, 18, 3 * 2.0 ** -10 * 0 + 2.0 ** -9]
    assert v[0, 128:131].tolist() == [448, 1.5, -0.5] and not v[1].any()
    wq, wd = oracle.quantize_weights_f8(np.concatenate([np.zeros((128, 160), np.float32), x]))
    assert wd.tolist() == [[0.0, 0.0], [1.0, 2.0]] and np.array_equal(wq[128:], q)


@pytest.mark.parametrize("rotate", [0, 32, 64, 128])
def test_reconstruction(rotate):
    """Codes times scale are within half an e4m3 step of the rotated values."""
    x = np.random.default_rng(rotate).standard_normal((5, 384)).astype(np.float32)
    v = oracle.fwht_n_f64(x, rotate) if rotate else x.astype(np.float64)
    q, d = oracle.quantize_act_f8(x, rotate)
    got = oracle.e4m3_values()[q] * np.repeat(d.astype(np.float64), 128, 1)
    step = np.maximum(np.abs(v) * 2.0 ** -4, np.repeat(d, 128, 1) * 2.0 ** -10)
    assert (np.abs(got - v) <= step * (1 + 1e-5) + 1e-5).all()


def test_gemm_against_blocks():
    r = np.random.default_rng(1)
    wq, xq = r.integers(0, 127, (200, 288), np.uint8), r.integers(128, 255, (3, 288), np.uint8)
    wd, xd = r.random((2, 3), np.float32), r.random((3, 3), np.float32)
    y, t = oracle.f8_gemm(wq, wd, xq, xd)
    val = oracle.e4m3_values()
    for m, n in ((0, 0), (1, 127), (2, 128), (2, 199)):
        s = [(val[xq[m, 128 * b:128 * b + 128]] * val[wq[n, 128 * b:128 * b + 128]]).sum() for b in range(3)]
        want = sum(float(xd[m, b]) * float(wd[n // 128, b]) * s[b] for b in range(3))
        assert abs(y[m, n] - want) <= 1e-12 * t[m, n]


def test_logprobs_against_torch_and_closed_forms():
    l = np.random.default_rng(2).standard_normal((6, 50)).astype(np.float32) * 3
    lp, ent, ids, tlp = oracle.token_logprobs(l, np.array([[3, -1]] * 6), 7)
    ref = torch.log_softmax(torch.from_numpy(l).double(), 1)
    assert np.allclose(lp[:, 0], ref[:, 3].numpy(), rtol=1e-13) and not lp[:, 1].any()
    assert np.allclose(ent, torch.distributions.Categorical(logits=torch.from_numpy(l).double()).entropy().numpy())
    want = torch.sort(torch.from_numpy(l), dim=1, descending=True, stable=True).indices[:, :7].numpy()
    assert np.array_equal(ids, want) and np.allclose(tlp, np.take_along_axis(ref.numpy(), ids, 1))
    inf, nan = np.inf, np.nan
    e = np.array([[0, 0, 0, 0], [-inf] * 4, [inf, 1, inf, -inf], [1, nan, 2, -inf], [5, -inf, -inf, -inf]], np.float32)
    lp, ent, ids, tlp = oracle.token_logprobs(e, np.array([[0, 3, 4]] * 5), 4)
    assert ids.tolist() == [[0, 1, 2, 3], [0, 1, 2, 3], [0, 2, 1, 3], [2, 0, 3, 1], [0, 1, 2, 3]]
    assert np.allclose(ent[:3], [np.log(4), 0, np.log(2)]) and np.isnan(ent[3]) and ent[4] == 0
    assert np.allclose(lp[0, :2], -np.log(4)) and lp[1, :2].tolist() == [-inf, -inf]
    assert np.allclose(lp[2, 0], -np.log(2)) and lp[2, 1] == -inf and np.isnan(lp[3, 0])
    assert lp[4, :2].tolist() == [0, -inf] and np.isnan(lp[:, 2]).all()
