"""The 8-bit floating-point operators run together, as the end of a prompt and an expert layer
use them: norm -> quantizer -> head product -> log probabilities; and norm -> router by
scores -> gathering quantizer -> expert product -> combine.  Every step is held to the
oracle on the very values the step before it left on the device, so nothing accumulates;
the whole is also replayed from a graph."""
import numpy as np
import pytest

import oracle
from hadamard_rotated_bit_gb300 import workloads as wl
from tests._gpu import np_of, torch_bf16, torch_of
from tests.test_gpu_f8 import U
from tests.test_gpu_logprobs import _compare as compare_logprobs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h32():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hadamard_rotated_bit_gb300 as m
    from hadamard_rotated_bit_gb300 import _build
    _build.build()
    return m


def _near_product(y, wq, wd, xq, xd, rows=None):
    """Within the roundings of a product of random codes (see test_gpu_f8)."""
    ref, mag = oracle.f8_gemm(wq, wd, xq, xd)
    nb = wd.shape[1]
    assert (np.abs(y.astype(np.float64) - ref) <= (256 + nb + 2) * U * mag).all()


@pytest.mark.parametrize("rotate", [0, 128])
@pytest.mark.parametrize("M", [1, 19, 70, 300])
def test_head(h32, M, rotate):
    import torch
    K, V, top = 512, 3001, 6
    w = wl.weights_normal(V, K, 0.05, 0, wl.CFG_TEST, 6000)
    wq, wd = h32.h32_quantize_weights_f8(torch_of(w), rotate=rotate)
    rwq, rwd = oracle.quantize_weights_f8(w, rotate)
    assert np.array_equal(np_of(wq), rwq) and np.array_equal(np_of(wd), rwd)
    wn = (1 + 0.1 * np.random.default_rng(0).standard_normal(K)).astype(np.float32)
    x0 = wl.act_normal_outliers(M, K, 0.005, 30.0, M, wl.CFG_TEST, 6001)
    targets = np.random.default_rng(1).integers(0, V, M).astype(np.int32)
    if M > 1:
        targets[-1] = -1
    x, wnt, tt = torch_of(x0), torch_of(wn), torch_of(targets)

    def head():
        _, _, _, n = h32.h32_add_rms_norm_quantize(x, wnt, form=None, norm_out=torch.bfloat16)
        q, d = h32.h32_quantize_act_f8(n, rotate=rotate)
        l = h32.h32_f8_gemm(wq, wd, q, d)
        return (n, q, d, l) + h32.h32_token_logprobs(l, tt, top=top)

    def check(n, q, d, l, lp, ent, ids, tlp):
        rq, rd = oracle.quantize_act_f8(np_of(n.view(torch.int16)).view(np.uint16), rotate)
        assert np.array_equal(np_of(q), rq) and np.array_equal(np_of(d)[:, :M].T, rd)
        _near_product(np_of(l), rwq, rwd, rq, rd)
        compare_logprobs(h32, np_of(l), l, targets, top)
        again = h32.h32_token_logprobs(l, tt, top=top)
        assert all(torch.equal(a, b) for a, b in zip((lp, ent, ids, tlp), again))

    first = head()
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    check(*first)
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = head()
    for seed in (1, 2):
        x.copy_(torch_of(wl.act_normal_outliers(M, K, 0.005, 30.0, seed, wl.CFG_TEST, 6002)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(*captured)
    assert not torch.equal(captured[3], first[3])


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (90, 6, 3), (257, 3, 2)])
def test_expert_layer(h32, T, E, k):
    import torch
    K, N = 384, 260
    w = wl.weights_normal(E * N, K, 0.05, 0, wl.CFG_TEST, 6010)
    planes = [oracle.quantize_weights_f8(w[e * N:(e + 1) * N], 64) for e in range(E)]
    quant = [h32.h32_quantize_weights_f8(torch_of(w[e * N:(e + 1) * N].copy()), rotate=64) for e in range(E)]
    wq, wd = torch.cat([q for q, _ in quant]), torch.cat([d for _, d in quant])
    assert np.array_equal(np_of(wq), np.concatenate([q for q, _ in planes]))
    xb = wl.f32_to_bf16_bits(wl.act_normal_outliers(T, K, 0.005, 30.0, 3, wl.CFG_TEST, 6011))
    logits = np.random.default_rng(T).standard_normal((T, E)).astype(np.float32)
    ids, tw, off, ridx, row_of = h32.h32_moe_route_scored(torch_of(logits), k)
    q, d = h32.h32_quantize_act_f8(torch_bf16(xb), rotate=64, row_idx=ridx)
    y = h32.h32_f8_gemm_experts(wq, wd, q, d, off, N)
    out = h32.h32_moe_combine(y, row_of, tw)
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    rq, rd = oracle.quantize_act_f8(xb[np_of(ridx)], 64)
    assert np.array_equal(np_of(q), rq) and np.array_equal(np_of(d)[:, :T * k].T, rd)
    o = np_of(off)
    for e in range(E):
        r = slice(o[e], o[e + 1])
        _near_product(np_of(y)[r], *planes[e], rq[r], rd[r])
    assert np.array_equal(np_of(out), oracle.moe_combine(np_of(y), np_of(row_of), np_of(tw)))
