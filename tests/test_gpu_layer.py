"""The operators around the products run together, as a decoder layer uses them:
residual + norm + quantizer -> gate/up with SwiGLU -> quantizer -> down with the
residual -> norm; and norm -> router by scores -> gather-quantizer -> expert GEMM ->
combine.  Every step is held to the oracle on the very values the step before it
left on the device, so nothing accumulates; the whole is also replayed from a graph."""
import numpy as np
import pytest

import oracle
from hadamard_rotated_bit_gb300 import workloads as wl
from tests._gpu import np_of, torch_bf16, torch_of
from tests.test_gpu_gemm_epilogue import _compare
from tests.test_gpu_norm import _check_codes, _f32, _same
from tests.test_gpu_tc import e4m3_value

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


def _weights(h32, N, K, tid):
    wq, wd = oracle.quantize_weights_q4_0(wl.weights_normal(N, K, 0.05, 0, wl.CFG_TEST, tid))
    return (wq, wd), h32.h32_prepack_weights_q4_0_tc(torch_of(wq), torch_of(wd.view(np.int16)))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 7, 16, 17, 130])
def test_dense_layer(h32, bits, M):
    import torch
    K, F = 512, 256
    form = "q4_tc" if bits == 4 else "q8_tc"
    quant = h32.h32_quantize_act_q4_tc if bits == 4 else h32.h32_quantize_act_q8_tc
    gemm = h32.q4_0_x_q4_gemm_tc_epilogue if bits == 4 else h32.q4_0_x_q8_gemm_tc_epilogue
    oq = oracle.quantize_act_q4 if bits == 4 else oracle.quantize_act_q8
    gu, gu_t = _weights(h32, 2 * F, K, 4000)    # gate and up rows interleaved
    dn, dn_t = _weights(h32, K, F, 4001)
    w1 = (1 + 0.1 * np.random.default_rng(0).standard_normal(K)).astype(np.float32)
    x0 = wl.act_normal_outliers(M, K, 0.005, 30.0, M, wl.CFG_TEST, 4002)
    r0 = wl.f32_to_bf16_bits(wl.act_normal_outliers(M, K, 0.005, 30.0, M, wl.CFG_TEST, 4003))
    x, w1t = torch_of(x0), torch_of(w1)

    def layer(res):
        xq, xd, r1, _ = h32.h32_add_rms_norm_quantize(x, w1t, residual=res, form=form)
        g = gemm(*gu_t, xq, xd, act="swiglu", y_dtype=torch.bfloat16)
        gq, gd = quant(g)
        out = gemm(*dn_t, gq, gd, residual=r1, y_dtype=torch.bfloat16)
        nq, nd, _, nrm = h32.h32_add_rms_norm_quantize(out, w1t, form=form, norm_out=torch.float32)
        return xq, xd, r1, g, gq, gd, out, nq, nd, nrm

    xq, xd, r1, g, gq, gd, out, nq, nd, nrm = layer(torch_bf16(r0))
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    h, n = oracle.add_rms_norm(x0, w1, r0)
    assert _same(_f32(r1), h)
    _check_codes(form, xq, xd, n, True)
    q, d = oq(n)
    z, _, _ = oracle.gemm(*gu, q, d, K)
    _compare(_f32(g), z, None, "swiglu", None, True)
    q, d = oq(wl.f32_to_bf16_bits(_f32(g)))
    z, _, _ = oracle.gemm(*dn, q, d, F)
    _compare(_f32(out), z, None, "none", r1, True)
    _, n2 = oracle.add_rms_norm(wl.f32_to_bf16_bits(_f32(out)), w1)
    assert _same(np_of(nrm), n2)
    _check_codes(form, nq, nd, n2, True)

    # the same from a graph, on a stream of its own, for other residuals
    res = torch_bf16(r0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(res)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        captured = layer(res)
    for seed in (1, 2):
        other = torch_bf16(wl.f32_to_bf16_bits(wl.act_normal_outliers(M, K, 0.005, 30.0, seed, wl.CFG_TEST, 4004)))
        res.copy_(other)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        eager = layer(other)
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            if a is captured[1] or a is captured[5] or a is captured[8]:
                a, b = a[:, :M], b[:, :M]       # scales: the padding is left as it was
            assert torch.equal(a, b)
    assert h32.h32_device_status() == 0


@pytest.mark.parametrize("T", [1, 40, 300])
def test_expert_layer(h32, T):
    import torch
    K, N, E, k = 256, 64, 16, 3
    w = wl.weights_normal(E * N, K, 0.05, 0, wl.CFG_TEST, 4010)
    wq, wd = oracle.quantize_weights_q4_0(w)
    wp, wsc = h32.h32_prepack_weights_q4_0_tc(torch_of(wq), torch_of(wd.view(np.int16)))
    x = wl.f32_to_bf16_bits(wl.act_normal_outliers(T, K, 0.01, 20.0, T, wl.CFG_TEST, 4011))
    gate = np.random.default_rng(1).standard_normal((K, E)).astype(np.float32) * np.float32(0.1)
    bias = np.random.default_rng(2).standard_normal(E).astype(np.float32) * np.float32(0.05)
    ones = np.ones(K, np.float32)
    _, _, _, nrm = h32.h32_add_rms_norm_quantize(torch_bf16(x), torch_of(ones), form=None,
                                                 norm_out=torch.bfloat16)
    logits = nrm.float() @ torch_of(gate)
    route = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, scale=2.5)
    ids, tw, off, ridx, row_of = h32.h32_moe_route_scored(logits, k, bias=torch_of(bias), **route)
    xw, xdt = h32.h32_quantize_act_q4_tc_gather(nrm, ridx)
    y = h32.q4_0_x_q4_gemm_tc_experts(wp, wsc, xw, xdt, off, N, R=T * k)
    out = h32.h32_moe_combine(y, row_of, tw)
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    _, n = oracle.add_rms_norm(x, ones)
    nb = wl.f32_to_bf16_bits(n)
    assert _same(_f32(nrm), wl.bf16_bits_to_f32(nb))
    rid, rw, roff, rridx, rrow = oracle.moe_route_scored(np_of(logits), k, bias=bias, **route)
    assert np.array_equal(np_of(ids), rid) and np.array_equal(np_of(off), roff)
    assert np.array_equal(np_of(ridx), rridx) and np.array_equal(np_of(row_of), rrow)
    rq, rd = oracle.quantize_act_q4(nb)
    assert np.array_equal(e4m3_value(np_of(xw)), oracle.decode_act4(rq, K).astype(np.float64)[rridx])
    R = T * k
    ri, ni = np.repeat(np.arange(R), N), np.tile(np.arange(N), R)
    ry, _, _ = oracle.gemm_experts_sampled(wq.reshape(E, N, K // 2), wd.reshape(E, N, K // 32), rq, rd,
                                           rridx, roff, N, K, ri, ni)
    assert _same(np_of(y), ry.reshape(R, N))
    assert _same(np_of(out), oracle.moe_combine(ry.reshape(R, N), rrow, np_of(tw)))
