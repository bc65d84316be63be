"""GPU parity of h32_add_rms_norm_quantize against the CPU oracle: residual rows,
normed rows, codes and scales bit for bit (the sum of squares is taken in a
stated order, so nothing here has a tolerance), in every form, rotation and
type, at ragged sizes, with pitched rows and in place."""
import numpy as np
import pytest

import oracle
from hadamard_rotated_bit_gb300 import workloads as wl
from tests._gpu import np_of, torch_bf16, torch_of
from tests.test_gpu_tc import _q8_codes_from_tc, e4m3_value
from tests.test_gpu_widen import e5m2_value

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


def _rows(M, K, seed, bf16, scale=1.0):
    x = wl.act_normal_outliers(M, K, 0.005, 30.0, seed, wl.CFG_TEST, 2000) * np.float32(scale)
    return wl.f32_to_bf16_bits(x) if bf16 else x


def _dev(a):
    return torch_bf16(a) if a.dtype == np.uint16 else torch_of(a)


def _f32(t):
    return np_of(t.float())


def _same(a, b):
    return np.array_equal(np.ascontiguousarray(a, np.float32).view(np.uint32),
                          np.ascontiguousarray(b, np.float32).view(np.uint32))


def _check_codes(form, xq, xd, n, rotate):
    M, K = n.shape
    xq, xd = np_of(xq), np_of(xd)
    if form in ("q8", "q8_tc"):
        rq, rd = oracle.quantize_act_q8(n, rotate)
        if form == "q8":
            assert np.array_equal(xq[:M], rq)
        else:
            assert np.array_equal(_q8_codes_from_tc(xq[:M], K)[0], rq.astype(np.float64))
    else:
        rq, rd = oracle.quantize_act_q4(n, rotate)
        if form == "q4":
            assert np.array_equal(xq[:M], rq)
        else:
            codes = oracle.decode_act4(rq, K).astype(np.float64)
            got = e4m3_value(xq[:M]) if form == "q4_tc" else e5m2_value(xq[:M]) / 512.0
            assert np.array_equal(got, codes)
    got_d = xd[:M] if form in ("q4", "q8") else xd[:, :M].T
    assert _same(got_d, rd)


def _run(h32, x, w, res, form, rotate, norm_out=None, eps=1e-6, **kw):
    import torch
    out = h32.h32_add_rms_norm_quantize(_dev(x), _dev(w), residual=None if res is None else _dev(res),
                                        eps=eps, form=form, rotate=rotate, norm_out=norm_out, **kw)
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    return out


@pytest.mark.parametrize("form", ["q4", "q8", "q4_tc", "q8_tc", "q4_tc_e5m2"])
@pytest.mark.parametrize("rotate", [0, 32, 64, 128])
def test_every_form_and_rotation(h32, form, rotate):
    import torch
    for M, K in ((1, 5120), (7, 128), (33, 1152)):
        x, res = _rows(M, K, M, False), _rows(M, K, M + 1, True, 2.0)
        w = (1 + 0.1 * np.random.default_rng(K).standard_normal(K)).astype(np.float32)
        xq, xd, ro, nrm = _run(h32, x, w, res, form, rotate, torch.float32)
        h, n = oracle.add_rms_norm(x, w, res)
        assert _same(_f32(ro), h) and ro.dtype == torch.bfloat16
        assert _same(np_of(nrm), n)
        _check_codes(form, xq, xd, n, rotate)


@pytest.mark.parametrize("xb", [False, True])
@pytest.mark.parametrize("rb", [None, False, True])
@pytest.mark.parametrize("wb", [False, True])
def test_types(h32, xb, rb, wb):
    import torch
    M, K = 19, 2048
    x = _rows(M, K, 5, xb)
    res = None if rb is None else _rows(M, K, 6, rb)
    w = (1 + 0.1 * np.random.default_rng(7).standard_normal(K)).astype(np.float32)
    w = wl.f32_to_bf16_bits(w) if wb else w
    for nd in (torch.bfloat16, torch.float32):
        xq, xd, ro, nrm = _run(h32, x, w, res, "q4_tc", 32, nd)
        h, n = oracle.add_rms_norm(x, w, res)
        if rb is None:
            assert ro is None
        else:
            assert _same(_f32(ro), h)
        assert nrm.dtype == nd
        assert _same(_f32(nrm), n if nd == torch.float32 else
                     wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(n)))
        _check_codes("q4_tc", xq, xd, n, 32)


# rows a warp shares (K <= 512), one piece a thread (K <= 8192) with fewer and more
# rows than resident blocks, two pieces (odd halves), the longest row; token counts
# that end inside a block
@pytest.mark.parametrize("M,K", [(1, 32), (300, 32), (31, 64), (9, 96), (65, 224), (5, 992),
                                 (3, 1024), (4, 1056), (2, 17408), (3, 24576), (2, 24608),
                                 (3, 32768), (700, 1280), (5, 512), (9, 544), (2, 8192),
                                 (3, 8224), (2, 16384), (2, 16416), (2000, 4096),
                                 (1900, 1056), (620, 8224), (5000, 96)])
def test_sizes(h32, M, K):
    x, res = _rows(M, K, M + K, True), _rows(M, K, M + K + 1, False)
    w = (1 + 0.1 * np.random.default_rng(K).standard_normal(K)).astype(np.float32)
    for form in ("q8_tc", "q4"):
        xq, xd, ro, _ = _run(h32, x, w, res, form, 32)
        h, n = oracle.add_rms_norm(x, w, res)
        assert _same(np_of(ro), h)
        _check_codes(form, xq, xd, n, 32)


def test_rounding_of_the_code_product(h32):
    """Enough values that some products v * fl(1/d) round onto a tie: the code is that
    of the rounded product, not of the exact one."""
    for form, seed in (("q8", 1), ("q8_tc", 2), ("q4_tc", 3), ("q4", 4)):
        M, K = 220, 4096
        x = _rows(M, K, seed, False)
        w = np.ones(K, np.float32)
        xq, xd, _, _ = _run(h32, x, w, None, form, 32)
        _, n = oracle.add_rms_norm(x, w, None)
        _check_codes(form, xq, xd, n, 32)


def test_zero_tiny_and_overflowing_rows(h32):
    """Rows of zeros, of subnormal size, with a sum of squares above fp32's range
    (beside ordinary rows of the same warp), one-hot rows; eps from 1e-30 to 1."""
    import torch
    for K in (128, 5120):
        x = _rows(12, K, 3, False)
        x[1] = 0.0
        x[2] *= np.float32(1e-30)
        x[3] *= np.float32(2.0 ** 90)
        x[5] = 0.0
        x[5, 7] = 3.0
        x[6] *= np.float32(2.0 ** 60)
        x[7] = np.float32(2.0 ** -140)
        w = np.ones(K, np.float32)
        for eps in (1e-30, 1e-6, 1.0):
            xq, xd, _, nrm = _run(h32, x, w, None, "q8", 32, torch.float32, eps=eps)
            _, n = oracle.add_rms_norm(x, w, None, eps)
            assert np.isfinite(n).all() and _same(np_of(nrm), n)
            _check_codes("q8", xq, xd, n, 32)


def test_pitched_rows_in_place_and_untouched_surroundings(h32):
    """Inputs and outputs as column ranges of wider arrays, the residual updated in
    place, larger code and scale arrays: nothing outside the rows changes."""
    import torch
    M, K = 21, 640
    x, res = _rows(M, K, 8, False), _rows(M, K, 9, True)
    w = np.ones(K, np.float32)
    wide_x = torch.full((M + 3, K + 64), 7.0, device="cuda")
    wide_x[:M, :K] = torch_of(x)
    wide_r = torch.full((M + 2, K + 128), 5.0, device="cuda", dtype=torch.bfloat16)
    wide_r[:M, 64:64 + K] = torch_bf16(res)
    wide_n = torch.full((M + 1, K + 32), 3.0, device="cuda")
    xq = torch.full((M + 4, K), 99, dtype=torch.uint8, device="cuda")
    xd = torch.full((K // 32 + 1, 28), -1.0, device="cuda")
    r_view = wide_r[:M, 64:64 + K]
    out = h32.h32_add_rms_norm_quantize(wide_x[:M, :K], torch_of(w), residual=r_view,
                                        residual_out=r_view, norm_out=wide_n[:, :K], xq=xq, xd=xd)
    torch.cuda.synchronize()
    assert out[0] is xq and out[1] is xd and out[2] is r_view
    h, n = oracle.add_rms_norm(x, w, res)
    assert _same(_f32(r_view), h) and _same(np_of(wide_n[:M, :K]), n)
    _check_codes("q4_tc", xq, xd[:K // 32], n, True)
    assert torch.all(wide_r[:, :64] == 5) and torch.all(wide_r[:, 64 + K:] == 5)
    assert torch.all(wide_r[M:] == 5) and torch.all(wide_n[M:] == 3) and torch.all(wide_n[:, K:] == 3)
    assert torch.all(xq[M:] == 99) and torch.all(xd[:, M:] == -1) and torch.all(xd[K // 32:] == -1)
    assert torch.all(wide_x[:, K:] == 7) and torch.all(wide_x[M:] == 7)


def test_outputs_over_inputs(h32):
    """residual_out over x (of the residual's type) and norm_out over x or the residual."""
    import torch
    M, K = 40, 1024
    x, res = _rows(M, K, 11, True), _rows(M, K, 12, True)
    w = np.ones(K, np.float32)
    h, n = oracle.add_rms_norm(x, w, res)
    nb = wl.bf16_bits_to_f32(wl.f32_to_bf16_bits(n))
    xt, rt = torch_bf16(x), torch_bf16(res)
    h32.h32_add_rms_norm_quantize(xt, torch_of(w), residual=rt, residual_out=xt, norm_out=rt)
    assert _same(_f32(xt), h) and _same(_f32(rt), nb)
    xt, rt = torch_bf16(x), torch_bf16(res)
    out = h32.h32_add_rms_norm_quantize(xt, torch_of(w), residual=rt, residual_out=False,
                                        norm_out=xt, form=None)
    assert out == (None, None, None, xt) and _same(_f32(xt), nb) and _same(_f32(rt), wl.bf16_bits_to_f32(res))


def test_empty_stream_and_graph(h32):
    """M = 0; a call on another stream; a captured call replayed on new contents."""
    import torch
    K = 512
    w = torch.ones(K, device="cuda")
    xq, xd, ro, _ = h32.h32_add_rms_norm_quantize(torch.empty((0, K), device="cuda"), w,
                                                  residual=torch.empty((0, K), device="cuda"))
    assert xq.shape == (0, K) and ro.shape == (0, K)
    x = torch_of(_rows(33, K, 1, False))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a = h32.h32_add_rms_norm_quantize(x, w, stream=s)
    b = h32.h32_add_rms_norm_quantize(x, w, stream=s.cuda_stream)
    s.synchronize()
    _, n = oracle.add_rms_norm(np_of(x), np_of(w))
    _check_codes("q4_tc", a[0], a[1], n, 32)
    _check_codes("q4_tc", b[0], b[1], n, 32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        xq, xd, _, _ = h32.h32_add_rms_norm_quantize(x, w)
    for seed in (4, 5):
        x.copy_(torch_of(_rows(33, K, seed, False)))
        g.replay()
        torch.cuda.synchronize()
        _, n = oracle.add_rms_norm(np_of(x), np_of(w))
        _check_codes("q4_tc", xq, xd, n, 32)
    assert h32.h32_device_status() == 0


def test_wait_that_gives_up_is_reported(h32):
    """A bound of one poll on the wait for a row's copy: the status reads timeout (or, as
    a poll is itself a short wait in hardware, nothing), once, and the same context
    then computes exact results."""
    import torch
    M, K = 2000, 1024
    x, w = _rows(M, K, 21, True), np.ones(K, np.float32)
    xt, wt = torch_bf16(x), torch_of(w)
    h32.h32_set_wait_limit(1)
    try:
        h32.h32_add_rms_norm_quantize(xt, wt)
        assert h32.h32_device_status() in (0, h32.H32_ERR_TIMEOUT)
    finally:
        h32.h32_set_wait_limit(0)
    assert h32.h32_device_status() == 0
    xq, xd, _, _ = _run(h32, x, w, None, "q4_tc", 32)
    _, n = oracle.add_rms_norm(x, w)
    _check_codes("q4_tc", xq, xd, n, 32)


@pytest.mark.parametrize("K", [96, 512, 5120, 12288])
def test_huge_eps(h32, K):
    """eps beside rows whose sum of squares leaves fp32's range, and beside small ones."""
    import torch
    for M in (5, 40):
        x = _rows(M, K, K, False)
        x[1] *= np.float32(2.0 ** 60)
        x[2] *= np.float32(2.0 ** 66)
        x[3] *= np.float32(2.0 ** 90)
        w = np.ones(K, np.float32)
        for eps in (1e30, 1e36, 1e38, 3.4028234e38):
            xq, xd, _, nrm = _run(h32, x, w, None, "q8", 32, torch.float32, eps=eps)
            _, n = oracle.add_rms_norm(x, w, None, eps)
            assert np.isfinite(n).all() and _same(np_of(nrm), n)
            _check_codes("q8", xq, xd, n, 32)
