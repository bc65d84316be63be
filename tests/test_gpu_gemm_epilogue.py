"""GPU parity of q4_0_x_q{4,8}_gemm_tc_epilogue: z is the oracle's fp32 product, bit
for bit, seen through act "none" without a residual; with bias, activation and
residual the output is compared with the formula in float64 on that z (fp32 bias
addition included, which is one exact IEEE rounding), within the roundings the
kernel makes, counted in half steps of fp32 (h = 2^-24), relative to v:
  relu, none   0
  silu         expf 2 ulp = 4, add 1, divide 1                        -> 6
  swiglu       silu, one product                                      -> 7
  gelu_tanh    as silu, and its argument t: |t| (constants 2, three products and an
               fma 4) in the exponent                                 -> 6 + 6 |t|
  gelu_erf     erfcf 4 ulp = 8, two products 2 (0.5 exact), the argument x (constant
               and product: 2) times |x erfc'(x) / erfc(x)| <= 2 x^2 + 2 -> 10 + 2 (2 x^2 + 2)
then the residual's addition (one half step of y) and the rounding to y's type
(fp32: none beyond; bf16: 2^-8 of y).  A factor 1 + 2^-10 covers second order terms;
floor 2^-120 where results vanish."""
import numpy as np
import pytest

import oracle
from hadamard_rotated_bit_gb300 import workloads as wl
from tests._gpu import np_of, torch_of

pytestmark = pytest.mark.gpu

H = 2.0 ** -24


@pytest.fixture(scope="module")
def h32():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hadamard_rotated_bit_gb300 as m
    from hadamard_rotated_bit_gb300 import _build
    _build.build()
    return m


def _operands(h32, M, N, K, bits, seed=0):
    x = wl.act_normal_outliers(M, K, 0.01, 20.0, seed, wl.CFG_TEST, 3000)
    w = wl.weights_normal(N, K, 0.02, seed, wl.CFG_TEST, 3001)
    wq, wd = oracle.quantize_weights_q4_0(w)
    q = oracle.quantize_act_q4 if bits == 4 else oracle.quantize_act_q8
    xq, xd = q(x)
    z, _, _ = oracle.gemm(wq, wd, xq, xd, K)
    wp, wsc = h32.h32_prepack_weights_q4_0_tc(torch_of(wq), torch_of(wd.view(np.int16)))
    qt = h32.h32_quantize_act_q4_tc if bits == 4 else h32.h32_quantize_act_q8_tc
    xw, xdt = qt(torch_of(x))
    return z, (wp, wsc, xw, xdt)


def _erfc(x):
    import torch
    return torch.special.erfc(torch.from_numpy(x)).numpy()


def _formula(z, act):
    """(v, allowed half steps relative to v) in float64 of fp32 z."""
    z = z.astype(np.float64)
    with np.errstate(over="ignore"):
        if act == "relu":
            return np.maximum(z, 0.0), 0.0
        if act == "silu":
            return z / (1 + np.exp(-z)), 6.0
        if act == "swiglu":
            g, u = z[:, 0::2], z[:, 1::2]
            return g / (1 + np.exp(-g)) * u, 7.0
        if act == "gelu_tanh":
            t = 2 * np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)
            return z / (1 + np.exp(-t)), 6 + 6 * np.abs(t)
        if act == "gelu_erf":
            x = -z / np.sqrt(2.0)
            return 0.5 * z * _erfc(x), 10 + 2 * (2 * x * x + 2)
    return z, 0.0


def _check(h32, z, ops, bits, M=None, bias=None, act="none", res=None, y_bf16=False, **kw):
    import torch
    call = h32.q4_0_x_q4_gemm_tc_epilogue if bits == 4 else h32.q4_0_x_q8_gemm_tc_epilogue
    y = call(*ops, M=M, bias=None if bias is None else torch_of(bias), act=act, residual=res,
             y_dtype=None if kw.get("y") is not None else (torch.bfloat16 if y_bf16 else torch.float32),
             **kw)
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0
    _compare(np_of(y.float())[:z.shape[0]], z, bias, act, None if res is None else kw.pop("res0", res),
             y_bf16)
    return y


def _compare(got, z, bias, act, res, y_bf16):
    zb = z if bias is None else z + bias   # fp32, one rounding
    v, steps = _formula(zb, act)
    r = 0.0 if res is None else np_of(res.float()).astype(np.float64)[:z.shape[0], :v.shape[1]]
    want = v + r
    got = got[:, :v.shape[1]]
    assert np.isfinite(got).all()
    if act in ("none", "relu") and res is None and not y_bf16:
        assert np.array_equal(got.astype(np.float64), v)
        return
    tol = steps * H * np.abs(v) + (H * np.abs(want) if res is not None else 0.0)
    if y_bf16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(got - want) <= tol * (1 + 2.0 ** -10) + 2.0 ** -120)


ACTS = ["none", "relu", "silu", "gelu_tanh", "gelu_erf", "swiglu"]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [1, 3, 40])
def test_every_activation(h32, bits, act, M):
    import torch
    N, K = 208, 384
    z, ops = _operands(h32, M, N, K, bits, M)
    r = np.random.default_rng(M)
    n_out = N // 2 if act == "swiglu" else N
    bias = r.standard_normal(N).astype(np.float32)
    res = torch_of(r.standard_normal((M, n_out)).astype(np.float32))
    for b in (None, bias):
        for rs in (None, res, res.bfloat16()):
            for yb in (False, True):
                _check(h32, z, ops, bits, bias=b, act=act, res=rs, y_bf16=yb)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [2, 40])
def test_nan_stays_where_it_is(h32, act, M):
    """A NaN of the bias comes out of its own outputs, and of no others."""
    import torch
    N, K = 64, 128
    z, ops = _operands(h32, M, N, K, 4, 3)
    bias = np.zeros(N, np.float32)
    bias[[5, 32]] = np.nan
    y = h32.q4_0_x_q4_gemm_tc_epilogue(*ops, M=M, bias=torch_of(bias), act=act)
    torch.cuda.synchronize()
    want = np.zeros(N // 2 if act == "swiglu" else N, bool)
    want[[2, 16] if act == "swiglu" else [5, 32]] = True
    assert np.array_equal(np.isnan(np_of(y)), np.broadcast_to(want, y.shape))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu_erf", "swiglu"])
def test_activation_range(h32, bits, act):
    """Arguments from -200 to 200 through the bias: saturated and vanishing results."""
    N, K = 256, 128
    z, ops = _operands(h32, 2, N, K, bits, 9)
    bias = np.linspace(-200, 200, N).astype(np.float32)
    if act == "swiglu":
        bias[1::2] = 1.5
    _check(h32, z, ops, bits, bias=bias, act=act)


# one token to many, odd counts around the few-token limit and the tile widths;
# ragged last weight tiles; one K stage to many; the split of the last wave
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 5120, 1024), (2, 48, 640), (4, 144, 2176),
                                   (5, 272, 256), (7, 128, 128), (8, 160, 512), (9, 96, 384),
                                   (12, 1040, 512), (15, 64, 896), (16, 336, 384), (17, 144, 256),
                                   (31, 32, 256), (33, 128, 384), (129, 272, 512), (300, 384, 256),
                                   (64, 20480, 256), (200, 5120, 512)])
def test_sizes(h32, bits, M, N, K):
    import torch
    z, ops = _operands(h32, M, N, K, bits, M + N)
    _check(h32, z, ops, bits)
    r = np.random.default_rng(M + K)
    bias = (0.3 * r.standard_normal(N)).astype(np.float32)
    _check(h32, z, ops, bits, bias=bias, res=torch_of(r.standard_normal((M, N)).astype(np.float32)))
    _check(h32, z, ops, bits, act="swiglu", y_bf16=True,
           res=torch_of(r.standard_normal((M, N // 2)).astype(np.float32)).bfloat16())


@pytest.mark.parametrize("bits,M,N,K,act,res", [
    (4, 130, 20480, 1024, "none", False), (4, 130, 20480, 896, "none", False),
    (8, 130, 20480, 1024, "relu", False), (4, 90, 40960, 1024, "relu", False),
    (4, 70, 40960, 2688, "none", True), (4, 257, 10256, 1920, "swiglu", False),
    (8, 200, 20480, 3456, "swiglu", True), (4, 130, 20496, 2944, "silu", False),
    (4, 130, 20480, 6144, "gelu_erf", False), (4, 512, 34816, 1024, "none", False)])
def test_several_tiles_a_block(h32, bits, M, N, K, act, res):
    """More tiles than SMs, long and short of K: finished while the next one runs, the
    last one (whole, cut or split along K) and the short ones by the warps that summed
    them.  Held to the formula on the bare product's own bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(N + K)
    w = 0.05 * torch.randn((N, K), device="cuda", generator=g)
    ws = h32.h32_prepack_weights_q4_0_tc(*h32.h32_rotate_quantize_weights_q4_0(w))
    del w
    x = torch.randn((M, K), device="cuda", generator=g) / 4
    ops = ws + (h32.h32_quantize_act_q4_tc if bits == 4 else h32.h32_quantize_act_q8_tc)(x)
    z = np_of((h32.q4_0_x_q4_gemm_tc if bits == 4 else h32.q4_0_x_q8_gemm_tc)(*ops, M=M))
    n_out = N // 2 if act == "swiglu" else N
    r = torch.randn((M, n_out), device="cuda", generator=g).bfloat16() if res else None
    bias = np_of(torch.randn(N, device="cuda", generator=g))
    for b, yb in ((None, False), (bias, True)):
        _check(h32, z, ops, bits, M=M, bias=b, act=act, res=r, y_bf16=yb)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 6, 70])
def test_rows_do_not_depend_on_the_batch(h32, bits, M):
    """The same rows as a batch of 70 or fewer tokens, or one by one: equal bits."""
    import torch
    z, ops = _operands(h32, 70, 320, 1280, bits, 4)
    call = h32.q4_0_x_q4_gemm_tc_epilogue if bits == 4 else h32.q4_0_x_q8_gemm_tc_epilogue
    full = call(*ops, act="silu")
    part = call(*ops, M=M, act="silu")
    assert part.shape[0] == M and torch.equal(part, full[:M])


@pytest.mark.parametrize("M", [3, 50])
def test_pitched_and_in_place(h32, M):
    """residual and y as column ranges of a wider array, y in place of the residual;
    more operand rows than tokens; nothing outside changes."""
    import torch
    N, K = 160, 256
    z, ops = _operands(h32, M + 4, N, K, 4, 5)
    for dt in (torch.float32, torch.bfloat16):
        wide = torch.randn((M + 4, N + 64), device="cuda").to(dt)
        before = wide.clone()
        view = wide[:M, 32:32 + N]
        y = h32.q4_0_x_q4_gemm_tc_epilogue(*ops, M=M, residual=view, y=view)
        torch.cuda.synchronize()
        assert y is view
        _compare(np_of(view.float()), z[:M], None, "none", before[:M, 32:32 + N], dt == torch.bfloat16)
        assert torch.equal(wide[:, :32], before[:, :32]) and torch.equal(wide[M:], before[M:])
        assert torch.equal(wide[:, 32 + N:], before[:, 32 + N:])


@pytest.mark.parametrize("bits", [4, 8])
def test_extreme_codes(h32, bits):
    """Every code at its limit (the largest block sums of either sign)."""
    M, N, K = 5, 32, 256
    w = np.where(np.arange(K) % 2 == 0, -8.0, 7.0)[None, :] * np.ones((N, 1))
    w[::3] = -8.0
    w = w.astype(np.float32)
    w[:, ::32] = -8.0
    top = 7.0 if bits == 4 else 127.0
    x = np.ones((M, K), np.float32) * np.float32(top)
    x[1] *= -1
    x[2, 1::2] *= -1
    x[3, ::2] *= -1
    wq, wd = oracle.quantize_weights_q4_0(w, rotate=False)
    q = oracle.quantize_act_q4 if bits == 4 else oracle.quantize_act_q8
    xq, xd = q(x, rotate=False)
    z, _, _ = oracle.gemm(wq, wd, xq, xd, K)
    wp, wsc = h32.h32_prepack_weights_q4_0_tc(torch_of(wq), torch_of(wd.view(np.int16)))
    qt = h32.h32_quantize_act_q4_tc if bits == 4 else h32.h32_quantize_act_q8_tc
    xw, xdt = qt(torch_of(x), rotate=False)
    _check(h32, z, (wp, wsc, xw, xdt), bits)


def test_tiny_scales(h32):
    """Products of scales below the normal range (bit-exact all the same)."""
    M, N, K = 3, 32, 256
    w = (wl.weights_normal(N, K, 0.02, 3, wl.CFG_TEST, 3010) * np.float32(2.0 ** -8)).astype(np.float32)
    x = (wl.act_normal_outliers(M, K, 0.0, 1.0, 3, wl.CFG_TEST, 3011) * np.float32(2.0 ** -112)).astype(np.float32)
    wq, wd = oracle.quantize_weights_q4_0(w)
    xq, xd = oracle.quantize_act_q4(x)
    z, _, _ = oracle.gemm(wq, wd, xq, xd, K)
    wp, wsc = h32.h32_prepack_weights_q4_0_tc(torch_of(wq), torch_of(wd.view(np.int16)))
    xw, xdt = h32.h32_quantize_act_q4_tc(torch_of(x))
    assert np.any(z != 0)
    _check(h32, z, (wp, wsc, xw, xdt), 4)


@pytest.mark.parametrize("M", [1, 64])
def test_empty_stream_and_graph(h32, M):
    """M = 0; another stream; two calls captured into two graphs, replayed in turn on
    new inputs (the split shapes keep a workspace of each graph's own)."""
    import torch
    N, K = 20480, 256
    z, ops = _operands(h32, M, N, K, 4, 1)
    assert h32.q4_0_x_q4_gemm_tc_epilogue(*ops, M=0).shape == (0, N)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = h32.q4_0_x_q4_gemm_tc_epilogue(*ops, stream=s)
    s.synchronize()
    assert np.array_equal(np_of(y), z)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = h32.q4_0_x_q4_gemm_tc_epilogue(*ops, act="relu")
        graphs.append((g, y))
    for seed in (2, 3):
        z, new = _operands(h32, M, N, K, 4, seed)
        for o, n in zip(ops, new):
            o.copy_(n)
        for g, y in graphs + graphs[::-1]:
            g.replay()
            torch.cuda.synchronize()
            assert np.array_equal(np_of(y), np.maximum(z, 0))
    assert h32.h32_device_status() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 40])
def test_waits_that_give_up_are_reported(h32, bits, M):
    """A bound of one poll on every wait of the few-token product and of the tensor-core
    GEMM: the status reads timeout (a poll is itself a short wait in hardware, so the
    few-token product's may all be long enough), once, and the same context then
    computes exact results."""
    z, ops = _operands(h32, M, 1024, 2048, bits, 6)
    call = h32.q4_0_x_q4_gemm_tc_epilogue if bits == 4 else h32.q4_0_x_q8_gemm_tc_epilogue
    assert h32.h32_device_status() == 0
    h32.h32_set_wait_limit(1)
    try:
        call(*ops)
        assert h32.h32_device_status() in ((0, h32.H32_ERR_TIMEOUT) if M == 1 else (h32.H32_ERR_TIMEOUT,))
    finally:
        h32.h32_set_wait_limit(0)
    assert h32.h32_device_status() == 0
    _check(h32, z, ops, bits)


def test_waits_between_tiles_that_give_up_are_reported(h32):
    """The same where tiles are handed from warps to warps: a timeout, then exact results."""
    import torch
    w = 0.05 * torch.randn((20480, 1024), device="cuda")
    x = torch.randn((130, 1024), device="cuda")
    ops = h32.h32_prepack_weights_q4_0_tc(*h32.h32_rotate_quantize_weights_q4_0(w)) + \
        h32.h32_quantize_act_q4_tc(x)
    z = np_of(h32.q4_0_x_q4_gemm_tc(*ops))
    assert h32.h32_device_status() == 0
    h32.h32_set_wait_limit(1)
    try:
        h32.q4_0_x_q4_gemm_tc_epilogue(*ops)
        assert h32.h32_device_status() == h32.H32_ERR_TIMEOUT
    finally:
        h32.h32_set_wait_limit(0)
    assert h32.h32_device_status() == 0
    _check(h32, z, ops, 4)


@pytest.mark.parametrize("M", [2, 40])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu_erf", "swiglu"])
def test_stated_bounds_of_the_activations(h32, act, M):
    """Dense arguments where the results cancel, vanish and leave fp32's range: within the
    relative bounds stated with the entry points, and within 2^-121 (SwiGLU: times |up|)
    where the exponential's range ends."""
    import torch
    K = 128
    for lo, hi, N in ((-14.0, 8.0, 4096), (-110.0, -80.0, 2048), (-13.5, -8.0, 2048)):
        z, ops = _operands(h32, M, N, K, 4, 11)
        bias = np.linspace(lo, hi, N).astype(np.float32)
        if act == "swiglu":
            bias[1::2] = 1000 * np.cos(np.arange(N // 2)).astype(np.float32)
        y = h32.q4_0_x_q4_gemm_tc_epilogue(*ops, M=M, bias=torch_of(bias), act=act)
        torch.cuda.synchronize()
        zb = z + bias
        v, steps = _formula(zb, act)
        floor = 2.0 ** -121 * (np.maximum(1.0, np.abs(zb[:, 1::2].astype(np.float64))) if act == "swiglu" else 1.0)
        assert np.all(np.abs(np_of(y) - v) <= steps * H * np.abs(v) * (1 + 2.0 ** -10) + floor)


@pytest.mark.parametrize("bits,M,N,K,act,res", [
    (4, 512, 5120, 9088, "silu", False), (4, 512, 5120, 9216, "silu", False),
    (4, 512, 6144, 9216, "swiglu", True), (8, 512, 5120, 9216, "gelu_erf", False),
    (8, 512, 5120, 9088, "swiglu", True)])
def test_one_tile_a_block_and_a_piece(h32, bits, M, N, K, act, res):
    """One whole tile a block and pieces of the last wave, K on both sides of the length
    from which the tile is finished while the piece runs."""
    test_several_tiles_a_block(h32, bits, M, N, K, act, res)
