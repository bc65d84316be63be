"""GPU parity of the 8-bit floating-point quantizers and products: codes and scales bit
for bit against the oracle; products exactly where the arithmetic is exact (small integer
codes, power-of-two scales), else within a bound derived from the roundings."""
import numpy as np
import pytest

import oracle
from hadamard_rotated_bit_gb300 import workloads as wl
from tests._gpu import np_of, torch_bf16, torch_of

pytestmark = pytest.mark.gpu

U = 2.0 ** -24   # half a step of fp32, relative


@pytest.fixture(scope="module")
def h32():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hadamard_rotated_bit_gb300 as m
    from hadamard_rotated_bit_gb300 import _build
    _build.build()
    return m


def _ok(h32):
    import torch
    torch.cuda.synchronize()
    assert h32.h32_device_status() == 0


def _rows(M, K, seed, bf16, scale=1.0):
    x = wl.act_normal_outliers(M, K, 0.01, 30.0, seed, wl.CFG_TEST, 5000) * np.float32(scale)
    return wl.f32_to_bf16_bits(x) if bf16 else x


def _dev(a):
    return torch_bf16(a) if a.dtype == np.uint16 else torch_of(a)


def _check_act(xq, xd, x, rotate):
    q, d = oracle.quantize_act_f8(x, rotate)
    R = q.shape[0]
    assert np.array_equal(np_of(xq)[:R], q), "codes"
    assert np.array_equal(np_of(xd)[:, :R].T, d), "scales"


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,K,rotate", [(1, 32, 0), (1, 5120, 128), (3, 96, 32), (5, 160, 0), (4, 192, 64),
                                        (7, 1152, 128), (33, 256, 64), (130, 4128, 32)])
def test_quantize_act(h32, M, K, rotate, bf16):
    x = _rows(M, K, M + K, bf16)
    x[M // 2, :min(K, 128)] = 0      # an all-zero group
    xq, xd = h32.h32_quantize_act_f8(_dev(x), rotate=rotate)
    _ok(h32)
    assert xd.shape == ((K + 127) // 128, (M + 3) // 4 * 4)
    _check_act(xq, xd, x, rotate)


@pytest.mark.parametrize("scale", [1e-38, 2.0 ** -130, 1e-41, 1e30, 3e36])
def test_quantize_act_extreme_scales(h32, scale):
    """Groups whose 1/d overflows (an IEEE divide takes its place), and large ones."""
    x = _rows(6, 256, 3, False, scale)
    xq, xd = h32.h32_quantize_act_f8(_dev(x))
    wq, wd = h32.h32_quantize_weights_f8(_dev(x))
    _ok(h32)
    _check_act(xq, xd, x, 0)
    q, d = oracle.quantize_weights_f8(x)
    assert np.array_equal(np_of(wq), q) and np.array_equal(np_of(wd), d)


def test_quantize_act_non_finite(h32):
    x = _rows(4, 256, 5, False)
    x[0, 7], x[1, 130], x[2, :128] = np.nan, -np.inf, np.nan
    xq, xd = h32.h32_quantize_act_f8(_dev(x))
    _ok(h32)
    q, d = np_of(xq), np_of(xd)[:, :4].T
    rq, rd = oracle.quantize_act_f8(x)
    assert np.array_equal(d, rd) and d[1, 1] == np.inf
    nan = (rq & 127) == 127
    assert np.array_equal((q & 127) == 127, nan) and np.array_equal(q[~nan], rq[~nan])
    assert nan[0, 7] and nan[1, 130] and not nan[1, 129] and nan[2, :128].all() and nan.sum() == 130


@pytest.mark.parametrize("bf16", [False, True])
def test_quantize_act_pitched_gathered_into(h32, bf16):
    """Rows of a wider array, gathered, into buffers larger than needed: what lies behind
    the rows stays; an index outside the rows is reported and gives zeros."""
    import torch
    x = _rows(40, 352, 9, bf16)
    t = _dev(x)[:, 32:352]
    idx = np.random.default_rng(0).integers(0, 40, 101).astype(np.int32)
    big = np.concatenate([[0], idx]).astype(np.int32)
    xq = torch.full((110, 320), 77, dtype=torch.uint8, device="cuda")
    xd = torch.full((4, 112), -5.0, device="cuda")
    r = h32.h32_quantize_act_f8(t, rotate=64, row_idx=torch_of(big)[1:], xq=xq, xd=xd)
    _ok(h32)
    assert r[0] is xq and r[1] is xd
    _check_act(xq, xd[:3], x[idx, 32:], 64)
    assert (np_of(xq)[101:] == 77).all() and (np_of(xd)[:3, 101:] == -5).all() and (np_of(xd)[3] == -5).all()
    idx[[3, 50]] = 40, -1
    xq, xd = h32.h32_quantize_act_f8(t, row_idx=torch_of(idx))
    torch.cuda.synchronize()
    assert h32.h32_device_status() == h32.H32_ERR_DEVICE_GUARD
    good = np.setdiff1d(np.arange(101), [3, 50])
    q, d = oracle.quantize_act_f8(x[idx[good], 32:])
    assert np.array_equal(np_of(xq)[good], q) and not np_of(xq)[[3, 50]].any()
    assert np.array_equal(np_of(xd).T[good], d) and not np_of(xd).T[[3, 50]].any()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N,K,rotate", [(1, 32, 0), (127, 160, 32), (128, 128, 128), (129, 192, 64), (300, 1024, 128),
                                        (260, 4128, 0)])
def test_quantize_weights(h32, N, K, rotate, bf16):
    w = _rows(N, K, N + K, bf16, 0.02)
    wide = np.concatenate([w, w], 1)
    wq, wd = h32.h32_quantize_weights_f8(_dev(wide)[:, :K], rotate=rotate)
    _ok(h32)
    q, d = oracle.quantize_weights_f8(w, rotate)
    assert np.array_equal(np_of(wq), q) and np.array_equal(np_of(wd), d)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("rotate,K", [(0, 416), (32, 416), (64, 448), (128, 384)])
def test_quantize_weights_many_blocks(h32, K, rotate, bf16):
    """More blocks of 128 x 128 than run at once: the next one is copied under this one."""
    import torch
    N = 20001
    assert (N + 127) // 128 * ((K + 127) // 128) > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    w = _rows(N, K, N + K, bf16, 0.02)
    wq, wd = h32.h32_quantize_weights_f8(_dev(w), rotate=rotate)
    _ok(h32)
    q, d = oracle.quantize_weights_f8(w, rotate)
    assert np.array_equal(np_of(wq), q) and np.array_equal(np_of(wd), d)


# --------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------
def _exact_operands(M, N, K, seed, E=1):
    """Integer codes of at most 8 and scales of 1/2, 1 and 2: every sum is a multiple of
    1/4 below 64 * K * 4, exact in fp32 for K < 16384."""
    r = np.random.default_rng(seed)
    byte = oracle.e4m3_round(np.arange(-8, 9))
    wq, xq = byte[r.integers(0, 17, (E * N, K))], byte[r.integers(0, 17, (M, K))]
    nb, nt = (K + 127) // 128, (N + 127) // 128
    wd = (2.0 ** r.integers(-1, 2, (E * nt, nb))).astype(np.float32)
    xd = (2.0 ** r.integers(-1, 2, (M, nb))).astype(np.float32)
    return wq, wd, xq, xd


def _xd(xd, pad=0.0):
    import torch
    M, nb = xd.shape
    t = torch.full((nb, (M + 3) // 4 * 4), pad, device="cuda")
    t[:, :M] = torch_of(xd.T.copy())
    return t


SHAPES = [(1, 1, 32), (1, 5120, 5120), (2, 129, 96), (7, 384, 4224), (15, 100, 160), (16, 128, 128), (17, 500, 640),
          (31, 1000, 2048), (33, 77, 1056), (64, 640, 512), (65, 2000, 384), (128, 257, 1024), (129, 128, 4096),
          (200, 1537, 96), (255, 4096, 320), (256, 256, 256), (257, 700, 5120), (333, 5120, 1024), (511, 96, 736),
          (1030, 1300, 288), (2048, 8192, 128), (33, 831, 4032), (150, 783, 8896), (380, 269, 6464)]


# more tiles than run at once, of several K steps each, on every kernel instance
# (tests/test_f8_plan.py holds this list and EXPERTS_MANY_TILES to that)
MANY_TILES = [(1, 40001, 2080), (20, 20103, 672), (50, 39001, 160), (100, 39001, 800), (300, 10001, 288),
              (140, 39001, 288), (300, 39001, 416)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,N,K", MANY_TILES)
def test_product_exact_many_tiles(h32, M, N, K, bf16):
    test_product_exact(h32, M, N, K, bf16)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_exact(h32, M, N, K, bf16):
    import torch
    wq, wd, xq, xd = _exact_operands(M, N, K, M * 7 + N * 3 + K)
    y = h32.h32_f8_gemm(torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd, np.nan),
                        y_dtype=torch.bfloat16 if bf16 else None)
    _ok(h32)
    ref = torch.from_numpy(oracle.f8_gemm(wq, wd, xq, xd)[0]).float()
    assert torch.equal(y.cpu(), ref.bfloat16() if bf16 else ref)


@pytest.mark.parametrize("M,N,K", [(300, 5120, 16000), (1000, 5001, 16000), (140, 5632, 16352)])
def test_product_shared_out_along_k(h32, M, N, K):
    """Sizes whose tiles are cut along K between the pairs of CTAs: with the binding's
    workspace, one of the caller's (dirty), and none; on two streams at once and from two
    graphs replayed together."""
    import torch
    need = h32.h32_f8_gemm_workspace_bytes(M, N, K)
    assert need > 0
    wq, wd, xq, xd = _exact_operands(M, N, K, M + N)
    t = torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd, np.nan)
    ref = torch.from_numpy(oracle.f8_gemm(wq, wd, xq, xd)[0]).float().cuda()
    assert torch.equal(h32.h32_f8_gemm(*t), ref)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    y = torch.empty((M, N), device="cuda")
    for p, n, want in ((ws.data_ptr(), need, 0), (ws.data_ptr(), need, 0), (None, 0, 0),
                       (ws.data_ptr(), need - 16, h32.H32_ERR_INVALID_ARG)):
        y.zero_()
        st = h32.lib().h32_f8_gemm(t[0].data_ptr(), t[1].data_ptr(), t[2].data_ptr(), t[3].data_ptr(), t[3].shape[1],
                                   M, N, K, y.data_ptr(), 0, N, p, n, torch.cuda.current_stream().cuda_stream)
        assert st == want
        _ok(h32)
        assert torch.equal(y, ref) == (want == 0)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ys = [h32.h32_f8_gemm(*t, stream=s) for _ in range(3) for s in (s1, s2)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, ref) for y in ys)
    graphs = []
    for s in (s1, s2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = h32.h32_f8_gemm(*t)
        graphs.append((g, y, s))
    for _ in range(3):
        for g, _, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    _ok(h32)
    assert all(torch.equal(y, ref) for _, y, _ in graphs)


def _same_every_time(h32, M, N, K, calls):
    """Equal calls give equal bits, call after call, while other calls come between them."""
    import torch
    fin = np.setdiff1d(np.arange(256), [127, 255]).astype(np.uint8)
    r = np.random.default_rng(M + N)
    wq, xq = fin[r.integers(0, 254, (N, K))], fin[r.integers(0, 254, (M, K))]
    nb = (K + 127) // 128
    wd = (10.0 ** r.uniform(-4, 0, ((N + 127) // 128, nb))).astype(np.float32)
    xd = (10.0 ** r.uniform(-4, 0, (M, nb))).astype(np.float32)
    a = torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd)
    b = a[0].flip(1).contiguous(), a[1].flip(1).contiguous(), a[2].flip(0).contiguous(), a[3]
    first = [h32.h32_f8_gemm(*a), h32.h32_f8_gemm(*b)]
    rows = r.integers(0, M, 6)
    ref, mag = oracle.f8_gemm(wq, wd, xq[rows], xd[rows])
    assert (np.abs(np_of(first[0])[rows].astype(np.float64) - ref) <= (256 + nb + 2) * U * mag).all()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(calls):
        differ += (h32.h32_f8_gemm(*(a, b)[i % 2]) != first[i % 2]).sum()
    _ok(h32)
    assert int(differ) == 0


@pytest.mark.parametrize("M,N,K", [(300, 9001, 4096), (700, 30001, 1056), (2000, 5001, 2080)])
def test_pairs_give_the_same_bits_every_time(h32, M, N, K):
    """Tiles of two CTAs, several a pair, of many K steps."""
    assert h32.h32_f8_gemm_workspace_bytes(M, N, K) == 0
    _same_every_time(h32, M, N, K, 100)


@pytest.mark.parametrize("M,N,K", [(300, 5120, 16000), (1000, 5001, 16000)])
def test_partial_sums_are_the_same_every_time(h32, M, N, K):
    assert h32.h32_f8_gemm_workspace_bytes(M, N, K) > 0
    _same_every_time(h32, M, N, K, 60)


@pytest.mark.parametrize("M,N,K", [(1, 640, 5120), (5, 300, 17408), (40, 256, 2080), (100, 130, 4096), (300, 520, 5120)])
def test_product_random_codes(h32, M, N, K):
    """Every finite code, scales over several octaves.  Per block the tensor core adds 128
    products: 128 additions off by at most 2 U each of the magnitudes' sum; then the
    scales' product, the fold and nb additions, U each."""
    r = np.random.default_rng(M + N)
    fin = np.setdiff1d(np.arange(256), [127, 255]).astype(np.uint8)
    wq, xq = fin[r.integers(0, 254, (N, K))], fin[r.integers(0, 254, (M, K))]
    nb = (K + 127) // 128
    wd = (10.0 ** r.uniform(-4, 0, ((N + 127) // 128, nb))).astype(np.float32)
    xd = (10.0 ** r.uniform(-4, 0, (M, nb))).astype(np.float32)
    y = h32.h32_f8_gemm(torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd))
    _ok(h32)
    ref, mag = oracle.f8_gemm(wq, wd, xq, xd)
    err = np.abs(np_of(y).astype(np.float64) - ref)
    print("largest error in U of the magnitudes:", (err / mag).max() / U)
    assert (err <= (256 + nb + 2) * U * mag).all()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("M", [3, 20, 40, 140, 300])
def test_product_scales_outside_the_normal_range(h32, M, bf16):
    """The product of two scales is rounded as it stands: to a multiple of 2^-149 below fp32's
    normal range (sums of codes are then exact), to infinity above."""
    import torch
    N, K = 300, 416
    wq, _, xq, _ = _exact_operands(M, N, K, M)
    nb, nt = (K + 127) // 128, (N + 127) // 128
    r = np.random.default_rng(M)
    wd = (r.integers(64, 128, (nt, nb)) * 2.0 ** -80).astype(np.float32)
    xd = (r.integers(64, 128, (M, nb)) * 2.0 ** -81).astype(np.float32)
    val = oracle.e4m3_values()
    sums = np.stack([val[xq[:, 128 * b:128 * b + 128]] @ val[wq[:, 128 * b:128 * b + 128]].T for b in range(nb)])

    def fold(xd, wd):
        acc = np.zeros((M, N), np.float32)
        with np.errstate(all="ignore"):
            for b in range(nb):
                acc = acc + (xd[:, b, None] * np.repeat(wd[:, b], 128)[None, :N]) * sums[b].astype(np.float32)
        return torch.from_numpy(acc)

    def run(xd, wd):
        y = h32.h32_f8_gemm(torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd), y_dtype=torch.bfloat16 if bf16 else None)
        _ok(h32)
        return y.cpu()

    # 64^2 to 127^2 times 2^-161, so 1 to 4 times 2^-149: sums of at most 4 * 8192 * 4 steps
    ref = fold(xd, wd)
    assert bool((ref != 0).any()) and float(ref.abs().max()) < 2.0 ** -126
    assert torch.equal(run(xd, wd), ref.bfloat16() if bf16 else ref)
    xd[M // 2], wd[1] = 2.0 ** 70, 2.0 ** 70
    ref = fold(xd, wd)
    assert bool(torch.isinf(ref[M // 2, 128:256]).any())
    assert torch.equal(torch.nan_to_num(run(xd, wd).float(), nan=1234.0),
                       torch.nan_to_num((ref.bfloat16() if bf16 else ref).float(), nan=1234.0))


def test_product_nan_stays_in_its_row_and_column(h32):
    wq, wd, xq, xd = _exact_operands(40, 300, 256, 1)
    wq[7, 3], xq[5, 200] = 0x7F, 0xFF
    for M in (6, 40):
        y = h32.h32_f8_gemm(torch_of(wq), torch_of(wd), torch_of(xq[:M]), _xd(xd[:M]))
        _ok(h32)
        want = np.zeros((M, 300), bool)
        want[:, 7] = want[5] = True
        assert np.array_equal(np.isnan(np_of(y)), want)


def test_product_into_pitched_rows_and_larger_buffers(h32):
    """Outputs into the middle of wider, longer arrays of odd pitch; M below the operands' rows."""
    import torch
    for M, N, dt in ((3, 133, torch.float32), (3, 133, torch.bfloat16), (150, 301, torch.bfloat16), (290, 700, torch.float32)):
        wq, wd, xq, xd = _exact_operands(M + 5, N, 384, M)
        full = torch.full((M + 2, N + 3), 9.0, dtype=dt, device="cuda")
        y = h32.h32_f8_gemm(torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd), M=M, y=full)
        _ok(h32)
        assert y is full
        ref = torch.from_numpy(oracle.f8_gemm(wq, wd, xq[:M], xd[:M])[0]).float().to(dt)
        assert torch.equal(full[:M, :N].cpu(), ref)
        assert bool((full[M:] == 9).all()) and bool((full[:, N:] == 9).all())


def test_empty_calls(h32):
    import torch
    wq, wd, xq, xd = _exact_operands(1, 40, 128, 0)
    y = h32.h32_f8_gemm(torch_of(wq), torch_of(wd), torch_of(xq)[:0], torch.zeros((1, 0), device="cuda"))
    assert y.shape == (0, 40)
    q, d = h32.h32_quantize_act_f8(torch.zeros((0, 128), device="cuda"))
    assert q.shape == (0, 128) and d.shape == (1, 0)
    q, d = h32.h32_quantize_weights_f8(torch.zeros((0, 128), device="cuda"))
    assert q.shape == (0, 128) and d.shape == (0, 1)
    _ok(h32)


# --------------------------------------------------------------------------
# expert products
# --------------------------------------------------------------------------
def _experts_ref(wq, wd, xq, xd, off, N):
    E, nt = len(off) - 1, (N + 127) // 128
    return np.concatenate([oracle.f8_gemm(wq[e * N:(e + 1) * N], wd[e * nt:(e + 1) * nt], xq[off[e]:off[e + 1]],
                                          xd[off[e]:off[e + 1]])[0] for e in range(E)])


def _uneven(E, per):
    """Counts of E groups, `per` on average, a few of them 0 or 1."""
    c = [per] * E
    for i in range(0, E - 3, 4):
        d = min(per, 3 * i // 4 + 1)
        c[i], c[i + 1] = per - d, per + d
    return c


# two rows or so each (tokens as columns), 20 to 120 (on the lanes, tiles of every width)
EXPERTS_MANY_TILES = [(_uneven(160, 2), 200, 416), (_uneven(64, 20), 1000, 288), (_uneven(64, 60), 260, 288),
                      (_uneven(64, 90), 260, 288), (_uneven(20, 120), 260, 288), (_uneven(64, 120), 260, 160),
                      (_uneven(20, 120), 1000, 416), (_uneven(20, 120), 2000, 416)]


@pytest.mark.parametrize("counts,N,K", EXPERTS_MANY_TILES)
@pytest.mark.parametrize("bf16", [False, True])
def test_experts_exact_many_tiles(h32, counts, N, K, bf16):
    test_experts_exact(h32, counts, N, K, bf16)


@pytest.mark.parametrize("counts,N,K", [([1], 128, 128), ([0, 5, 0, 1, 16], 130, 288), ([3, 17, 29, 0, 2, 15], 300, 512),
                                        ([40, 61, 0, 64, 65, 3], 384, 256), ([100, 7, 131, 128, 129], 96, 640),
                                        ([300, 0, 1, 513, 255], 520, 384), ([0, 0, 900], 257, 160), ([2] * 160, 64, 96)])
@pytest.mark.parametrize("bf16", [False, True])
def test_experts_exact(h32, counts, N, K, bf16):
    import torch
    E, R = len(counts), sum(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    wq, wd, xq, xd = _exact_operands(R, N, K, R + N, E)
    y = torch.full((R + 1, N), 9.0, dtype=torch.bfloat16 if bf16 else torch.float32, device="cuda")
    h32.h32_f8_gemm_experts(torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd, np.nan), torch_of(off), N, y=y)
    _ok(h32)
    ref = torch.from_numpy(_experts_ref(wq, wd, xq, xd, off, N)).float()
    assert torch.equal(y[:R].cpu(), ref.to(y.dtype)) and bool((y[R] == 9).all())


def test_experts_bad_offsets_are_reported(h32):
    import torch
    for R, bad in ((24, [0, 10, 9, 24]), (24, [1, 2, 3, 24]), (24, [0, 4, 8, 23]), (600, [0, 4, 2000000000, 600]),
                   (24, [0, -5, 3, 24])):
        wq, wd, xq, xd = _exact_operands(R, 140, 128, 1, 3)
        y = torch.full((R, 140), 9.0, device="cuda")
        h32.h32_f8_gemm_experts(torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd),
                                torch_of(np.array(bad, np.int32)), 140, y=y)
        torch.cuda.synchronize()
        assert h32.h32_device_status() == h32.H32_ERR_DEVICE_GUARD and h32.h32_device_status() == 0
        assert bool((y == 9).all())


# --------------------------------------------------------------------------
# streams, graphs
# --------------------------------------------------------------------------
@pytest.mark.parametrize("M,N,K", [(2, 640, 5120), (40, 300, 512), (300, 1000, 640)])
def test_streams_and_graphs(h32, M, N, K):
    """On a stream of its own, two at once, and captured; every run gives the same bits."""
    import torch
    x = _rows(M, K, 11, True)
    w = _rows(N, K, 12, False, 0.02)
    tx, (wq, wd) = torch_bf16(x), h32.h32_quantize_weights_f8(torch_of(w), rotate=32)

    def path(stream=None):
        q, d = h32.h32_quantize_act_f8(tx, rotate=32, stream=stream)
        return h32.h32_f8_gemm(wq, wd, q, d, stream=stream)

    torch.cuda.synchronize()
    first = path()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = [], []
    for _ in range(4):
        a.append(path(s1))
        b.append(path(s2))
    torch.cuda.synchronize()
    for y in a + b:
        assert torch.equal(y, first)
    graphs = []
    for s in (s1, s2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            y = path()
        graphs.append((g, y, s))
    x2 = _rows(M, K, 13, True)
    tx.copy_(torch_bf16(x2))
    torch.cuda.synchronize()
    for g, _, s in graphs:
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    want = path()
    _ok(h32)
    for _, y, _ in graphs:
        assert torch.equal(y, want)
    assert not torch.equal(want, first)


@pytest.mark.parametrize("M,N,K", [(2, 4096, 4096), (24, 4096, 4096), (60, 4096, 4096), (100, 8192, 4096),
                                   (700, 4096, 4096), (300, 5120, 16000)])
def test_one_poll_wait_bound(h32, M, N, K):
    """A bound of one poll: waits give up, the status says so once, and the same context
    then computes exactly."""
    wq, wd, xq, xd = _exact_operands(M, N, K, M)
    t = torch_of(wq), torch_of(wd), torch_of(xq), _xd(xd)
    ref = oracle.f8_gemm(wq[:256], wd[:2], xq, xd)[0].astype(np.float32)
    assert h32.h32_device_status() == 0
    h32.h32_set_wait_limit(1)
    try:
        for _ in range(3):
            h32.h32_f8_gemm(*t)
        st = h32.h32_device_status()
    finally:
        h32.h32_set_wait_limit(0)
    assert st == h32.H32_ERR_TIMEOUT and h32.h32_device_status() == 0
    y = h32.h32_f8_gemm(*t)
    _ok(h32)
    assert np.array_equal(np_of(y)[:, :256], ref)
