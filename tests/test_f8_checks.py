"""Refusals of the 8-bit floating-point quantizers and products and of h32_token_logprobs:
in the binding (wrong tensors) and in the library (bad sizes, types, alignment) before
anything touches a device."""
import ctypes

import pytest
import torch

import hadamard_rotated_bit_gb300 as h32
from hadamard_rotated_bit_gb300 import _build

f32, bf16, u8, i32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
BAD, MIS, OK = h32.H32_ERR_INVALID_ARG, h32.H32_ERR_ALIGNMENT, h32.H32_OK


def _raises(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        getattr(h32, fn)(*args, **kw)


def test_binding_refusals_quantizers():
    x = torch.zeros((4, 256))
    for fn in ("h32_quantize_act_f8", "h32_quantize_weights_f8"):
        _raises("must be a CUDA tensor", fn, x)
        _raises("dtype", fn, x.half())
        _raises("must be 2-D with contiguous", fn, torch.zeros((256, 4)).t())
        _raises("shape", fn, torch.zeros(256))
    a, w = "h32_quantize_act_f8", "h32_quantize_weights_f8"
    _raises("row_idx: dtype", a, x, row_idx=torch.zeros(3, dtype=torch.int64))
    _raises("row_idx: shape", a, x, row_idx=torch.zeros((3, 1), dtype=i32))
    _raises("xq: shape", a, x, xq=torch.zeros((4, 128), dtype=u8))
    _raises("xq: shape", a, x, row_idx=torch.zeros(9, dtype=i32), xq=torch.zeros((4, 256), dtype=u8))
    _raises("xd: shape", a, x, xd=torch.zeros((1, 4)))
    _raises("xd: shape", a, x, xd=torch.zeros((2, 3)))
    _raises("wd: shape", w, torch.zeros((129, 256)), wd=torch.zeros((1, 2)))
    _raises("wq: dtype", w, x, wq=torch.zeros((4, 256), dtype=torch.int8))


def test_binding_refusals_products():
    wq, xq = torch.zeros((200, 256), dtype=u8), torch.zeros((3, 256), dtype=u8)
    wd, xd = torch.zeros((2, 2)), torch.zeros((2, 4))
    g, e = "h32_f8_gemm", "h32_f8_gemm_experts"
    _raises("must be a CUDA tensor", g, wq, wd, xq, xd)
    _raises("wd: shape", g, wq, wd[:1], xq, xd)
    _raises("xd: shape", g, wq, wd, xq, xd[:, :2].contiguous())
    _raises("xq: shape", g, wq, wd, xq[:, :128].contiguous(), xd)
    _raises("xq: shape", g, wq, wd, xq, xd, M=4)
    _raises("wq: dtype", g, wq.to(torch.int8), wd, xq, xd)
    _raises("y: shape", g, wq, wd, xq, xd, y=torch.zeros((3, 199)))
    _raises("y_dtype must", g, wq, wd, xq, xd, y_dtype=torch.float16)
    _raises("y is", g, wq, wd, xq, xd, y=torch.zeros((3, 200)), y_dtype=bf16)
    off = torch.zeros(3, dtype=i32)
    _raises("must be a CUDA tensor", e, wq, wd, xq, xd, off, 100)
    _raises("E \\* N rows", e, wq, wd, xq, xd, off, 150)
    _raises("E \\* N rows", e, wq, wd, xq, xd, off, 0)
    _raises("expert_off: shape", e, wq, wd, xq, xd, off[:2], 100)
    _raises("expert_off: dtype", e, wq, wd, xq, xd, off.long(), 100)
    _raises("wd: shape", e, wq, torch.zeros((4, 2)), xq, xd, off, 100)


def test_binding_refusals_logprobs():
    l, t, f = torch.zeros((4, 50)), torch.zeros(4, dtype=i32), "h32_token_logprobs"
    _raises("must be a CUDA tensor", f, l, t)
    _raises("logits: dtype", f, l.half())
    _raises("logits must be 2-D with contiguous", f, torch.zeros((50, 4)).t())
    _raises("logits: shape", f, torch.zeros((4, 0)))
    _raises("top must be between 0 and 32", f, l, t, top=33)
    _raises("top must be between 0 and 3", f, l[:, :3].contiguous(), t, top=4)
    _raises("top must be between", f, l, t, top=-1)
    _raises("targets: dtype", f, l, t.long())
    _raises("targets: shape", f, l, t[:3])
    _raises("targets: shape", f, l, torch.zeros((3, 2), dtype=i32))
    _raises("logprob needs targets", f, l, logprob=torch.zeros(4))
    _raises("logprob: shape", f, l, t, logprob=torch.zeros((4, 1)))
    _raises("entropy: shape", f, l, t, entropy=torch.zeros(3))
    _raises("need top", f, l, t, top_id=torch.zeros((4, 2), dtype=i32))
    _raises("top_id: shape", f, l, t, top=3, top_id=torch.zeros((4, 2), dtype=i32))
    _raises("top_logprob: dtype", f, l, t, top=3, top_logprob=torch.zeros((4, 3), dtype=bf16))


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return h32.lib()


def _p(v):
    return ctypes.c_void_p(v)


def _end(call, **kw):
    """A call whose arguments are fine gets as far as the device."""
    if not torch.cuda.is_available():
        assert call(**kw) == h32.H32_ERR_UNSUPPORTED, kw


def test_library_refusals_quantizers(lib):
    P = 4096

    def act(x=P, dt=0, T=4, K=256, ldx=256, idx=None, R=4, xq=2 * P, xd=3 * P, ldxd=4, rot=0):
        return lib.h32_quantize_act_f8(_p(x), dt, T, K, ldx, _p(idx), R, _p(xq), _p(xd), ldxd, rot, _p(0))

    for kw in (dict(T=-1, R=-1), dict(K=0), dict(K=48), dict(ldx=128), dict(dt=2), dict(rot=16),
               dict(rot=128, K=192), dict(R=3), dict(R=-1, idx=P), dict(ldxd=3), dict(ldxd=6, T=6, R=6) | {"ldxd": 7},
               dict(x=None), dict(xq=None), dict(xd=None), dict(T=0, R=4, idx=P),
               dict(T=1 << 31, R=1, idx=P), dict(R=1 << 29, T=1 << 29, ldxd=1 << 29)):
        assert act(**kw) == BAD, kw
    for kw in (dict(x=P + 8), dict(xq=P + 4), dict(xd=P + 4), dict(ldx=258), dict(ldx=260, dt=1), dict(idx=P + 2)):
        assert act(**kw) == MIS, kw
    assert act(T=0, R=0) == OK and act(R=0, idx=P) == OK
    _end(act)
    _end(act, R=9, idx=P + 4, ldxd=12, rot=128, dt=1)

    def weights(w=P, dt=0, N=4, K=256, ldw=256, rot=0, wq=2 * P, wd=3 * P):
        return lib.h32_quantize_weights_f8(_p(w), dt, N, K, ldw, rot, _p(wq), _p(wd), _p(0))

    for kw in (dict(N=-1), dict(K=0), dict(K=40), dict(ldw=255), dict(dt=-1), dict(rot=3), dict(rot=64, K=96),
               dict(w=None), dict(wq=None), dict(wd=None), dict(N=1 << 31)):
        assert weights(**kw) == BAD, kw
    for kw in (dict(w=P + 4), dict(wq=P + 8), dict(wd=P + 4), dict(ldw=257)):
        assert weights(**kw) == MIS, kw
    assert weights(N=0) == OK
    _end(weights, rot=1)


def test_library_refusals_long_rows(lib):
    """Rows of 2^31 values or more, which no product takes and whose places are numbered in 32
    bits, and row counts whose product with the blocks of a row wraps around 64 bits."""
    P = 4096
    for K in (1 << 31, 1 << 32, (1 << 32) + 32, (1 << 33) + 128, 1 << 40):
        for dt in (0, 1):
            assert lib.h32_quantize_act_f8(_p(P), dt, 1, K, K, _p(None), 1, _p(2 * P), _p(3 * P), 4, 0, _p(0)) == BAD
            assert lib.h32_quantize_weights_f8(_p(P), dt, 1, K, K, 0, _p(2 * P), _p(3 * P), _p(0)) == BAD
    for R, K in ((1 << 38, 1 << 31), (1 << 40, 1 << 29), (1 << 60, 512), (1 << 32, 32)):
        assert lib.h32_quantize_act_f8(_p(P), 0, 4, K, K, _p(5 * P), R, _p(2 * P), _p(3 * P), R, 0, _p(0)) == BAD
    for N in ((1 << 31) - 128, 1 << 31, (1 << 63) - 1):
        assert lib.h32_quantize_weights_f8(_p(P), 0, N, 256, 256, 0, _p(2 * P), _p(3 * P), _p(0)) == BAD
    # the longest rows allowed get as far as the device (a call without a GPU)
    if not torch.cuda.is_available():
        K = (1 << 31) - 288
        assert lib.h32_quantize_weights_f8(_p(P), 1, 1, K, K, 0, _p(2 * P), _p(3 * P), _p(0)) == h32.H32_ERR_UNSUPPORTED


def test_library_refusals_products(lib):
    P = 4096

    def dense(wq=P, wd=2 * P, xq=3 * P, xd=4 * P, ldxd=4, M=4, N=100, K=256, y=5 * P, dt=0, ldy=100,
              ws=None, ws_bytes=0):
        return lib.h32_f8_gemm(_p(wq), _p(wd), _p(xq), _p(xd), ldxd, M, N, K, _p(y), dt, ldy, _p(ws), ws_bytes, _p(0))

    def experts(wq=P, wd=2 * P, E=3, xq=3 * P, xd=4 * P, ldxd=4, off=6 * P, M=4, N=100, K=256, y=5 * P, dt=0, ldy=100):
        return lib.h32_f8_gemm_experts(_p(wq), _p(wd), E, _p(xq), _p(xd), ldxd, _p(off), M, N, K, _p(y), dt, ldy, _p(0))

    for call in (dense, experts):
        for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(K=80), dict(ldxd=3), dict(ldxd=6), dict(ldy=99), dict(dt=2),
                   dict(wq=None), dict(wd=None), dict(xq=None), dict(xd=None), dict(y=None),
                   dict(M=(1 << 31) - 4, ldxd=1 << 31), dict(N=1 << 31, ldy=1 << 31)):
            assert call(**kw) == BAD, kw
        for kw in (dict(wq=P + 8), dict(wd=P + 4), dict(xq=P + 1), dict(xd=P + 4), dict(y=P + 2)):
            assert call(**kw) == MIS, kw
        assert call(M=0) == OK
        _end(call)
        _end(call, N=1, ldy=1, K=32, dt=1)
    assert dense(ws=P + 8, ws_bytes=1 << 30) == MIS
    n = ctypes.c_size_t(7)
    for kw in ((-1, 4, 128), (1, 0, 128), (1, 4, 0), (1, 4, 100)):
        assert lib.h32_f8_gemm_workspace_bytes(*kw, ctypes.byref(n)) == BAD
    assert lib.h32_f8_gemm_workspace_bytes(1, 4, 128, None) == BAD
    # sizes that the product refuses, some of which would wrap around 64 bits in its plan
    for kw in ((1 << 31, 4, 128), (1, 1 << 31, 128), (1, 4, 1 << 31), (1 << 62, 1 << 40, 1 << 40),
               ((1 << 63) - 1, 4, 128), (1, (1 << 63) - 1, 128), (1, 4, (1 << 63) - 32), (1 << 30, 1 << 30, 128)):
        assert lib.h32_f8_gemm_workspace_bytes(*kw, ctypes.byref(n)) == BAD, kw
        M, N, K = kw
        assert dense(M=M, N=N, K=K, ldy=N, ldxd=(M + 3) // 4 * 4 if M < 1 << 62 else M // 4 * 4) == BAD, kw
    if not torch.cuda.is_available():
        assert lib.h32_f8_gemm_workspace_bytes(1, 4, 128, ctypes.byref(n)) == h32.H32_ERR_UNSUPPORTED
    assert experts(E=0) == BAD and experts(E=1025) == BAD and experts(off=None) == BAD
    assert experts(off=P + 2) == MIS


def test_library_refusals_logprobs(lib):
    P = 4096

    def call(l=P, dt=0, T=4, V=50, ldl=50, t=2 * P, n=1, top=3, lp=3 * P, ent=4 * P, ids=5 * P, tlp=6 * P):
        return lib.h32_token_logprobs(_p(l), dt, T, V, ldl, _p(t), n, top, _p(lp), _p(ent), _p(ids), _p(tlp), _p(0))

    for kw in (dict(T=-1), dict(V=0), dict(V=1 << 31, ldl=1 << 31), dict(ldl=49), dict(dt=2), dict(n=-1), dict(top=-1),
               dict(top=33), dict(V=2, top=3), dict(T=1 << 28), dict(l=None), dict(t=None), dict(lp=None),
               dict(ids=None), dict(tlp=None)):
        assert call(**kw) == BAD, kw
    for kw in (dict(l=P + 2), dict(l=P + 1, dt=1), dict(t=P + 2), dict(lp=P + 1), dict(ent=P + 2), dict(ids=P + 3),
               dict(tlp=P + 2)):
        assert call(**kw) == MIS, kw
    assert call(T=0) == OK
    _end(call)
    _end(call, l=P + 2, dt=1, n=0, t=None, lp=None, top=0, ids=None, tlp=None, ent=None)
