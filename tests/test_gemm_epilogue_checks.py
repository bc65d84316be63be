"""Refusals of the products with an epilogue, in the binding and in the library."""
import ctypes

import pytest
import torch

import hadamard_rotated_bit_gb300 as h32
from hadamard_rotated_bit_gb300 import _build

u8, f32, bf16 = torch.uint8, torch.float32, torch.bfloat16


def test_binding_refusals():
    N, K, M = 32, 128, 8
    wp, wsc, xw, xdt = (torch.zeros((N, K), dtype=u8), torch.zeros((N, 4)),
                        torch.zeros((M, K), dtype=u8), torch.zeros((4, 8)))

    def raises(match, *a, fn=h32.q4_0_x_q4_gemm_tc_epilogue, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*(a or (wp, wsc, xw, xdt)), **kw)

    raises("must be a CUDA tensor")
    raises("act must be", act="tanh")
    raises("xw: shape", M=9)
    raises("xw: shape", fn=h32.q4_0_x_q8_gemm_tc_epilogue)
    raises("bias: shape", bias=torch.zeros(31))
    raises("bias: dtype", bias=torch.zeros(32, dtype=bf16))
    raises("residual: shape", residual=torch.zeros((8, 31)))
    raises("residual: shape", residual=torch.zeros((7, 32)))
    raises("residual: shape", residual=torch.zeros((8, 15)), act="swiglu")
    raises("residual: dtype", residual=torch.zeros((8, 32), dtype=torch.float16))
    raises("residual must be 2-D with contiguous", residual=torch.zeros((32, 32)).t()[:, ::1])
    raises("y: shape", y=torch.zeros((8, 16)))
    raises("y: dtype", y=torch.zeros((8, 32), dtype=torch.float64))
    raises("y is torch.float32, y_dtype torch.bfloat16", y=torch.zeros((8, 32)), y_dtype=bf16)
    raises("y_dtype must be", y_dtype=torch.float16)
    raises("workspace: dtype", workspace=torch.zeros(64))


@pytest.mark.parametrize("name", ["q4_0_x_q4_gemm_tc_epilogue", "q4_0_x_q8_gemm_tc_epilogue"])
def test_library_refusals(name):
    _build.build()
    p = 4096

    def call(wp=p, wsc=p, ldws=4, xw=p, xdt=p, ldxd=8, M=8, N=32, K=128, bias=p, act=0, res=2 * p,
             res_dt=0, ldr=32, y=p, y_dt=0, ldy=32, ws=None, nws=0):
        v = ctypes.c_void_p
        return getattr(h32.lib(), name)(v(wp), v(wsc), ldws, v(xw), v(xdt), ldxd, M, N, K, v(bias), act,
                                        v(res), res_dt, ldr, v(y), y_dt, ldy, v(ws), nws, v(0))

    assert call(M=0) == h32.H32_OK and call(M=0, y=None) == h32.H32_OK
    for kw in (dict(M=-1), dict(N=24), dict(K=96), dict(ldws=3), dict(ldws=5), dict(ldxd=4),
               dict(ldxd=9), dict(act=-1), dict(act=6), dict(ldy=31), dict(ldr=28), dict(y_dt=2),
               dict(res_dt=5), dict(y=None), dict(wp=None), dict(wsc=None), dict(xw=None),
               dict(xdt=None), dict(act=5, ldy=15), dict(y=2 * p, y_dt=1), dict(y=2 * p, ldy=64)):
        assert call(**kw) == h32.H32_ERR_INVALID_ARG, kw
    for kw in (dict(wp=4100), dict(wsc=4104), dict(xw=4100), dict(xdt=4108), dict(bias=4098),
               dict(res=8200), dict(y=4104), dict(ldy=33), dict(ldr=34), dict(y_dt=1, ldy=36)):
        assert call(**kw) == h32.H32_ERR_ALIGNMENT, kw
    if not torch.cuda.is_available():
        for kw in ({}, dict(y=2 * p), dict(bias=None, res=None), dict(act=5, ldy=16, ldr=16)):
            assert call(**kw) == h32.H32_ERR_UNSUPPORTED, kw
