"""Refusals of h32_add_rms_norm_quantize, in the binding (wrong tensors) and in the
library (bad sizes, types, alignment, overlaps) before anything touches a device."""
import ctypes

import pytest
import torch

import hadamard_rotated_bit_gb300 as h32
from hadamard_rotated_bit_gb300 import _build

f32, bf16, u8 = torch.float32, torch.bfloat16, torch.uint8


def _raises(match, *args, **kw):
    with pytest.raises(ValueError, match=match):
        h32.h32_add_rms_norm_quantize(*args, **kw)


def test_binding_refusals():
    x, w, r = torch.zeros((4, 64)), torch.ones(64), torch.zeros((4, 64), dtype=bf16)
    _raises("must be a CUDA tensor", x, w, residual=r)
    _raises("x: dtype", x.half(), w)
    _raises("x must be 2-D with contiguous", torch.zeros((64, 4)).t(), w)
    _raises("weight: shape", x, w[:32])
    _raises("residual: shape", x, w, residual=r[:3])
    _raises("residual: dtype", x, w, residual=r.half())
    _raises("residual_out: dtype", x, w, residual=r, residual_out=torch.zeros((4, 64)))
    _raises("residual_out: shape", x, w, residual=r, residual_out=r[:3])
    _raises("residual_out needs a residual", x, w, residual_out=r)
    _raises("norm_out must be bf16 or fp32", x, w, norm_out=torch.float16)
    _raises("norm_out: shape", x, w, norm_out=torch.zeros((3, 64)))
    _raises("form must be", x, w, form="q5")
    _raises("form=None needs norm_out", x, w, form=None)
    _raises("form=None writes no", x, w, form=None, norm_out=f32, xq=torch.zeros((4, 64), dtype=u8))
    _raises("xq: shape", x, w, xq=torch.zeros((4, 32), dtype=u8))
    _raises("xq: shape", x, w, form="q8_tc", xq=torch.zeros((4, 64), dtype=u8))
    _raises("xd: shape", x, w, xd=torch.zeros((2, 3)))
    _raises("xd: shape", x, w, form="q8", xd=torch.zeros((4, 3)))


@pytest.fixture(scope="module")
def call():
    _build.build()
    p = 4096

    def f(x=p, x_dt=0, ldx=64, res=2 * p, res_dt=1, ldr=64, w=3 * p, w_dt=0, eps=1e-6, M=4, K=64,
          ro=4 * p, ldro=64, no=None, n_dt=0, ldn=64, form=2, rot=1, xq=5 * p, xd=6 * p, ldxd=4):
        v = ctypes.c_void_p
        return h32.lib().h32_add_rms_norm_quantize(
            v(x), x_dt, ldx, v(res), res_dt, ldr, v(w), w_dt, eps, M, K, v(ro), ldro, v(no), n_dt,
            ldn, form, rot, v(xq), v(xd), ldxd, v(0))
    return f


def test_library_refusals(call):
    bad, mis = h32.H32_ERR_INVALID_ARG, h32.H32_ERR_ALIGNMENT
    assert call(M=0) == h32.H32_OK
    for kw in (dict(M=-1), dict(K=48), dict(K=0), dict(K=32800, ldx=32800, ldr=32800, ldro=32800),
               dict(ldx=32), dict(ldr=32), dict(ldro=32), dict(x_dt=2), dict(res_dt=2), dict(w_dt=7),
               dict(eps=0.0), dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")),
               dict(rot=16), dict(rot=128), dict(form=5), dict(form=-1), dict(xq=None), dict(xd=None),
               dict(xq=None, xd=None), dict(ldxd=3), dict(ldxd=6), dict(x=None), dict(w=None),
               dict(res=None), dict(no=4096 * 7, ldn=32), dict(no=4096 * 7, n_dt=3),
               # an output over an input in another type or pitch, two outputs over each other
               dict(ro=4096), dict(ro=8192, ldro=128), dict(no=16384, n_dt=1), dict(no=4096, n_dt=1),
               dict(no=4096, ldn=128), dict(no=8192)):
        assert call(**kw) == bad, kw
    for kw in (dict(x=4100), dict(w=4104), dict(res=8200), dict(ro=16392), dict(no=28680),
               dict(xq=20488), dict(xd=24580), dict(ldx=66), dict(ldr=68), dict(no=28672, ldn=65)):
        assert call(**kw) == mis, kw
    if not torch.cuda.is_available():
        assert call() == h32.H32_ERR_UNSUPPORTED
        assert call(ro=None) == h32.H32_ERR_UNSUPPORTED
        assert call(ro=8192, no=28672, xq=None, xd=None) == h32.H32_ERR_UNSUPPORTED
