"""Refusals of h32_moe_route_scored, in the binding and in the library, and pins of
the float64 rule it is tested against (closed forms)."""
import ctypes

import numpy as np
import pytest
import torch

import hadamard_rotated_bit_gb300 as h32
import oracle
from hadamard_rotated_bit_gb300 import _build

f32, i32 = torch.float32, torch.int32


def _raises(match, *args, **kw):
    with pytest.raises(ValueError, match=match):
        h32.h32_moe_route_scored(*args, **kw)


def test_binding_refusals():
    l = torch.zeros((6, 16))
    _raises("must be a CUDA tensor", l, 4)
    _raises("logits: dtype", l.double(), 4)
    _raises("logits must be 2-D with contiguous", l.t(), 4)
    _raises("score must be", l, 4, score="tanh")
    _raises("k must be", l, 0)
    _raises("bias: shape", l, 4, bias=torch.zeros(15))
    _raises("bias: dtype", l, 4, bias=torch.zeros(16, dtype=torch.bfloat16))
    _raises("topk_id: shape", l, 4, topk_id=torch.zeros((6, 3), dtype=i32))
    _raises("topk_w: dtype", l, 4, topk_w=torch.zeros((6, 4), dtype=torch.float64))
    _raises("expert_off: shape", l, 4, expert_off=torch.zeros(16, dtype=i32))
    _raises("row_idx: shape", l, 4, row_idx=torch.zeros(23, dtype=i32))
    _raises("row_of: shape", l, 4, row_of=torch.zeros((5, 4), dtype=i32))


def test_library_refusals():
    _build.build()
    p = 4096

    def call(l=p, T=4, E=16, ldl=16, score=0, bias=None, G=1, tg=1, gt=1, k=2, rn=1, scale=1.0,
             ids=p, w=p, off=p, ridx=p, rof=p, ws=None, nws=0):
        v = ctypes.c_void_p
        return h32.lib().h32_moe_route_scored(v(l), T, E, ldl, score, v(bias), G, tg, gt, k, rn, scale,
                                              v(ids), v(w), v(off), v(ridx), v(rof), v(ws), nws,
                                              v(0))

    for kw in (dict(T=-1), dict(E=0), dict(E=1025, ldl=1025), dict(ldl=15), dict(k=0), dict(k=17),
               dict(E=64, ldl=64, k=33), dict(score=2), dict(score=-1), dict(G=0), dict(G=3),
               dict(E=128, ldl=128, G=64), dict(G=4, tg=5), dict(G=4, tg=0), dict(gt=0), dict(gt=3),
               dict(G=8, tg=1, k=3), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(l=None), dict(ids=None), dict(w=None), dict(off=None), dict(ridx=None),
               dict(rof=None), dict(T=1 << 30), dict(T=65, ws=p, nws=100)):
        assert call(**kw) == h32.H32_ERR_INVALID_ARG, kw
    for kw in (dict(l=4098), dict(bias=4097), dict(ids=4104), dict(w=4098), dict(off=4097),
               dict(ridx=4098), dict(rof=4099), dict(T=65, ws=4100, nws=1 << 20)):
        assert call(**kw) == h32.H32_ERR_ALIGNMENT, kw
    if not torch.cuda.is_available():
        assert call() == h32.H32_ERR_UNSUPPORTED


def test_rule_without_groups_is_the_plain_router():
    l = np.random.default_rng(3).standard_normal((50, 24)).astype(np.float32)
    a = oracle.moe_route(l, 5)
    for kw in ({}, dict(n_group=4, topk_group=4, group_top=2)):
        b = oracle.moe_route_scored(l, 5, **kw)
        for i in (0, 2, 3, 4):
            assert np.array_equal(a[i], b[i])
        assert np.allclose(a[1], b[1], rtol=2e-6, atol=0)


def test_rule_closed_forms():
    l = np.zeros((1, 8), np.float32)
    ids, w, off, _, _ = oracle.moe_route_scored(l, 3, score="sigmoid", scale=2.0)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 2.0 / 3.0)
    ids, w, _, _, _ = oracle.moe_route_scored(l, 3, score="sigmoid", renormalize=False)
    assert np.allclose(w, 0.5)
    _, w, _, _, _ = oracle.moe_route_scored(l, 3, renormalize=False)
    assert np.allclose(w, 1.0 / 8.0)
    # the bias moves the choice, not the weight
    b = np.zeros(8, np.float32)
    b[6] = 1.0
    ids, w, _, _, _ = oracle.moe_route_scored(l, 1, score="sigmoid", bias=b, renormalize=False)
    assert ids.tolist() == [[6]] and w.tolist() == [[0.5]]
    # groups by their best, or by their two best: {0.9, -9, ..} against {0.8, 0.8, ..}
    l = np.full((1, 8), -9.0, np.float32)
    l[0, 0], l[0, 4], l[0, 5] = 2.2, 1.4, 1.4
    assert oracle.moe_route_scored(l, 1, "sigmoid", n_group=2, topk_group=1)[0].tolist() == [[0]]
    assert oracle.moe_route_scored(l, 1, "sigmoid", n_group=2, topk_group=1,
                                   group_top=2)[0].tolist() == [[4]]
    # a masked expert is not chosen while others are left, whatever its bias
    l[0, 0] = -np.inf
    b = np.zeros(8, np.float32)
    b[0] = 5.0
    assert 0 not in oracle.moe_route_scored(l, 7, "sigmoid", bias=b)[0]


def test_token_counts_whose_row_count_wraps():
    """T k above 2^63: refused, not taken modulo 2^64 (by both routers)."""
    _build.build()
    v = ctypes.c_void_p
    p, E, k = v(4096), 64, 32
    for T in (1 << 59, (1 << 59) + 5, 1 << 62, (1 << 63) - 1):
        assert h32.lib().h32_moe_route_scored(p, T, E, E, 0, v(0), 1, 1, 1, k, 1, 1.0, p, p, p, p, p, v(0), 0,
                                              v(0)) == h32.H32_ERR_INVALID_ARG
        assert h32.lib().h32_moe_route(p, T, E, E, k, p, p, p, p, p, v(0)) == h32.H32_ERR_INVALID_ARG
