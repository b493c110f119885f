"""Routed expert layer without a GPU: the formulas' gradients against differences, the plain forms
against each other, and what the entry points refuse on the host."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from fp8_fine_grained_fp8q_b200 import build, ops, synth
from tests import _moe

OK, ERR_ARG, ERR_SHAPE, ERR_ALIGN, ERR_UNSUPPORTED = 0, 1, 2, 3, 5
FAKE = 1 << 40
P = ctypes.c_void_p
A = P(FAKE)
ODD = P(FAKE + 2)
HALF = P(FAKE + 8)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.lib()


# -- formulas ------------------------------------------------------------------------------------- #

@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(5)
    T, E, k, scale, h = 4, 12, 3, 2.5, 1e-6
    l, dw = rng.normal(size=(T, E)), rng.normal(size=(T, k))
    idx, _ = _moe.route(l, k, score=score, renormalize=renorm, scale=scale)

    def loss(x):
        total = 0.0
        for t in range(T):
            s, masked = _moe.scores(x[t], score)
            total += (dw[t] * _moe.weights_of(x[t], idx[t], masked, s, score, renorm, scale)).sum()
        return total

    got, _ = _moe.route_backward(dw, idx, l, score, renorm, scale)
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(l)
            d[t, e] = h
            # Central differences: h^2 / 6 times the third derivative (below 10 here), and 2^-53 |L| / h.
            assert abs((loss(l + d) - loss(l - d)) / (2 * h) - got[t, e]) < 1e-8


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(6)
    g, u, da, h = rng.normal(size=200) * 3, rng.normal(size=200), rng.normal(size=200), 1e-6
    (dg, du, a), _ = _moe.swiglu_backward(da, g, u)
    f = lambda g, u: g * _moe.sigmoid(g) * u   # noqa: E731
    assert np.allclose(a, f(g, u), rtol=1e-14)
    assert np.allclose(dg, da * (f(g + h, u) - f(g - h, u)) / (2 * h), atol=2e-8)
    assert np.allclose(du, da * (f(g, u + h) - f(g, u - h)) / (2 * h), atol=2e-8)


def test_plain_quantisers_agree_with_the_oracle():
    off = np.array([0, 1, 1, 130, 200], np.int32)
    bits = synth.activations_channel_outliers(200, 256, seed=3)
    v = synth.bf16_bits_to_f32(bits)
    for got, want in ((_moe.quant_rows(v), oracle.quant_1x128(bits)),
                      (_moe.quant_cols(v, off), oracle.quant_128x1_t_ragged(bits, off))):
        assert np.array_equal(got[0], want[0])
        assert np.array_equal(got[1].view(np.uint32), want[1].view(np.uint32))


# -- refusals on the host --------------------------------------------------------------------------- #

def test_route_host_checks(L):
    def f(logits=A, kind=0, bias=None, T=4, E=64, k=8, ng=1, kg=1, score=0, renorm=1, scale=1.0, idx=A, w=A):
        return L.fp8q_moe_route(logits, kind, bias, T, E, k, ng, kg, score, renorm, scale, idx, w, None)

    assert f(T=-1) == f(E=0) == f(k=0) == f(k=65) == f(kind=2) == f(score=2) == f(ng=0) == ERR_ARG
    assert f(ng=3) == f(ng=8, kg=9) == f(ng=8, kg=0) == f(ng=16, kg=1) == ERR_ARG   # 64 % 3; 4 experts for k = 8
    assert f(scale=0.0) == f(scale=INF) == f(scale=NAN) == ERR_ARG
    assert f(E=1025) == f(k=33) == f(ng=64, kg=64) == f(T=1 << 40) == f(T=(1 << 31) // 8) == ERR_UNSUPPORTED
    assert f(logits=None) == f(idx=None) == f(w=None) == ERR_ARG
    assert f(logits=ODD) == f(bias=ODD) == f(idx=ODD) == f(w=ODD) == ERR_ALIGN
    assert f(T=0, logits=None, idx=None, w=None) == OK


def test_route_backward_host_checks(L):
    def f(dw=A, w=A, idx=A, logits=A, kind=0, T=4, E=64, k=8, score=0, renorm=1, scale=1.0, out=A):
        return L.fp8q_moe_route_backward(dw, w, idx, logits, kind, T, E, k, score, renorm, scale, out, None)

    assert f(T=-1) == f(E=0) == f(k=65) == f(kind=-1) == f(score=5) == f(scale=0.0) == ERR_ARG
    assert f(E=2000) == f(k=33) == ERR_UNSUPPORTED
    assert f(dw=None) == f(w=None) == f(idx=None) == f(logits=None) == f(out=None) == ERR_ARG
    assert f(dw=ODD) == f(out=ODD) == ERR_ALIGN
    assert f(T=0) == OK


def test_plan_host_checks(L):
    def f(idx=A, T=4, k=8, E=64, offsets=A, slots=A, rows=A):
        return L.fp8q_moe_plan(idx, T, k, E, offsets, slots, rows, None)

    assert f(T=-1) == f(k=0) == f(E=0) == ERR_ARG
    assert f(E=1025) == f(k=33) == f(T=1 << 31) == ERR_UNSUPPORTED
    assert f(idx=None) == f(offsets=None) == f(slots=None) == f(rows=None) == f(T=0, offsets=None) == ERR_ARG
    assert f(idx=ODD) == f(rows=ODD) == ERR_ALIGN


def test_dispatch_host_checks(L):
    def f(x=A, off=A, slots=A, rows=A, w=None, E=4, T=4, k=2, C=128, q=A, s=A, qt=None, st=None, cap=0):
        return L.fp8q_moe_dispatch(x, off, slots, rows, w, E, T, k, C, q, s, qt, st, cap, None)

    assert f(T=-1) == f(k=0) == f(E=0) == f(C=-128) == f(cap=-128) == ERR_ARG
    assert f(C=64) == f(qt=A, st=A, cap=100) == ERR_SHAPE
    assert f(E=1025) == f(k=64) == f(T=1 << 31) == f(C=1 << 32) == ERR_UNSUPPORTED
    assert f(x=None) == f(off=None) == f(slots=None) == f(rows=None) == f(q=None) == f(s=None) == ERR_ARG
    assert f(qt=A, cap=128) == f(st=A, cap=128) == ERR_ARG              # one of the two
    assert f(x=HALF) == f(q=HALF) == f(s=HALF) == f(off=ODD) == f(w=ODD) == f(qt=HALF, st=A, cap=128) == ERR_ALIGN
    assert f(T=0) == f(C=0) == OK


def test_combine_host_checks(L):
    def f(y=A, rows=A, w=None, add=None, T=4, k=2, C=64, out=A):
        return L.fp8q_moe_combine(y, rows, w, add, T, k, C, out, None)

    assert f(T=-1) == f(k=0) == f(C=-8) == f(y=None) == f(rows=None) == f(out=None) == ERR_ARG
    assert f(C=4) == ERR_SHAPE
    assert f(k=33) == f(T=1 << 31) == ERR_UNSUPPORTED
    assert f(y=HALF) == f(add=HALF) == f(out=HALF) == f(rows=ODD) == f(w=ODD) == ERR_ALIGN
    assert f(T=0) == f(C=0) == OK

    def g(dout=A, y=A, rows=A, T=4, k=2, C=64, dw=A):
        return L.fp8q_moe_combine_dweight(dout, y, rows, T, k, C, dw, None)

    assert g(T=-1) == g(k=0) == g(dout=None) == g(y=None) == g(rows=None) == g(dw=None) == ERR_ARG
    assert g(C=12) == ERR_SHAPE
    assert g(k=33) == ERR_UNSUPPORTED
    assert g(dout=HALF) == g(y=HALF) == g(rows=ODD) == g(dw=ODD) == ERR_ALIGN
    assert g(T=0) == OK


def test_swiglu_host_checks(L):
    def f(h=A, M=4, I=128, q=A, s=A, hq=A, hs=A):
        return L.fp8q_swiglu_quant(h, M, I, q, s, hq, hs, None)

    assert f(M=-1) == f(h=None) == f(q=None) == f(s=None) == f(hq=None) == f(hs=None) == ERR_ARG
    assert f(I=64) == ERR_SHAPE
    assert f(M=1 << 31) == f(I=1 << 30) == ERR_UNSUPPORTED
    assert f(h=HALF) == f(q=HALF) == f(hs=HALF) == ERR_ALIGN
    assert f(M=0) == f(I=0) == OK

    def g(da=A, hq=A, hs=A, off=A, E=2, M=4, I=128, q=A, s=A, qt=A, st=A, aqt=A, ast=A, cap=384):
        return L.fp8q_swiglu_backward_quant(da, hq, hs, off, E, M, I, q, s, qt, st, aqt, ast, cap, None)

    assert g(M=-1) == g(E=0) == g(off=None) == g(da=None) == g(aqt=None) == g(ast=None) == g(st=None) == ERR_ARG
    assert g(I=192) == g(cap=200) == g(off=None, E=1, M=300, cap=256) == ERR_SHAPE
    assert g(E=1025) == g(M=1 << 31) == ERR_UNSUPPORTED
    assert g(da=HALF) == g(qt=HALF) == g(off=ODD) == ERR_ALIGN
    assert g(M=0) == g(I=0) == OK


def test_binding_refuses_host_tensors_and_wrong_types():
    bf = torch.zeros(4, 256, dtype=torch.bfloat16)
    idx = torch.zeros(4, 2, dtype=torch.int32)
    plan = ops.MoePlan(torch.zeros(9, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), idx)
    for call in (lambda: ops.moe_route(torch.zeros(4, 8), 2), lambda: ops.moe_plan(idx, 8),
                 lambda: ops.moe_dispatch(bf, plan), lambda: ops.moe_combine(bf, plan),
                 lambda: ops.moe_combine_dweight(bf, bf, plan), lambda: ops.swiglu_quant(bf),
                 lambda: ops.swiglu_backward_quant(bf, idx, idx)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        ops.moe_route(torch.zeros(4, 8, dtype=torch.float16), 2)
