"""CPU tests of the routed feed-forward's and the 4-bit weights' entry points: what the host refuses
before any launch, and what the binding refuses before the C call."""
import ctypes

import pytest
import torch

import fp16_gemm_b200 as sp


def _raw(fn, *args):
    return getattr(sp.lib(), fn)(*args)


def test_route_refusals():
    f = lambda dt=sp.F32, T=4, E=8, k=2, sc=0, a=16, r=16, w=16: _raw("sp24_moe_route", a, dt, T, E, k, sc, 1, r, w, None)  # noqa: E731
    assert f(dt=sp.NVFP4) == sp.ERR_DTYPE
    assert f(sc=2) == sp.ERR_INVALID_ARG
    assert f(T=-1) == f(E=0) == f(k=0) == f(k=9) == sp.ERR_SHAPE
    assert f(E=1025) == f(E=64, k=33) == f(T=2**31) == sp.ERR_UNSUPPORTED
    assert f(a=None) == f(r=None) == f(w=None) == sp.ERR_INVALID_ARG
    assert f(a=18) == f(r=18) == f(w=18) == f(dt=sp.BF16, a=17) == sp.ERR_ALIGN
    assert f(T=0, a=None, r=None, w=None) == sp.OK
    b = lambda T=4, d=16, dl=16, r=16, dt=sp.F32: _raw("sp24_moe_route_backward", 16, dt, r, d, T, 8, 2, 0, 1, dl, None)  # noqa: E731
    assert b(d=None) == b(dl=None) == b(r=None) == sp.ERR_INVALID_ARG
    assert b(dl=18) == b(d=18) == b(dl=17, dt=sp.F16) == sp.ERR_ALIGN
    assert b(T=0, d=None) == sp.OK


def test_sort_refusals():
    def f(x=16, dt=sp.BF16, T=4, k=2, E=8, H=16, xs=16, pos=16, src=16, re=16, off=16, r=16):
        return _raw("sp24_moe_sort", x, dt, r, T, k, E, H, xs, pos, src, re, off, None, 0, None)
    assert f(dt=sp.NVFP4) == sp.ERR_DTYPE
    assert f(T=-1) == f(k=0) == f(E=0) == f(H=-1) == sp.ERR_SHAPE
    assert f(E=2**16 + 1) == f(T=2**30, k=2) == f(T=2**31) == sp.ERR_UNSUPPORTED
    assert f(pos=None) == f(src=None) == f(re=None) == f(off=None) == f(r=None) == sp.ERR_INVALID_ARG
    assert f(x=None) == f(xs=None) == sp.ERR_INVALID_ARG
    assert f(x=17) == f(xs=17) == f(pos=18) == f(off=18) == sp.ERR_ALIGN
    n = ctypes.c_int64(-1)
    assert _raw("sp24_moe_sort_workspace_size", 4, 2, 8, None) == sp.ERR_INVALID_ARG
    assert _raw("sp24_moe_sort_workspace_size", 4, 2, 0, ctypes.byref(n)) == sp.ERR_SHAPE
    assert _raw("sp24_moe_sort_workspace_size", 4, 2, 8, ctypes.byref(n)) == sp.OK and n.value >= 0


def test_unsort_refusals():
    def f(ys=16, a=sp.BF16, pos=16, w=16, T=4, k=2, rows=8, H=16, y=16, b=sp.BF16):
        return _raw("sp24_moe_unsort", ys, a, pos, w, T, k, rows, H, y, b, None)
    assert f(a=sp.NVFP4) == f(b=9) == f(a=sp.BF16, b=sp.F16) == f(a=sp.F16, b=sp.BF16) == sp.ERR_DTYPE
    assert f(T=-1) == f(k=0) == f(rows=-1) == f(H=-1) == sp.ERR_SHAPE
    assert f(k=65) == f(T=2**30) == f(rows=2**31) == sp.ERR_UNSUPPORTED
    assert f(ys=None) == f(pos=None) == f(y=None) == sp.ERR_INVALID_ARG
    assert f(ys=17) == f(y=17) == f(pos=18) == f(w=18) == sp.ERR_ALIGN
    assert f(T=0, ys=None, y=None, pos=None) == f(H=0, y=None) == sp.OK

    def g(dy=16, ys=16, dys=16, dw=16, a=sp.BF16, b=sp.BF16, T=4, k=2):
        return _raw("sp24_moe_unsort_backward", dy, b, ys, a, 16, 16, T, k, 8, 16, dys, dw, None)
    assert g(dy=None) == g(ys=None) == g(dys=None) == sp.ERR_INVALID_ARG
    assert g(a=sp.F16) == sp.ERR_DTYPE and g(k=65) == sp.ERR_UNSUPPORTED
    assert g(dys=17) == g(dw=18) == sp.ERR_ALIGN
    assert g(T=0, dy=None) == sp.OK


def test_rows_beyond_the_widest():
    h = 2**30 + 1
    assert _raw("sp24_moe_sort", 16, sp.BF16, 16, 4, 2, 8, h, 16, 16, 16, 16, 16, None, 0, None) == sp.ERR_UNSUPPORTED
    assert _raw("sp24_moe_unsort", 16, sp.BF16, 16, 16, 4, 2, 8, h, 16, sp.BF16, None) == sp.ERR_UNSUPPORTED
    assert _raw("sp24_moe_unsort_backward", 16, sp.BF16, 16, sp.BF16, 16, 16, 4, 2, 8, h, 16, 16, None) == sp.ERR_UNSUPPORTED


def _op(scale=sp.BF16, group=128, codes=16, scales=16, zeros=None):
    return sp._W4Operand(scale, group, codes, scales, zeros)


def test_w4_refusals():
    q = lambda w=16, dt=sp.BF16, R=4, K=256, G=128, z=0, c=16, s=16, zp=None: _raw("sp24_quantize_w4", w, dt, R, K, G, z, c, s, zp, None)  # noqa: E731
    assert q(dt=sp.F32) == sp.ERR_DTYPE
    assert q(G=16) == q(G=256) == q(G=0) == sp.ERR_UNSUPPORTED
    assert q(R=-1) == q(K=-128) == q(K=192) == sp.ERR_SHAPE
    assert q(z=1) == q(zp=16) == q(w=None) == q(c=None) == q(s=None) == sp.ERR_INVALID_ARG
    assert q(w=24) == q(c=24) == q(s=24) == sp.ERR_ALIGN
    assert q(R=0, w=None, c=None, s=None) == sp.OK
    d = lambda op, K=256, dt=sp.F32, out=16: _raw("sp24_dequantize_w4", ctypes.byref(op), 4, K, dt, out, None)  # noqa: E731
    assert d(_op(scale=sp.F32)) == d(_op(), dt=sp.NVFP4) == sp.ERR_DTYPE
    assert d(_op(group=48)) == sp.ERR_UNSUPPORTED and d(_op(), K=64) == sp.ERR_SHAPE
    assert d(_op(codes=None)) == d(_op(scales=None)) == d(_op(), out=None) == sp.ERR_INVALID_ARG
    assert d(_op(codes=8)) == d(_op(), out=8) == sp.ERR_ALIGN


@pytest.mark.parametrize("grouped", [False, True])
def test_gemv_w4_refusals(grouped):
    def f(op=None, x=16, dt=sp.BF16, M=2, E=3, N=6, K=256, act=0, y=16, ydt=sp.F32, off=16):
        op = _op() if op is None else op
        if grouped:
            return _raw("sp24_gemv_w4_grouped", x, dt, ctypes.byref(op), off, M, E, N, K, act, y, ydt, None)
        return _raw("sp24_gemv_w4", x, dt, ctypes.byref(op), M, N, K, act, y, ydt, None)
    assert f(dt=sp.F32) == f(ydt=sp.F16) == f(ydt=sp.NVFP4) == f(_op(scale=sp.F32)) == sp.ERR_DTYPE
    assert f(act=2) == f(x=None) == f(y=None) == f(_op(codes=None)) == f(_op(scales=None)) == sp.ERR_INVALID_ARG
    assert f(_op(group=96)) == f(K=2**24 + 128) == f(M=2**31) == f(N=2**31) == sp.ERR_UNSUPPORTED
    assert f(K=192) == f(K=-128) == f(M=-1) == f(N=-1) == f(N=5, act=1) == sp.ERR_SHAPE
    assert f(x=24) == f(y=18) == f(_op(codes=24)) == f(_op(scales=24)) == f(_op(zeros=24)) == sp.ERR_ALIGN
    assert f(M=0, x=None, y=None) == f(N=0, y=None) == sp.OK
    if grouped:
        assert f(E=0) == sp.ERR_SHAPE and f(off=None) == sp.ERR_INVALID_ARG and f(off=18) == sp.ERR_ALIGN


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    w = sp.W4Tensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.bfloat16))
    for call in (lambda: sp.moe_route(x, 2), lambda: sp.moe_route(logits=x, topk=2),
                 lambda: sp.moe_route_backward(x, x, ids), lambda: sp.moe_sort(x, ids, 8),
                 lambda: sp.moe_sort_tables(ids, 8), lambda: sp.moe_sort_backward(x, ids), lambda: sp.moe_unsort(x, ids),
                 lambda: sp.moe_unsort_backward(x, x, ids), lambda: sp.quantize_w4(x), lambda: sp.dequantize_w4(w),
                 lambda: sp.gemv_w4(x, w), lambda: sp.gemv_w4_grouped(x, w, ids)):
        with pytest.raises(ValueError):
            call()
