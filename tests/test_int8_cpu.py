"""Refusals of the integer entry points (host validation; nothing is launched) and
the reference's own pins."""
import pytest
import torch

import int8_ref as R
from fp8_block_scaled_x128_amd import ops

P = 1 << 20                                   # never dereferenced: validation fails first
NULL, SHAPE, STRIDE, ALIGN, UNSUPPORTED = 1, 2, 3, 4, 5
GIB4 = 1 << 32


def quant(x=P, rows=4, cols=64, ld=64, axis=0, q=P, ldq=64, s=P):
    return ops.int8_quant(x, rows, cols, ld, axis, q, ldq, s, stream=0, raise_on_error=False)


@pytest.mark.parametrize("want,a", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=-8)), (SHAPE, dict(cols=20, ld=24)), (SHAPE, dict(rows=1 << 31)),
    (SHAPE, dict(axis=1, rows=65535 * 128 + 1)), (UNSUPPORTED, dict(axis=2)), (NULL, dict(x=None)), (NULL, dict(q=None)),
    (NULL, dict(s=None)), (STRIDE, dict(ld=56)), (STRIDE, dict(ldq=48)), (STRIDE, dict(cols=56, ldq=56)),
    (STRIDE, dict(axis=1, rows=70, ldq=72)), (ALIGN, dict(x=P + 8)), (ALIGN, dict(ld=68)), (ALIGN, dict(q=P + 8)),
    (ALIGN, dict(ldq=72)), (ALIGN, dict(s=P + 2))])
def test_quant_refuses(want, a):
    assert quant(**a) == want


@pytest.mark.parametrize("a", [dict(rows=1 << 26), dict(rows=1 << 24, cols=4104, ld=4104, ldq=4112),
                               dict(axis=1, cols=1 << 28, ld=1 << 28)])
def test_quant_refuses_more_than_a_launch_holds(a):
    assert quant(**a) == SHAPE
    assert gemm(N=(1 << 26) + 8, ldc=1 << 27) == SHAPE and linear(rows=1 << 26) == SHAPE


def silu(gu=P, rows=4, I=64, ld=128, live=None, q=P, ldq=64, s=P, h=None, ldh=0):
    return ops.int8_silu_mul_quant(gu, rows, I, ld, live, q, ldq, s, h, ldh, stream=0, raise_on_error=False)


@pytest.mark.parametrize("want,a", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(I=12)), (NULL, dict(gu=None)), (NULL, dict(q=None)), (STRIDE, dict(ld=120)),
    (STRIDE, dict(h=P, ldh=56)), (ALIGN, dict(h=P + 8, ldh=64)), (ALIGN, dict(live=P + 1)), (ALIGN, dict(gu=P + 2))])
def test_silu_refuses(want, a):
    assert silu(**a) == want


def gemm(M=4, N=64, K=64, a=P, lda=64, sa=P, b=P, ldb=64, sb=P, c=P, ldc=64, out=0, ws=None, wsn=0):
    return ops.int8_gemm(M, N, K, a, lda, sa, b, ldb, sb, c, ldc, out, ws, wsn, stream=0, raise_on_error=False)


PRODUCT = [(SHAPE, dict(M=-1)), (SHAPE, dict(K=72, lda=80, ldb=80)), (SHAPE, dict(N=60)),
           (SHAPE, dict(K=131072, lda=131072, ldb=131072)), (UNSUPPORTED, dict(out=2)), (NULL, dict(a=None)),
           (NULL, dict(b=None)), (NULL, dict(c=None)), (NULL, dict(sa=None)), (NULL, dict(sb=None)),
           (STRIDE, dict(lda=48)), (STRIDE, dict(ldb=48)), (STRIDE, dict(ldc=56)), (ALIGN, dict(a=P + 8)),
           (ALIGN, dict(b=P + 8)), (ALIGN, dict(lda=72)), (ALIGN, dict(ldb=72)), (ALIGN, dict(c=P + 8)),
           (ALIGN, dict(ldc=68)), (ALIGN, dict(sa=P + 1)), (ALIGN, dict(sb=P + 1)), (SHAPE, dict(lda=GIB4 // 4)),
           (SHAPE, dict(ldb=GIB4 // 64))]


@pytest.mark.parametrize("want,a", PRODUCT + [(ALIGN, dict(ws=P + 8, wsn=1 << 20)),
                                              (SHAPE, dict(M=64, N=2560, K=9728, lda=9728, ldb=9728, ldc=2560, ws=P, wsn=16))])
def test_gemm_refuses(want, a):
    assert gemm(**a) == want


def test_workspace_sizes():
    assert ops.int8_gemm_ws_size(0, 64, 64) == 0 and ops.int8_gemm_ws_size(4096, 9728, 2560) == 0
    n = ops.int8_gemm_ws_size(64, 2560, 9728)
    assert n > 0 and n % (64 * 2560 * 4) == 0
    for bad in ((-1, 8, 16), (8, -8, 16), (8, 8, -16), (8, 8, 131072), (1 << 31, 8, 16)):
        with pytest.raises(ops.Fp8bsError):
            ops.int8_gemm_ws_size(*bad)
        with pytest.raises(ops.Fp8bsError):
            ops.int8_linear_ws_size(*bad)


def grouped(M=4, N=64, K=64, G=2, offsets=P, rows=None, count=0, a=P, lda=64, sa=P, b=P, ldb=64, bsg=4096, sb=P, ssg=64,
            c=P, ldc=64, out=0):
    return ops.int8_grouped_gemm(M, N, K, G, offsets, rows, count, a, lda, sa, b, ldb, bsg, sb, ssg, c, ldc, out,
                                 stream=0, raise_on_error=False)


@pytest.mark.parametrize("want,a", PRODUCT + [
    (SHAPE, dict(G=0)), (SHAPE, dict(G=65536)), (NULL, dict(offsets=None)), (ALIGN, dict(offsets=P + 2)),
    (ALIGN, dict(rows=P + 2, count=4)), (SHAPE, dict(rows=P, count=0)), (ALIGN, dict(bsg=4104)), (STRIDE, dict(bsg=-16)),
    (STRIDE, dict(ssg=-1))])
def test_grouped_refuses(want, a):
    assert grouped(**a) == want


def linear(rows=4, N=64, cols=64, x=P, ldx=64, w=P, ldw=64, sw=P, y=P, ldy=64, out=0, ws=P, wsn=1 << 16):
    return ops.int8_linear(rows, N, cols, x, ldx, w, ldw, sw, y, ldy, out, ws, wsn, stream=0, raise_on_error=False)


@pytest.mark.parametrize("want,a", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=60)), (SHAPE, dict(N=4)), (NULL, dict(x=None)), (NULL, dict(w=None)),
    (NULL, dict(ws=None)), (SHAPE, dict(wsn=100)), (ALIGN, dict(ws=P + 8)), (STRIDE, dict(ldx=56)),
    (STRIDE, dict(cols=56, ldx=56, ldw=56)), (ALIGN, dict(x=P + 8)), (UNSUPPORTED, dict(out=7))])
def test_linear_refuses(want, a):
    assert linear(**a) == want


def backward(T=4, O=64, I=32, dy=P, ld_dy=64, w=P, ld_w=32, x=P, ld_x=32, dx=P, ld_dx=32, dw=P, ld_dw=32, ws=P, wsn=1 << 20):
    return ops.int8_linear_backward(T, O, I, dy, ld_dy, w, ld_w, x, ld_x, dx, ld_dx, dw, ld_dw, ws, wsn, stream=0,
                                    raise_on_error=False)


@pytest.mark.parametrize("want,a", [
    (SHAPE, dict(T=-1)), (SHAPE, dict(O=60)), (SHAPE, dict(I=20)), (SHAPE, dict(T=131057)), (SHAPE, dict(O=131064, ld_dy=131064)),
    (SHAPE, dict(T=131056, I=65536, ld_x=65536, ld_w=65536)), (NULL, dict(dy=None)), (NULL, dict(w=None)), (NULL, dict(x=None)),
    (NULL, dict(dx=None)), (NULL, dict(dw=None)), (NULL, dict(ws=None)), (SHAPE, dict(wsn=100)), (STRIDE, dict(ld_dy=56)),
    (STRIDE, dict(ld_w=24)), (STRIDE, dict(ld_x=24)), (STRIDE, dict(ld_dx=24)), (STRIDE, dict(ld_dw=24)), (ALIGN, dict(dy=P + 8)),
    (ALIGN, dict(w=P + 2)), (ALIGN, dict(ld_x=36)), (ALIGN, dict(dx=P + 8)), (ALIGN, dict(dw=P + 4)), (ALIGN, dict(ws=P + 8))])
def test_linear_backward_refuses(want, a):
    assert backward(**a) == want


def test_linear_backward_workspace():
    # scales (4 + 64 + 2 x 32 floats), codes (4 x 64, 64 x 16, 32 x 64, 32 x 16), the runs' maxima
    assert ops.int8_linear_backward_ws_size(4, 64, 32) == 16 + 256 + 256 + 256 + 1024 + 2048 + 512 + 128 + 64 + 64
    assert backward(I=0) == 0 and backward(T=0, O=0) == 0
    for bad in ((-1, 8, 8), (8, 12, 8), (8, 8, 4), (1 << 20, 8, 8)):
        with pytest.raises(ops.Fp8bsError):
            ops.int8_linear_backward_ws_size(*bad)


def test_empty_calls_need_no_device():
    assert quant(rows=0) == 0 and quant(axis=1, cols=0, ld=0) == 0 and silu(rows=0) == 0
    assert gemm(M=0) == 0 and gemm(N=0) == 0 and grouped(M=0) == 0 and linear(rows=0) == 0
    assert ops.int8_linear_ws_size(0, 8, 64) == 0 and ops.int8_linear_ws_size(5, 8, 40) == 32 + 5 * 48


def test_reference_codes():
    """Hand-made rows: a scale of 1 (ties to even), of 1/2, a subnormal one."""
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 3.0, -127.0], [63.5, 0.25, 0.75, -0.25, 1.0, 0.0, 0.3, -63.5]])
    q, s = R.codes(x)
    assert s.tolist() == [1.0, 0.5]
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, 3, -127] and q[1].tolist() == [127, 0, 2, 0, 2, 0, 1, -127]
    q, s = R.codes(torch.tensor([[0.0, 0.0], [torch.nan, 1.0], [torch.inf, 1.0]]))
    assert (q == 0).all() and s[0] == 0 and torch.isnan(s[1]) and s[2] == torch.inf
