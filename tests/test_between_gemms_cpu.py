"""Host validation of the block norms, the router and the combine's gradient:
every refusal happens before a device is touched (CPU only)."""
import pytest

from fp8_block_scaled_x128_amd import ops

A = 1 << 20     # never dereferenced
INF, NAN = float("inf"), float("nan")


def norm(rows=4, cols=256, x=A, ld=None, res=A, st=0, gate=None, R=1, scale=1.0, w_post=A, w_pre=A, wt=0, eps=1e-6,
         h=A, y=A, q=A, s=A, ld_x=None, ld_h=None, ld_q=None):
    ld = cols if ld is None else ld
    o = lambda v: ld if v is None else v
    return ops.fp8_block_norm(rows, cols, x, o(ld_x), res, ld, st, gate, ld, R, scale, w_post, w_pre, wt, eps, h,
                              o(ld_h), y, ld, q, o(ld_q), s, 1, max(rows, 1), stream=0, raise_on_error=False)


@pytest.mark.parametrize("args,status", [
    (dict(rows=-1), 2), (dict(cols=100), 2), (dict(cols=16392), 2), (dict(rows=1 << 31), 2), (dict(gate=A, R=0), 2),
    (dict(st=2), 5), (dict(wt=7), 5), (dict(eps=0.0), 5), (dict(eps=1e-40), 5), (dict(eps=NAN), 5), (dict(eps=INF), 5),
    (dict(scale=NAN), 5), (dict(scale=INF), 5),
    (dict(x=None, res=None, w_post=None), 1), (dict(x=None), 1), (dict(x=None, w_post=None, gate=A), 1),
    (dict(s=None), 1), (dict(q=None), 1), (dict(w_pre=None), 1), (dict(y=None, q=None, s=None), 1),
    (dict(w_pre=None, y=None, q=None, s=None, h=None), 1),
    (dict(ld_x=248), 3), (dict(ld_h=128), 3), (dict(ld_q=0), 3),
    (dict(ld_x=260), 4), (dict(x=A + 2), 4), (dict(res=A + 8), 4), (dict(w_pre=A + 4), 4), (dict(w_post=A + 8), 4),
    (dict(h=A + 8), 4), (dict(y=A + 4), 4), (dict(q=A + 4), 4), (dict(s=A + 2), 4), (dict(gate=A + 8), 4),
    (dict(rows=0, x=None, res=None), 0), (dict(cols=0), 0)])
def test_block_norm(args, status):
    assert norm(**args) == status


def norm_bwd(rows=4, cols=256, dy=A, dyt=0, dh=A, h=A, st=0, x=A, gate=None, R=1, scale=1.0, w_post=A, w_pre=A, wt=0,
             eps=1e-6, dx=A, dres=A, dgate=None, dgt=1, dw_post=A, dw_pre=A, ws=A, wsb=1 << 40, ld_dx=None):
    ld = cols
    return ops.fp8_block_norm_backward(rows, cols, dy, ld, dyt, dh, ld, h, ld, st, x, ld, gate, ld, R, scale, w_post,
                                       w_pre, wt, eps, dx, ld if ld_dx is None else ld_dx, dres, ld, dgate, ld, dgt,
                                       dw_post, dw_pre, ws, wsb, stream=0, raise_on_error=False)


@pytest.mark.parametrize("args,status", [
    (dict(rows=-1), 2), (dict(cols=12), 2), (dict(gate=A, dgate=A, R=0), 2), (dict(wsb=16), 2),
    (dict(dyt=9), 5), (dict(dgt=-1), 5), (dict(st=3), 5), (dict(eps=-1.0), 5), (dict(scale=NAN), 5),
    (dict(dy=None), 1), (dict(h=None), 1), (dict(w_pre=None), 1), (dict(x=None), 1), (dict(dgate=A), 1),
    (dict(w_post=None), 1), (dict(ws=None), 1),
    (dict(dy=None, h=None, w_pre=None, dw_pre=None, dh=None), 1),
    (dict(dx=None, dres=None, dw_post=None, dw_pre=None), 1),
    (dict(ld_dx=128), 3), (dict(ld_dx=260), 4), (dict(dy=A + 8), 4), (dict(dw_pre=A + 4), 4), (dict(ws=A + 8), 4),
    (dict(cols=0), 0)])
def test_block_norm_backward(args, status):
    assert norm_bwd(**args) == status


def test_block_norm_backward_workspace():
    f = ops.fp8_block_norm_backward_ws_size
    assert f(4096, 2560, 1, False, False, False) == 0
    assert f(0, 2560, 1, True, True, False) == 0
    one = f(4096, 2560, 1, True, False, False)
    assert 0 < one <= 4096 * 2560 * 4 and one % (2560 * 4) == 0
    assert f(4096, 2560, 1, True, True, False) == 2 * one
    # a gate row of one token has its gradient written straight out
    assert f(4096, 2560, 1, True, True, True) == 2 * one
    assert f(4096, 2560, 2048, False, False, True) > 0
    with pytest.raises(ops.Fp8bsError):
        f(4096, 2560, 0, False, False, True)
    with pytest.raises(ops.Fp8bsError):
        f(4096, 2561, 1, False, False, False)


def route(T=100, E=16, ld=None, t=1, k=2, renorm=1, z=A, mask=None, experts=A, counts=A, loss=A, ws=A, wsb=1 << 30,
          lse=A):
    return ops.fp8_moe_route(z, T, E, E if ld is None else ld, t, k, renorm, mask, experts, A, counts, A, A, A, lse,
                             loss, ws, wsb, stream=0, raise_on_error=False)


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), 2), (dict(T=(1 << 22) + 1), 2), (dict(E=0), 2), (dict(E=1025), 2),
    (dict(k=0), 2), (dict(k=17), 2), (dict(E=64, k=33), 2), (dict(wsb=8), 2), (dict(t=2), 5), (dict(renorm=2), 5),
    (dict(ld=15), 3), (dict(z=None), 1), (dict(experts=None), 1), (dict(counts=None), 1), (dict(loss=None), 1),
    (dict(lse=None), 1), (dict(ws=None), 1), (dict(z=A + 2), 4), (dict(t=0, z=A + 1), 4), (dict(counts=A + 2), 4),
    (dict(ws=A + 8), 4)])
def test_route(args, status):
    assert route(**args) == status


def test_route_workspace():
    assert ops.fp8_moe_route_ws_size(0, 128) == 0 and ops.fp8_moe_route_ws_size(64, 128) == 0
    assert ops.fp8_moe_route_ws_size(65, 128) > 0
    with pytest.raises(ops.Fp8bsError):
        ops.fp8_moe_route_ws_size(-1, 128)
    with pytest.raises(ops.Fp8bsError):
        ops.fp8_moe_route_ws_size(10, 2000)


def route_bwd(T=100, E=16, ld=None, t=1, k=2, renorm=1, z=A, experts=A, weights=A, counts=A, lse=A, dw=A, dl=A, out=A,
              ld_d=None):
    return ops.fp8_moe_route_backward(z, T, E, E if ld is None else ld, t, k, renorm, experts, weights, counts, lse,
                                      dw, dl, out, E if ld_d is None else ld_d, stream=0, raise_on_error=False)


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), 2), (dict(k=17), 2), (dict(E=2000), 2), (dict(t=5), 5), (dict(renorm=-1), 5), (dict(ld=3), 3),
    (dict(ld_d=3), 3), (dict(dw=None, dl=None), 1), (dict(experts=None), 1), (dict(weights=None), 1),
    (dict(counts=None), 1), (dict(lse=None), 1), (dict(out=None), 1), (dict(z=None), 1), (dict(out=A + 2), 4),
    (dict(dl=A + 1), 4), (dict(T=0, z=None, out=None), 0)])
def test_route_backward(args, status):
    assert route_bwd(**args) == status


def comb_bwd(T=10, k=2, rows=20, H=64, dout=A, t=0, y=A, pos=A, w=A, dy=A, dw=A, ld_do=None, ld_y=None, ld_dy=None):
    o = lambda v: H if v is None else v
    return ops.fp8_moe_combine_backward(dout, o(ld_do), t, y, rows, H, o(ld_y), pos, w, T, k, dy, o(ld_dy), dw,
                                        stream=0, raise_on_error=False)


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), 2), (dict(k=0), 2), (dict(H=60), 2), (dict(rows=-1), 2), (dict(T=1 << 26), 2), (dict(t=3), 5),
    (dict(dout=None), 1), (dict(y=None), 1), (dict(pos=None), 1), (dict(w=None), 1), (dict(dy=None, dw=None), 1),
    (dict(ld_do=56), 3), (dict(ld_y=56), 3), (dict(ld_dy=56), 3), (dict(ld_do=68), 4), (dict(y=A + 8), 4),
    (dict(dy=A + 2), 4), (dict(dw=A + 2), 4), (dict(T=0, dout=None), 0)])
def test_combine_backward(args, status):
    assert comb_bwd(**args) == status


def test_routed_combine_keeps_the_combines_checks():
    c = lambda y=A, rows=4, H=64, k=2, out=A: ops.fp8_moe_combine_routed(y, rows, H, H, A, A, 3, k, out, H, 0,
                                                                         stream=0, raise_on_error=False)
    assert c(H=60) == 2 and c(k=0) == 2 and c(y=None) == 1 and c(out=None) == 1 and c(out=A + 4) == 4
