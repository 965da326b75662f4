"""The operators between the GEMMs at the edges of what they document: no
columns, the largest token counts, expert weights that do not fit."""
import pytest
import torch

from fp8_block_scaled_x128_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def test_no_columns():
    """Rows without columns: empty results, forward and backward."""
    e = lambda *s: torch.empty(s, dtype=BF, device="cuda")
    w = e(0)
    o = ops.block_norm(e(4, 0), e(4, 0), w_pre=w, w_post=w, gate=e(2, 0), rows_per_gate=2)
    assert o.h.shape == (4, 0) and o.y.shape == (4, 0) and o.q.shape == (4, 0) and o.s.shape == (4, 0)
    g = ops.block_norm_backward(e(4, 0), e(4, 0), o.h, e(4, 0), w_pre=w, w_post=w, gate=e(2, 0), rows_per_gate=2)
    assert g.dres.shape == (4, 0) and g.dgate.shape == (2, 0) and g.dw_pre.shape == (0,) and g.ws is None


# wide rows have four waves a token, narrower ones two and one: a workgroup of
# 256 threads per token, per two and per four
@pytest.mark.parametrize("T,H,k", [(1 << 24, 1544, 4), (1 << 25, 520, 4), ((1 << 26) - 1, 8, 1)])
def test_combine_gradient_of_many_tokens(T, H, k):
    """Up to the documented number of tokens (more threads than one launch
    holds).  Only some tokens have rows; dout of the others is as allocated."""
    toks = [0, 5, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, T - 2, T - 1]
    n = len(toks)
    g = torch.Generator().manual_seed(H)
    dout = torch.empty(T, H, dtype=BF, device="cuda")
    pos = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros(T, k, device="cuda")
    vals, wv = torch.randn(n, H, generator=g).to(BF), torch.randn(n, k, generator=g)
    y = torch.randn(n * k, H, generator=g).to(BF)
    at = torch.tensor(toks, device="cuda")
    dout[at], w[at] = vals.cuda(), wv.cuda()
    pos[at] = torch.arange(n * k, dtype=torch.int32).view(n, k).cuda()
    dy, dw = ops.moe_combine_backward(dout, y.cuda(), pos, w)
    u = torch.finfo(F32).eps / 2
    # a dot product: H / 64 terms per lane, the lanes' six steps, four waves
    terms = vals.double()[:, None, :] * y.double().view(n, k, H)
    err = (dw[at].cpu().double() - terms.sum(2)).abs()
    assert (err <= (H / 64 + 16) * u * terms.abs().sum(2)).all()
    want = wv.double()[:, :, None] * vals.double()[:, None, :]
    got = dy.cpu().double().view(n, k, H)
    assert ((got - want).abs() <= (torch.finfo(BF).eps / 2 + u) * want.abs() + 1e-38).all()
    dw[at] = 0
    assert int(torch.count_nonzero(dw)) == 0
    del dout, pos, w, dw
    torch.cuda.empty_cache()


def _small_layer(T=64, H=256, G=4, I=128):
    g = torch.Generator().manual_seed(5)
    bf = lambda *s: (0.1 * torch.randn(*s, generator=g)).to(BF).cuda()
    x = bf(T, H)
    qgu, sgu, _ = ops.quant_block2d(bf(G, 2 * I, H))
    wd = bf(G, I, H)
    qdt = torch.empty(G, H, I, dtype=torch.uint8, device="cuda")
    sdt = torch.empty(G, I // 128, H // 128, device="cuda")
    ops.fp8_quant_block2d(wd, G, I, H, H, None, 0, qdt, I, sdt)
    return x, [qgu, sgu, qdt, sdt], torch.randn(T, G, generator=g).cuda()


def test_expert_weights_that_do_not_fit_are_refused():
    """Shape, type, layout and device of the experts' codes and scales: a
    refusal before the products (they walk the experts by the sizes of qgu
    alone)."""
    x, w, z = _small_layer()
    codes = ops.quant_rowblock(x)
    ops.moe_forward_routed(codes, z, 2, *w)
    r = ops.moe_route(z, 2)
    qgu, sgu, qdt, sdt = w
    bad = [(0, qgu[:, :, ::2].expand(4, 256, 128)), (0, qgu.transpose(1, 2)), (0, qgu.float()), (0, qgu.cpu()),
           (0, qgu[:, :192].contiguous()), (1, sgu[:3]), (1, sgu[:, :1]), (1, sgu.double()), (1, sgu.cpu()),
           (1, sgu.reshape(4, 4)), (2, qdt[:3]), (2, qdt.transpose(1, 2).contiguous().transpose(1, 2)),
           (2, qdt.to(torch.int16)), (2, qdt.cpu()), (3, sdt[:, :, :1]), (3, sdt[0]), (3, sdt.half()), (3, sdt.cpu())]
    for i, t in bad:
        v = list(w)
        v[i] = t
        with pytest.raises(ValueError):
            ops.moe_forward_routed(codes, z, 2, *v)
        with pytest.raises(ValueError):
            ops.moe_forward(x, *v, r.offsets, r.row_token, r.token_rows, r.weights)


def test_scales_with_strides_of_their_own():
    """The scales' strides are used: a transposed buffer gives the same bytes."""
    x, w, z = _small_layer()
    codes = ops.quant_rowblock(x)
    a, _, _ = ops.moe_forward_routed(codes, z, 2, *w)
    v = [w[0], w[1].transpose(1, 2).contiguous().transpose(1, 2), w[2], w[3].transpose(0, 2).contiguous().transpose(0, 2)]
    b, _, _ = ops.moe_forward_routed((codes[0], codes[1].contiguous()), z, 2, *v)
    assert torch.equal(a, b)
