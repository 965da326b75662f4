"""The block norms on rows whose mean square is in fp32's range and whose sum of
squares is not, against 64-bit references.

Bounds, in roundings of U = 2^-24 on the terms' magnitude: such a row's sum is
at most 32 terms a lane, 6 lane steps and 8 waves, 46 roundings, half of them
in its square root; with the products around it fewer than 64 enter a value of
the forward pass, 128 where two sums meet in the gradient, and a column sum
over 11 rows adds fewer than 64."""
import pytest
import torch

import block_ref as R
from fp8_block_scaled_x128_amd import ops
from test_gpu_block_norm import make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def wide_range(cols, dt, seed):
    """Rows of mean squares up to fp32's largest, between ordinary ones: the
    row sums of squares of rows 1, 2, 4, 7, 8 are past it."""
    g = torch.Generator().manual_seed(seed)
    edge = (2.0 ** 128 / cols) ** 0.5
    v = torch.randn(11, cols, generator=g, dtype=torch.float64)
    for i, sigma in enumerate([1.0, 1e19, 0.0, 0.5 * edge, 1.5 * edge, 1e-3, 1.0, 1.2e19, 1e19, 3e4, 1.0]):
        v[i] *= sigma / v[i].square().mean().sqrt()
    v[2, cols // 2] = (2e38 * cols) ** 0.5              # one value has it all
    v = v.to(dt)
    assert (v.double().square().mean(1) < 3.4e38).all()
    assert ((v.double().square().sum(1) > 3.5e38).nonzero()[:, 0] == torch.tensor([1, 2, 4, 7, 8])).all()
    return v.cuda()


WIDTHS = [64, 128, 200, 256, 512, 1000, 2560, 4104, 9728, 16384]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("kind,stream,wt", [("both", BF, BF), ("both", F32, F32), ("pre", BF, F32), ("pre", F32, BF),
                                            ("post", F32, BF)])
def test_forward_of_large_values(cols, kind, stream, wt):
    """Finite rows whose sum of squares overflows keep their factor, and the
    rows beside them their bytes."""
    t = make(11, cols, kind, stream, wt, 0, cols)
    ordinary = ops.block_norm(t["residual"], t["x"], w_pre=t["w_pre"], w_post=t["w_post"], scale=0.7)
    res, x = t["residual"], t["x"]
    if kind != "post":
        res = wide_range(cols, stream, cols)
    if x is not None:
        x = wide_range(cols, BF, cols + 1).flip(0).contiguous()
    o = ops.block_norm(res, x, w_pre=t["w_pre"], w_post=t["w_post"], scale=0.7)
    h, mh, y, my = R.norm(res, x, t["w_pre"], t["w_post"], None, 1, 0.7, EPS)
    R.close(o.h, h, mh, 64, "h")
    if kind != "post":
        R.close(o.y, y, my, 64, "y")
        R.check_codes(o.q, o.s, y, my, 64, "codes")
        assert (o.s > 0).any(1).all()
    mixed_r, mixed_x = t["residual"].clone(), None if x is None else t["x"].clone()
    mixed_r[7], mixed_r[8] = res[7], torch.inf
    if x is not None:
        mixed_x[2], mixed_x[3, 0] = x[2], torch.nan
    m = ops.block_norm(mixed_r, mixed_x, w_pre=t["w_pre"], w_post=t["w_post"], scale=0.7)
    same = [0, 1, 4, 5, 6, 9, 10]
    assert all(p is None or torch.equal(p[same], q[same]) for p, q in zip(m, ordinary))


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("stream,wt,gate_rows,dy_dt", [(BF, BF, 0, F32), (F32, F32, 3, BF), (F32, BF, 1, F32)])
def test_backward_of_large_values(cols, stream, wt, gate_rows, dy_dt):
    t = make(11, cols, "both", stream, wt, gate_rows, cols)
    Rg = max(1, gate_rows)
    g = torch.Generator().manual_seed(cols)
    dy = torch.randn(11, cols, generator=g).to(dy_dt).cuda()
    h, x = wide_range(cols, stream, cols), wide_range(cols, BF, cols + 1).flip(0).contiguous()
    a = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], rows_per_gate=Rg, scale=0.7, eps=EPS)
    o = ops.block_norm_backward(dy, None, h, x, **a)
    ref = R.norm_grad(dy, None, h, x, t["w_pre"], t["w_post"], t["gate"], Rg, 0.7, EPS)
    for name, (v, mag) in ref.items():
        R.close(getattr(o, name), v, mag, 192, name)
    # rows beside them: their bytes as without
    plain_h, plain_x = t["residual"].clone(), t["x"].clone()
    base = ops.block_norm_backward(dy, None, plain_h, plain_x, **a)
    plain_h[7], plain_x[2], plain_h[4, 1] = h[7], x[2], torch.inf
    m = ops.block_norm_backward(dy, None, plain_h, plain_x, **a)
    same = [0, 1, 3, 5, 6, 8, 9, 10]
    assert torch.equal(m.dres[same], base.dres[same]) and torch.equal(m.dx[same], base.dx[same])
