"""256 x 256 tiles of the integer products by their number of K slices (128 codes each) and
the length of the last one: the copies' offsets move back, and the last slice's missing
codes are cleared, at another place for one, two, three and more slices."""
import pytest
import torch

import int8_ref as R
from fp8_block_scaled_x128_amd import ops
from test_gpu_int8 import BF, F32, acts, groups_of, operands

pytestmark = pytest.mark.gpu
SLICES = [16, 128, 144, 240, 256, 272, 368, 384, 400, 496, 528, 656]


@pytest.mark.parametrize("K", SLICES)
def test_dense(K):
    """130 tiles, the last row and column of them partial."""
    M, N = 2500, 3080
    a, sa, b, sb = operands(M, N, K, K, full=True)
    for out in (BF, F32):
        c = ops.i8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out)
        R.check_product(c, R.product(a, sa, b, sb))


@pytest.mark.parametrize("K", SLICES)
@pytest.mark.parametrize("gather", [True, False])
def test_grouped(K, gather):
    counts, N = [300, 1, 0, 257, 256, 130], 520
    offsets, rows = groups_of(counts, 500, K)
    n, G = int(offsets[-1]), len(counts)
    a, sa, b, sb = operands(500 if gather else n, G * N, K, K + 1)
    at = rows.long() if gather else torch.arange(n)
    c = ops.i8_grouped_gemm(a.cuda(), sa.cuda(), b.view(G, N, K).cuda(), sb.view(G, N).cuda(), offsets.cuda(),
                            rows.cuda() if gather else None, F32)
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        R.check_product(c[lo:hi], R.product(a[at[lo:hi]], sa[at[lo:hi]], b[g * N:(g + 1) * N], sb[g * N:(g + 1) * N]))


@pytest.mark.parametrize("T,O", [(272, 368), (368, 272), (256, 400), (264, 520)])
def test_gradient_in_one_launch(T, O):
    """Both products of the gradient: sums over three and more slices of outputs and tokens."""
    I = 16392
    x, w, dy = acts(T, I, 61), acts(O, I, 62), acts(T, O, 63)
    g = ops.i8_linear_backward(dy.cuda(), (w.cuda(), x.cuda()))
    R.check_product(g.dx, R.product(*R.codes(dy), *R.codes(w.t().contiguous())))
    R.check_product(g.dw, R.product(*R.codes(dy.t().contiguous()), *R.codes(x.t().contiguous())))
