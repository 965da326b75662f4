"""The largest sizes that the integer entry points take."""
import pytest
import torch

import int8_ref as R
from fp8_block_scaled_x128_amd import ops

pytestmark = pytest.mark.gpu


def test_most_columns():
    """A row of 2^28 - 64 columns, each with its own scale: codes of 127 and its sign (0
    for a zero), zeros behind them, scales |x| / 127."""
    cols = (1 << 28) - 64
    x = torch.randn(1, cols, dtype=torch.bfloat16, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[0, ::1001] = 0
    q, s = ops.i8_quant(x, ops.AXIS_COL)
    assert q.shape == (cols, 16)
    v = x[0].float()
    assert torch.equal(s, v.abs() / torch.full((), 127.0, device="cuda"))
    assert torch.equal(q[:, 0], (127 * torch.sign(v)).to(torch.int8)) and not q[:, 1:].any()


def test_most_tiles_of_groups():
    """30 groups of five rows in tiles of 64 x 128, at most 32 x 524287 of them: the first
    and last columns and every 100003rd against the exact product, and no tile left out."""
    G, N, K = 30, 524287 * 128, 16
    M = 5 * G
    g = torch.Generator("cuda").manual_seed(2)
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    offsets = torch.arange(G + 1, device="cuda", dtype=torch.int32) * 5
    c = torch.full((M, N), torch.nan, dtype=torch.bfloat16, device="cuda")
    ops.int8_grouped_gemm(M, N, K, G, offsets, None, 0, a, K, sa, b, K, 0, sb, 0, c, N, ops.OUT_BF16)
    at = torch.cat([torch.arange(300), torch.arange(0, N, 100003), torch.arange(N - 300, N)]).cuda()
    R.check_product(c[:, at], R.product(a, sa, b[at], sb[at]))
    assert not torch.isnan(c[::5, ::64]).any() and not torch.isnan(c[4::5, 63::64]).any()
