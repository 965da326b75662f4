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
    """65535 groups of five rows in tiles of 64 x 128, 70654 x 237 of them: one expert's
    weights for all groups, every 4999th row against the exact product."""
    G, N, K = 65535, 237 * 128, 16
    M = 5 * G
    g = torch.Generator("cuda").manual_seed(2)
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    b = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sb = torch.rand(M, generator=g, device="cuda"), torch.rand(N, generator=g, device="cuda")
    offsets = torch.arange(G + 1, device="cuda", dtype=torch.int32) * 5
    c = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    ops.int8_grouped_gemm(M, N, K, G, offsets, None, 0, a, K, sa, b, K, 0, sb, 0, c, N, ops.OUT_BF16)
    at = torch.cat([torch.arange(0, M, 4999, device="cuda"), torch.arange(M - 70, M, device="cuda")])
    R.check_product(c[at], R.product(a[at].cpu(), sa[at].cpu(), b.cpu(), sb.cpu()))
    assert not (c[:, ::61] == 3.0).all(dim=1).any()         # no row left out
