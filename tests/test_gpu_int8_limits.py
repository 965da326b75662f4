"""The largest sizes that the integer entry points take."""
import pytest
import torch

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
