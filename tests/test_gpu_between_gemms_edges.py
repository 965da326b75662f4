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
