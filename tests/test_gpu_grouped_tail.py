"""The grouped products with fewer rows in their offsets than the buffers hold
(a padded batch): rows behind offsets[G] are not written, and what stands
there in the operands has no effect.  The rows in front are checked against
the oracle and the datapath model."""
import numpy as np
import pytest
import torch

from fp8_block_scaled_x128_amd import inputs, ops
from gpu_util import dev, dev_bf16, host, verify

pytestmark = pytest.mark.gpu
NAN = 0x7F                                   # E4M3 NaN
SIZES = [[0, 40, 0, 200, 1, 128, 0, 77], [300, 0, 0, 0, 0, 0, 0, 0], [0, 0, 0, 0, 0, 0, 0, 3]]


def _problem(sizes, tail, gather):
    """Quantized operands of a small layer whose offsets take sum(sizes) of
    `rows` rows; NaN codes and scales behind them (gather: tokens of their
    own, row indices 0 behind them)."""
    d = inputs.small_moe(seed=9, tokens=96)
    G, N2, K = d["w_gu"].shape
    n = sum(sizes)
    rows = n + tail
    rng = np.random.default_rng(n + tail)
    token = rng.integers(0, 96, n).astype(np.int32)
    offs = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    return d, G, N2, K, n, rows, token, offs


def _rows_of(q, s, token, rows, fill):
    """The rows of a non-gathered operand: token's, then NaN rows."""
    at = torch.from_numpy(token.astype(np.int64)).cuda()
    qa = torch.full((rows, q.shape[1]), NAN, dtype=torch.uint8, device="cuda")
    sa = torch.full((rows, s.shape[1]), fill, dtype=s.dtype, device="cuda")
    qa[:at.numel()], sa[:at.numel()] = q[at], s[at]
    return qa, sa


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("tail", [1, 150])
@pytest.mark.parametrize("gather", [True, False])
def test_block_scaled(sizes, tail, gather):
    d, G, N2, K, n, rows, token, offs = _problem(sizes, tail, gather)
    qx, sx = ops.quant_rowblock(dev_bf16(d["x"]), ops.AXIS_ROW, "m_major")
    qw, sw, _ = ops.quant_block2d(dev_bf16(d["w_gu"]))
    if gather:
        a, sa, count = qx, sx, qx.shape[0]
        a_rows = dev(np.concatenate([token, np.zeros(tail, np.int32)]))
    else:
        a, sa = _rows_of(qx, sx, token, rows, float("nan"))
        a_rows, count = None, rows
    arg = (G, dev(offs), a_rows, count, a, a.stride(0), sa, sa.stride(0), sa.stride(1), qw, K, N2 * K, sw,
           sw.stride(0), sw.stride(1), sw.stride(2))
    c32 = torch.full((rows, N2), 9.0, device="cuda")
    c16 = torch.full((rows, N2 + 8), 9.0, dtype=torch.bfloat16, device="cuda")
    ops.fp8_grouped_gemm(rows, N2, K, *arg, c32, N2, ops.OUT_FP32)
    ops.fp8_grouped_gemm(rows, N2, K, *arg, c16, N2 + 8, ops.OUT_BF16)
    I = N2 // 2
    qh = torch.full((rows, I), 0xA5, dtype=torch.uint8, device="cuda")
    sh = torch.full((I // 128, rows), 9.0, device="cuda")
    ops.fp8_grouped_gemm_swiglu_quant(rows, I, K, *arg, qh, I, sh, 1, rows)
    torch.cuda.synchronize()
    assert (c32[n:] == 9).all() and (c16[n:] == 9).all() and (c16[:, N2:] == 9).all()
    assert (qh[n:] == 0xA5).all() and (sh[:, n:] == 9).all()
    qx_h, sx_h, qw_h, sw_h = host(qx), host(sx.contiguous()), host(qw), host(sw)
    for g in range(G):
        r0, r1 = int(offs[g]), int(offs[g + 1])
        if r1 > r0:
            t = token[r0:r1]
            verify(qx_h[t], sx_h[t], qw_h[g], sw_h[g], host(c32[r0:r1]), np.ascontiguousarray(host(c16[r0:r1, :N2])))
    # the fused epilogue is the two calls in one
    gu = c16[:n, :N2].contiguous()
    q2, s2 = torch.empty((n, I), dtype=torch.uint8, device="cuda"), torch.empty((I // 128, n), device="cuda")
    ops.fp8_silu_mul_quant(gu, n, I, N2, 0, q2, I, s2, 1, n, None, 0)
    assert torch.equal(qh[:n], q2) and torch.equal(sh[:, :n], s2)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("tail", [1, 150])
@pytest.mark.parametrize("gather", [True, False])
def test_mx(sizes, tail, gather):
    d, G, N2, K, n, rows, token, offs = _problem(sizes, tail, gather)
    qx, sx = ops.mx_quant(dev_bf16(d["x"]))
    qw, sw = ops.mx_quant(dev_bf16(d["w_gu"]).view(G * N2, K))
    if gather:
        a, sa, count = qx, sx, qx.shape[0]
        a_rows = dev(np.concatenate([token, np.zeros(tail, np.int32)]))
    else:
        a, sa = _rows_of(qx, sx, token, rows, 0xFF)          # UE8M0 NaN
        a_rows, count = None, rows
    arg = (G, dev(offs), a_rows, count, a, K, sa, K // 32, qw, K, N2 * K, sw, K // 32, N2 * (K // 32))
    c32 = torch.full((rows, N2), 9.0, device="cuda")
    c16 = torch.full((rows, N2), 9.0, dtype=torch.bfloat16, device="cuda")
    ops.mxfp8_gemm(rows, N2, K, *arg, c32, N2, ops.OUT_FP32)
    ops.mxfp8_gemm(rows, N2, K, *arg, c16, N2, ops.OUT_BF16)
    I = N2 // 2
    qh = torch.full((rows, I), 0xA5, dtype=torch.uint8, device="cuda")
    sh = torch.full((rows, I // 32), 0xA5, dtype=torch.uint8, device="cuda")
    ops.mxfp8_grouped_gemm_swiglu_quant(rows, I, K, *arg, qh, I, sh, I // 32, 1)
    torch.cuda.synchronize()
    assert (c32[n:] == 9).all() and (c16[n:] == 9).all() and (qh[n:] == 0xA5).all() and (sh[n:] == 0xA5).all()
    qx_h, sx_h, qw_h, sw_h = host(qx), host(sx), host(qw).reshape(G, N2, K), host(sw).reshape(G, N2, K // 32)
    for g in range(G):
        r0, r1 = int(offs[g]), int(offs[g + 1])
        if r1 > r0:
            t = token[r0:r1]
            verify(qx_h[t], sx_h[t], qw_h[g], sw_h[g], host(c32[r0:r1]), host(c16[r0:r1]), mx=True)
    q2, s2 = torch.empty((n, I), dtype=torch.uint8, device="cuda"), torch.empty((n, I // 32), dtype=torch.uint8, device="cuda")
    ops.fp8_silu_mul_quant(c16[:n].contiguous(), n, I, N2, 1, q2, I, s2, I // 32, 1, None, 0)
    assert torch.equal(qh[:n], q2) and torch.equal(sh[:n], s2)
