"""The block norms beyond one pass of their row loops against 64-bit references.

How the kernels deal rows (so that each case here takes the path it says, and
for the bounds): a row of up to 128 / 256 / 512 columns has 16 / 32 / 64 lanes
of a wave, a wider one 64 lanes of up to eight waves with up to four chunks of
eight columns a lane.  The forward kernel starts a fixed number of workgroups
at most and walks the rows beyond.  The gradient deals units: every `splits`-th
run of rows, or with a shared gate a run inside one gate row, each walked by a
workgroup (or wave); column sums are a chain over a lane's rows, a sum over the
waves, and over the partial rows every 128th of them and a tree of 7.

Bounds, in roundings of U = 2^-24 on the terms' magnitude: a row's sum is at
most 32 terms a lane, 6 lane steps and 8 waves, 46 roundings, half of them in
its square root; with the products around it fewer than 64 enter a value of the
forward pass, 128 where two sums meet in the gradient."""
import pytest
import torch

import block_ref as R
from fp8_block_scaled_x128_amd import ops
from test_gpu_block_norm import make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
CUS = 256
ceil = lambda a, b: -(-a // b)


def layout(cols):
    """(waves of a row, chunks of a lane, lanes of a row within a wave)."""
    groups = ceil(cols // 8, 64)
    nv = ceil(groups, 8)
    return ceil(groups, nv), nv, 16 if cols <= 128 else 32 if cols <= 256 else 64


def forward_rows(cols):
    """Rows that the largest forward launch has in its first pass."""
    wpr, nv, lanes = layout(cols)
    waves = wpr if wpr > 1 else 4
    blocks = max(2 * CUS, 5120 // (waves * nv) // CUS * CUS)
    return blocks * (1 if wpr > 1 else 4 * 64 // lanes)


def backward_plan(rows, cols, gate_rows, fp32_rows=False):
    """(walked by waves, slots, rows a slot has at once, units, rows of a unit)."""
    wpr, nv, lanes = layout(cols)
    grouped = gate_rows > 1
    unit = min(gate_rows, rows) if grouped else rows
    groups = ceil(rows, unit)
    waves, wave_rows = 4 if grouped else 8, 64 // lanes
    if wpr == 1:
        most = (3 if grouped else 1 if fp32_rows else 2) * CUS
    else:
        most = min(max(2560 // (wpr * nv) // CUS * CUS, CUS), 4 * CUS)
    passes = ceil(unit, wave_rows)
    by_wave = wpr == 1 and grouped and passes <= 8 and groups >= 256 * passes
    at_once = waves * wave_rows if wpr == 1 and not by_wave else 1
    splits = 1 if by_wave else max(1, min(most // groups, ceil(unit, at_once)))
    units = groups * splits
    slots = min(ceil(units, waves) if by_wave else units, most)
    return by_wave, slots, wave_rows if by_wave else at_once, units, ceil(unit, splits)


def depths(rows, cols, gate_rows, fp32_rows=False):
    """Additions that a term of dw_pre / dw_post and of dgate goes through."""
    by_wave, slots, at_once, units, chunk = backward_plan(rows, cols, gate_rows, fp32_rows)
    walkers = slots * (4 if by_wave else 1)
    chain = ceil(units, walkers) * ceil(chunk, at_once) + 1
    waves = 8 + 2                                       # the waves of a workgroup, the rows of a wave
    return chain + waves + ceil(slots, 128) + 7, ceil(chunk, at_once) + waves + 32 + 7


FORWARD = [(20503, 128), (41001, 64), (10307, 256), (10250, 136), (5203, 512), (2600, 1000), (1301, 2048), (2100, 2560),
           (1601, 4104), (600, 9728), (540, 12296), (530, 16384)]


@pytest.mark.parametrize("rows,cols", FORWARD)
@pytest.mark.parametrize("kind,stream,wt,gate_rows", [("both", BF, BF, 0), ("both", F32, F32, 7), ("pre", BF, F32, 0),
                                                      ("post", BF, F32, 1)])
def test_forward_beyond_one_pass(rows, cols, kind, stream, wt, gate_rows):
    assert rows > forward_rows(cols)
    t = make(rows, cols, kind, stream, wt, gate_rows, rows + cols)
    Rg = max(1, gate_rows)
    a = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], rows_per_gate=Rg, scale=0.7, eps=EPS)
    o = ops.block_norm(t["residual"], t["x"], **a)
    h, mh, y, my = R.norm(t["residual"], t["x"], t["w_pre"], t["w_post"], t["gate"], Rg, 0.7, EPS)
    R.close(o.h, h, mh, 64, "h")
    if kind != "post":
        R.close(o.y, y, my, 64, "y")
        R.check_codes(o.q, o.s, y, my, 64, "codes")
    again = ops.block_norm(t["residual"], t["x"], **a)
    assert all(p is None or torch.equal(p, q) for p, q in zip(o, again))


def check_backward(rows, cols, kind, stream, wt, gate_rows, dy_dt, dg_dt):
    t = make(rows, cols, kind, stream, wt, gate_rows, rows * 3 + cols)
    Rg = max(1, gate_rows)
    g = torch.Generator().manual_seed(rows + cols)
    dh = (1e-2 * torch.randn(rows, cols, generator=g)).to(stream).cuda()
    h = dy = None
    if kind != "post":
        h = t["residual"]
        dy = (1e-2 * torch.randn(rows, cols, generator=g)).to(dy_dt).cuda()
    o = ops.block_norm_backward(dy, dh, h, t["x"], w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"],
                                rows_per_gate=Rg, scale=0.7, eps=EPS, dgate_dtype=dg_dt)
    ref = R.norm_grad(dy, dh, h, t["x"], t["w_pre"], t["w_post"], t["gate"], Rg, 0.7, EPS)
    col, gate = depths(rows, cols, gate_rows if t["gate"] is not None else 0,
                       stream == F32 or (dy_dt == F32 and cols <= 256))
    c = {"dres": 128, "dx": 128, "dw_pre": 128 + col, "dw_post": 128 + col, "dgate": 128 + (gate if gate_rows > 1 else 0)}
    for name in ("dres", "dx", "dgate", "dw_post", "dw_pre"):
        got = getattr(o, name)
        assert (got is not None) == (name in ref), name
        if got is not None:
            R.close(got, ref[name][0], ref[name][1], c[name], name)


@pytest.mark.parametrize("rows,cols", [(1400, 2560), (1403, 2048), (1301, 1000), (601, 4104), (600, 9728), (530, 12296),
                                       (520, 16384), (16500, 128), (8300, 256), (4205, 512)])
@pytest.mark.parametrize("kind,stream,wt,gate_rows,dy_dt,dg_dt", [
    ("both", BF, BF, 0, BF, F32), ("both", F32, F32, 0, F32, F32), ("both", BF, F32, 1, F32, BF),
    ("both", F32, BF, 7, BF, F32), ("both", BF, BF, 200, F32, BF), ("pre", BF, F32, 0, BF, F32),
    ("post", F32, F32, 10 ** 9, BF, F32)])
def test_backward_beyond_one_pass(rows, cols, kind, stream, wt, gate_rows, dy_dt, dg_dt):
    by_wave, slots, at_once, units, chunk = backward_plan(rows, cols, gate_rows if gate_rows else 0,
                                                          stream == F32 or (dy_dt == F32 and cols <= 256))
    if gate_rows <= 1:
        assert rows > slots * at_once
    elif layout(cols)[0] > 1:
        assert chunk > 1 or units > slots
    check_backward(rows, cols, kind, stream, wt, gate_rows, dy_dt, dg_dt)


@pytest.mark.parametrize("rows,cols,gate_rows,by_wave", [
    # gate rows of one to eight passes of a wave, as many as go to single
    # waves and one fewer, the last one short
    (256 * 4 - 1, 128, 4, True), (255 * 4 - 1, 128, 4, False), (512 * 5 - 2, 64, 5, True), (511 * 5, 64, 5, False),
    (2048 * 32 - 7, 128, 32, True), (2047 * 32 - 7, 128, 32, False), (512, 256, 2, True), (510, 256, 2, False),
    (1024 * 7 - 3, 256, 7, True), (1023 * 7, 256, 7, False), (512 * 2 - 1, 512, 2, True), (511 * 2, 512, 2, False),
    (2048 * 8 - 5, 264, 8, True), (2047 * 8 - 5, 264, 8, False), (3000 * 33, 64, 33, False), (2600 * 9, 512, 9, False)])
@pytest.mark.parametrize("stream", [BF, F32])
def test_gate_rows_on_both_sides_of_the_rule(rows, cols, gate_rows, by_wave, stream):
    assert backward_plan(rows, cols, gate_rows)[0] == by_wave
    check_backward(rows, cols, "both", stream, BF, gate_rows, F32, F32)
