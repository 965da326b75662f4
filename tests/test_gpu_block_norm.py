"""The norms around a block with its gate, residual scale and 1x128
quantization (fp8_block_norm) and their gradient (fp8_block_norm_backward)
against 64-bit references.

Bounds: a row's sum of squares is a chain of at most 32 terms per lane, 6 lane
steps and 16 waves, so its relative error is below 54 U and that of its rsqrt
below 30 U; with the products around it fewer than 64 roundings enter any
value, on the magnitude of its terms.  In the backward pass two such sums
meet: 128.  A column sum adds one rounding per row of a slot, per 64th slot
and per tree step: `rows + 64` covers every split of the rows."""
import pytest
import torch

import block_ref as R
from fp8_block_scaled_x128_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def make(rows, cols, kind, stream, wt, gate_rows, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)

    def mat(r, dt, sigma=1.0):
        v = (sigma * n(r, cols + pad)).to(dt)
        return v.cuda()[:, :cols]
    t = dict(residual=mat(rows, stream, 3.0), x=None, w_pre=None, w_post=None, gate=None)
    if kind != "pre":
        t["x"] = mat(rows, BF)
        if kind != "plain":
            t["w_post"] = (1 + 0.2 * n(cols)).to(wt).cuda()
        if gate_rows:
            t["gate"] = mat(-(-rows // gate_rows), BF, 0.5)
    if kind != "post":
        t["w_pre"] = (1 + 0.2 * n(cols)).to(wt).cuda()
    return t


SHAPES = [(1, 8), (1, 2560), (3, 128), (5, 1000), (67, 136), (130, 2048), (33, 4104), (9, 9728), (4, 12296),
          (2, 16384), (1, 512), (700, 64), (1001, 128), (333, 256), (50, 200), (77, 24)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind,stream,wt,gate_rows", [
    ("both", BF, BF, 0), ("both", F32, F32, 1), ("both", F32, BF, 7), ("pre", BF, F32, 0), ("pre", F32, F32, 0),
    ("post", BF, BF, 10 ** 9), ("post", F32, F32, 0), ("plain", BF, BF, 2), ("plain", F32, F32, 0)])
def test_forward(rows, cols, kind, stream, wt, gate_rows):
    t = make(rows, cols, kind, stream, wt, gate_rows, rows * 7 + cols, pad=8 * (rows % 3))
    Rg = max(1, gate_rows)
    o = ops.block_norm(t["residual"], t["x"], w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"],
                       rows_per_gate=Rg, scale=0.7, eps=EPS)
    h, mh, y, my = R.norm(t["residual"], t["x"], t["w_pre"], t["w_post"], t["gate"], Rg, 0.7, EPS)
    R.close(o.h, h, mh, 64, "h")
    if kind != "post":
        R.close(o.y, y, my, 64, "y")
        R.check_codes(o.q, o.s, y, my, 64, "codes")
    else:
        assert o.y is None and o.q is None and o.s is None


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 2560), (5, 1000), (67, 136), (130, 2048), (33, 4104), (6, 9728),
                                       (3, 12296), (2, 16384), (2500, 64), (3000, 520), (1001, 128), (9000, 128), (333, 256), (50, 200),
                                       (77, 24)])
@pytest.mark.parametrize("kind,stream,wt,gate_rows,dy_dt,dg_dt", [
    ("both", BF, BF, 0, F32, F32), ("both", F32, F32, 1, BF, BF), ("both", F32, BF, 7, BF, F32),
    ("both", BF, F32, 10 ** 9, F32, F32), ("pre", BF, F32, 0, BF, F32), ("pre", F32, F32, 0, F32, F32),
    ("post", BF, BF, 2, BF, BF), ("post", F32, F32, 0, BF, F32), ("plain", BF, BF, 33, BF, F32),
    ("plain", F32, F32, 0, F32, F32)])
def test_backward(rows, cols, kind, stream, wt, gate_rows, dy_dt, dg_dt):
    t = make(rows, cols, kind, stream, wt, gate_rows, rows * 11 + cols, pad=8 * (rows % 2))
    Rg = max(1, gate_rows)
    g = torch.Generator().manual_seed(rows + cols)
    dh = (1e-2 * torch.randn(rows, cols, generator=g)).to(stream).cuda()
    h = dy = None
    if kind != "post":
        h = t["residual"]
        dy = (1e-2 * torch.randn(rows, cols, generator=g)).to(dy_dt).cuda()
    a = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], rows_per_gate=Rg, scale=0.7, eps=EPS)
    o = ops.block_norm_backward(dy, dh, h, t["x"], dgate_dtype=dg_dt, **a)
    ref = R.norm_grad(dy, dh, h, t["x"], t["w_pre"], t["w_post"], t["gate"], Rg, 0.7, EPS)
    for name in ("dres", "dx", "dgate", "dw_post", "dw_pre"):
        got = getattr(o, name)
        assert (got is not None) == (name in ref), name
        if got is not None:
            c = 128 if name in ("dres", "dx") else 192 + rows
            R.close(got, ref[name][0], ref[name][1], c, name)
    # the same bits again, into the same tensors
    keep = [v.clone() for v in o[:5] if v is not None]
    o2 = ops.block_norm_backward(dy, dh, h, t["x"], dgate_dtype=dg_dt, out=o, **a)
    assert all(torch.equal(p, q) for p, q in zip(keep, [v for v in o2[:5] if v is not None]))


def test_against_differences():
    """The kernels' gradient along a direction against central differences of
    the 64-bit forward: with step 1e-4 on O(1) inputs the differences are good
    to 1e-7 of the terms; the kernel's fp32 stream to 128 U and its bf16 dx and
    dgate (per token) to half a bf16 step, each on the terms' magnitude."""
    rows, cols = 6, 264
    t = make(rows, cols, "both", F32, F32, 1, 5)
    g = torch.Generator().manual_seed(9)
    dy = torch.randn(rows, cols, generator=g).cuda()
    dhe = torch.randn(rows, cols, generator=g).cuda()
    h = ops.block_norm(t["residual"], t["x"], w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], scale=0.7).h
    o = ops.block_norm_backward(dy, dhe, h, t["x"], w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], scale=0.7)
    names = {"residual": o.dres, "x": o.dx, "gate": o.dgate, "w_pre": o.dw_pre, "w_post": o.dw_post}
    base = {k: R.d(v) for k, v in t.items()}

    def loss(v):
        hh, _, y, _ = R.norm(v["residual"], v["x"], v["w_pre"], v["w_post"], v["gate"], 1, 0.7, EPS)
        return float((y * R.d(dy)).sum() + (hh * R.d(dhe)).sum())
    for name, grad in names.items():
        v = torch.randn(base[name].shape, generator=g, dtype=torch.float64)
        up, dn = dict(base), dict(base)
        up[name], dn[name] = base[name] + 1e-4 * v, base[name] - 1e-4 * v
        diff = (loss(up) - loss(dn)) / 2e-4
        terms = float((R.d(grad) * v).abs().sum())
        tol = (R.HALF[grad.dtype] + 256 * R.U + 1e-6) * terms
        assert abs(float((R.d(grad) * v).sum()) - diff) <= tol, name


def test_rows_of_zeros_and_large_values():
    rows, cols = 5, 384
    x = torch.zeros(rows, cols, dtype=BF, device="cuda")
    x[1] = 1e15
    x[2, 7] = 3.0
    w = torch.ones(cols, dtype=BF, device="cuda")
    o = ops.block_norm(None, x, w_pre=w, w_post=w)
    h, mh, y, my = R.norm(None, x, w, w, None, 1, 1.0, EPS)
    R.close(o.h, h, mh, 64, "h")
    R.close(o.y, y, my, 64, "y")
    R.check_codes(o.q, o.s, y, my, 64, "codes")
    assert (o.q[0] == 0).all() and (o.s[0] == 0).all()


def test_infinities_and_nan_stay_in_their_rows():
    """An infinity makes its row's factor 0 (so 0 beside it, NaN at it), as in
    the formula; other rows are as without it."""
    rows, cols = 6, 520
    t = make(rows, cols, "both", BF, BF, 0, 8)
    clean = ops.block_norm(t["residual"], t["x"], w_pre=t["w_pre"], w_post=t["w_post"])
    x = t["x"].clone()
    x[1, 5] = torch.inf
    x[3, 7] = torch.nan
    o = ops.block_norm(t["residual"], x, w_pre=t["w_pre"], w_post=t["w_post"])
    ok = [0, 2, 4, 5]
    for a, b in zip(o, clean):
        assert torch.equal(a[ok], b[ok])
    assert torch.isnan(o.h[1, 5]) and torch.isnan(o.h[3]).all()
    rest = [c for c in range(cols) if c != 5]
    assert torch.equal(o.h[1, rest], t["residual"][1, rest])


def test_in_place_strides_and_untouched_columns():
    """h over residual in place, outputs as views of wider tensors: columns
    past the view keep their bytes."""
    rows, cols, wide = 37, 520, 536
    t = make(rows, cols, "both", BF, BF, 0, 3)
    a = dict(w_pre=t["w_pre"], w_post=t["w_post"], scale=0.5)
    ref = ops.block_norm(t["residual"], t["x"], **a)
    buf = {k: torch.full((rows, wide), 9, dtype=dt, device="cuda") for k, dt in (("h", BF), ("y", BF), ("q", torch.uint8))}
    buf["h"][:, :cols] = t["residual"]
    s = torch.full((rows, 7), 9.0, device="cuda")
    ng = (cols + 127) // 128
    out = ops.BlockNorm(buf["h"][:, :cols], buf["y"][:, :cols], buf["q"][:, :cols], s[:, :ng])
    o = ops.block_norm(buf["h"][:, :cols], t["x"], out=out, **a)
    for k in ("h", "y", "q", "s"):
        assert torch.equal(getattr(o, k), getattr(ref, k)), k
    assert all((b[:, cols:] == 9).all() for b in buf.values()) and (s[:, ng:] == 9).all()
    # the gradient arriving at h, replaced by the residual's in place
    dh = torch.randn(rows, cols, device="cuda").to(BF)
    dy = torch.randn(rows, cols, device="cuda").to(BF)
    b = dict(w_pre=t["w_pre"], w_post=t["w_post"], scale=0.5)
    g = ops.block_norm_backward(dy, dh, ref.h, t["x"], **b)
    held = dh.clone()
    g2 = ops.block_norm_backward(dy, held, ref.h, t["x"], out=g._replace(dres=held), **b)
    want = ops.block_norm_backward(dy, dh, ref.h, t["x"], **b)
    assert torch.equal(g2.dres, want.dres) and torch.equal(g2.dx, want.dx)


def test_no_rows():
    e = lambda dt: torch.empty((0, 256), dtype=dt, device="cuda")
    w = torch.ones(256, dtype=BF, device="cuda")
    o = ops.block_norm(e(BF), e(BF), w_pre=w, w_post=w)
    assert o.h.shape == (0, 256) and o.s.shape == (0, 2)
    g = ops.block_norm_backward(e(BF), e(BF), e(BF), e(BF), w_pre=w, w_post=w, gate=e(BF))
    assert (g.dw_pre == 0).all() and (g.dw_post == 0).all() and g.dgate.shape == (0, 256)


def test_graph_replays():
    """Forward and backward captured once; replayed with new inputs in the same
    tensors, eager calls between, each replay against the eager result."""
    rows, cols = 300, 2560
    t = make(rows, cols, "both", BF, BF, 0, 1)
    dy, dh = torch.zeros(rows, cols, device="cuda"), torch.zeros(rows, cols, dtype=BF, device="cuda")
    a = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=None, scale=0.9)

    def both(o=None, g=None):
        o = ops.block_norm(t["residual"], t["x"], out=o, **a)
        return o, ops.block_norm_backward(dy, dh, o.h, t["x"], out=g, **a)
    o, g = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(o, g)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(o, g)
    for rep in range(4):
        t["x"].copy_(torch.randn(rows, cols, device="cuda"))
        t["residual"].copy_(torch.randn(rows, cols, device="cuda"))
        dy.normal_()
        dh.normal_()
        for v in (*o, *g[:5]):
            if v is not None:
                v.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        eo, eg = both()
        torch.cuda.synchronize()
        for p, q in zip((*o, *g[:5]), (*eo, *eg[:5])):
            assert p is None and q is None or torch.equal(p, q), rep


def test_two_streams_at_once():
    """Two callers on two streams, each with its own tensors and workspace."""
    rows, cols = 2000, 1024
    ts = [make(rows, cols, "both", BF, BF, 0, s) for s in (1, 2)]
    gs = [torch.randn(rows, cols, device="cuda").to(BF) for _ in range(2)]

    def call(i):
        t = ts[i]
        o = ops.block_norm(t["residual"], t["x"], w_pre=t["w_pre"], w_post=t["w_post"])
        return o, ops.block_norm_backward(gs[i], gs[i], o.h, t["x"], w_pre=t["w_pre"], w_post=t["w_post"])
    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for rep in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, call(i)))
    torch.cuda.synchronize()
    for i, (o, g) in got:
        for p, q in zip((*o, *g[:5]), (*want[i][0], *want[i][1][:5])):
            assert p is None and q is None or torch.equal(p, q)


def test_linear_on_the_fused_codes():
    """The codes feed the block-scaled GEMM as quant_rowblock's do: the GEMM on
    them equals the 64-bit product of their decoded values to the GEMM's own
    bound (products are truncated inside runs of 8 K: 1e-4 of the terms)."""
    rows, cols, outf = 96, 512, 256
    t = make(rows, cols, "both", BF, BF, 0, 4)
    o = ops.block_norm(t["residual"], t["x"], w_pre=t["w_pre"], w_post=t["w_post"], y=False)
    w = (0.02 * torch.randn(outf, cols, generator=torch.Generator().manual_seed(3))).to(BF).cuda()
    qw, sw, _ = ops.quant_block2d(w)
    c = ops.gemm(o.q, o.s, qw, sw, out_dtype=F32)
    a = R.d(o.q.view(torch.float8_e4m3fn).float()) * R.d(o.s).repeat_interleave(128, 1)
    b = R.d(qw.view(torch.float8_e4m3fn).float()) * R.d(sw).repeat_interleave(128, 0).repeat_interleave(128, 1)
    err = (R.d(c) - a @ b.T).abs()
    assert (err <= 1e-4 * (a.abs() @ b.abs().T) + 1e-30).all()


def test_refusals():
    t = make(4, 256, "both", BF, BF, 0, 1)
    w = t["w_pre"]
    with pytest.raises(ValueError):
        ops.block_norm(t["residual"].cpu(), None, w_pre=w)
    with pytest.raises(ValueError):
        ops.block_norm(t["residual"], t["x"][:, :128], w_pre=w)
    with pytest.raises(ValueError):
        ops.block_norm(t["residual"], None, w_pre=w[:128])
    with pytest.raises(ValueError):
        ops.block_norm(t["residual"], t["x"].float(), w_pre=w)
    with pytest.raises(ValueError):
        ops.block_norm(None, None, w_pre=w)
    with pytest.raises(ValueError):
        ops.block_norm(t["residual"], t["x"], gate=t["x"], rows_per_gate=2)
    with pytest.raises(ValueError):
        ops.block_norm(t["residual"].t(), None, w_pre=w)
    with pytest.raises(ops.Fp8bsError):
        ops.block_norm(t["residual"], None, w_post=w, w_pre=w)
    with pytest.raises(ops.Fp8bsError):
        ops.block_norm(t["residual"], t["x"], w_pre=w, eps=0.0)
    with pytest.raises(ValueError):
        ops.block_norm_backward(t["x"], None, None, t["x"], w_pre=w)
    with pytest.raises(ValueError):
        ops.block_norm_backward(None, t["x"], None, None, w_post=w)


@pytest.mark.parametrize("rows,cols", [(70, 128), (9, 1000), (5, 10240)])
@pytest.mark.parametrize("gate_rows", [0, 1, 3])
def test_without_residual_and_single_outputs(rows, cols, gate_rows):
    """x alone (h = scale gate N(x)); each forward output alone has the bytes
    it has beside the others."""
    t = make(rows, cols, "both", BF, BF, gate_rows, rows + cols)
    a = dict(w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"], rows_per_gate=max(1, gate_rows), scale=0.7)
    o = ops.block_norm(None, t["x"], **a)
    h, mh, y, my = R.norm(None, t["x"], t["w_pre"], t["w_post"], t["gate"], max(1, gate_rows), 0.7, EPS)
    R.close(o.h, h, mh, 64, "h")
    R.close(o.y, y, my, 64, "y")
    R.check_codes(o.q, o.s, y, my, 64, "codes")
    for keep in ("h", "y", "quant"):
        only = dict(a, h=keep == "h", y=keep == "y", quant=keep == "quant")
        if keep == "h":
            only["w_pre"] = None
        b = ops.block_norm(None, t["x"], **only)
        for n, v in zip(b._fields, b):
            assert (v is not None) == (n in {"h": "h", "y": "y", "quant": "qs"}[keep])
            assert v is None or torch.equal(v, getattr(o, n)), n


@pytest.mark.parametrize("rows,cols", [(70, 128), (300, 64), (9, 1000), (5, 10240), (600, 2560)])
@pytest.mark.parametrize("gate_rows", [0, 1, 3, 200])
def test_gradients_one_at_a_time(rows, cols, gate_rows):
    """Each gradient asked for alone, and without a gradient past y: bounds as
    in test_backward."""
    t = make(rows, cols, "both", BF, BF, gate_rows, rows + cols)
    g = torch.Generator().manual_seed(7)
    dy = (1e-2 * torch.randn(rows, cols, generator=g)).cuda()
    Rg, ngate = max(1, gate_rows), -(-rows // max(1, gate_rows))
    ref = R.norm_grad(dy, None, t["residual"], t["x"], t["w_pre"], t["w_post"], t["gate"], Rg, 0.7, EPS)
    full = ops.block_norm_backward(dy, None, t["residual"], t["x"], w_pre=t["w_pre"], w_post=t["w_post"],
                                   gate=t["gate"], rows_per_gate=Rg, scale=0.7, eps=EPS)
    for name, (v, mag) in ref.items():
        R.close(getattr(full, name), v, mag, 128 if name in ("dres", "dx") else 192 + rows, name)
        o = torch.full_like(getattr(full, name), 9)
        need = ops.fp8_block_norm_backward_ws_size(rows, cols, Rg, name == "dw_post", name == "dw_pre", name == "dgate")
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        pick = lambda n: o if n == name else None
        ops.fp8_block_norm_backward(rows, cols, dy, cols, ops.OUT_FP32, None, 0, t["residual"], cols, ops.OUT_BF16,
                                    t["x"], cols, t["gate"], cols, Rg, 0.7, t["w_post"], t["w_pre"], ops.OUT_BF16, EPS,
                                    pick("dx"), cols, pick("dres"), cols, pick("dgate"), cols, ops.OUT_FP32,
                                    pick("dw_post"), pick("dw_pre"), ws, need)
        R.close(o, v, mag, 128 if name in ("dres", "dx") else 192 + rows, name + " alone")


def test_rows_past_32_bit_offsets():
    """Three rows 2^30 + 8 elements apart in every tensor: the last one starts
    past 2^31 elements (and 2^32 bytes) from the first."""
    rows, cols, ld = 3, 1000, 2 ** 30 + 8
    t = make(rows, cols, "both", BF, BF, 1, 12)
    g = torch.Generator().manual_seed(3)
    dy, dh = [(1e-2 * torch.randn(rows, cols, generator=g)).to(BF).cuda() for _ in range(2)]
    big = torch.empty(2 * ld + 8 * 1024, dtype=BF, device="cuda")
    codes = torch.empty(2 * ld + 1024, dtype=torch.uint8, device="cuda")
    at = lambda i: big[i * 1024:i * 1024 + 2 * ld + 1024].as_strided((rows, cols), (ld, 1))
    a = dict(w_pre=t["w_pre"], w_post=t["w_post"], scale=0.7)
    near = ops.block_norm(t["residual"], t["x"], gate=t["gate"], **a)
    res, x, gate = at(0), at(1), at(2)
    for far, v in ((res, "residual"), (x, "x"), (gate, "gate")):
        far.copy_(t[v])
    o = ops.block_norm(res, x, gate=gate, out=ops.BlockNorm(at(3), at(4), codes.as_strided((rows, cols), (ld, 1)), near.s.clone()), **a)
    assert all(torch.equal(p, q) for p, q in zip(o, near))
    ng = ops.block_norm_backward(dy, dh, near.h, t["x"], gate=t["gate"], dgate_dtype=BF, **a)
    fdy, fdh = at(0), at(5)
    fdy.copy_(dy)
    fdh.copy_(dh)
    out = ng._replace(dres=at(6), dx=at(7), dgate=at(4), dw_post=ng.dw_post.clone(), dw_pre=ng.dw_pre.clone(), ws=ng.ws.clone())
    fg = ops.block_norm_backward(fdy, fdh, o.h, x, gate=gate, dgate_dtype=BF, out=out, **a)
    assert all(torch.equal(p, q) for p, q in zip(fg[:5], ng[:5]))


@pytest.mark.parametrize("rows,cols,gate_rows", [(1500, 64, 5), (2403, 128, 33), (3001, 128, 48), (6401, 256, 24),
                                                 (4002, 512, 2), (2600, 512, 4), (5000, 264, 2),
                                                 (2600, 64, 5), (20001, 128, 16), (9000, 256, 6)])
def test_many_gate_rows(rows, cols, gate_rows):
    """Gate rows that go to single waves, whole, and the last one short."""
    t = make(rows, cols, "both", F32, BF, gate_rows, rows + cols)
    g = torch.Generator().manual_seed(5)
    dy, dh = [(1e-2 * torch.randn(rows, cols, generator=g)).cuda() for _ in range(2)]
    o = ops.block_norm_backward(dy, dh, t["residual"], t["x"], w_pre=t["w_pre"], w_post=t["w_post"], gate=t["gate"],
                                rows_per_gate=gate_rows, scale=0.7, eps=EPS)
    ref = R.norm_grad(dy, dh, t["residual"], t["x"], t["w_pre"], t["w_post"], t["gate"], gate_rows, 0.7, EPS)
    for name, (v, mag) in ref.items():
        c = 128 if name in ("dres", "dx") else 192 + (gate_rows if name == "dgate" else rows)
        R.close(getattr(o, name), v, mag, c, name)
