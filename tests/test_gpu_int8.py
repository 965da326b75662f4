"""Linear layers in 8-bit integers against 64-bit references: codes and scales must
be equal, products within their three fp32 roundings and the output's own."""
import pytest
import torch

import int8_ref as R
from fp8_block_scaled_x128_amd import ops

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def acts(rows, cols, seed, ld=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, max(cols, ld), generator=g)
    x[torch.rand(x.shape, generator=g) < 2e-3] *= 30
    return x.to(BF)[:, :cols]


def dev(t, ld=0):
    """t on the GPU with rows of ld elements (a view when ld is larger)."""
    if ld <= t.shape[1]:
        return t.contiguous().cuda()
    out = torch.full((t.shape[0], ld), 7, dtype=t.dtype, device="cuda")
    out[:, :t.shape[1]] = t.cuda()
    return out[:, :t.shape[1]]


def same_codes(got, x):
    q, s = R.codes(x)
    assert torch.equal(got[1].cpu().double().nan_to_num(nan=-1.0), s.nan_to_num(nan=-1.0)), "scales"
    assert torch.equal(got[0].cpu(), R.pad(q)), "codes"


# ------------------------------------------------------------------ codes
@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 2560), (3, 24), (5, 520), (130, 1000), (1023, 72), (1025, 512),
                                       (1025, 1032), (1024, 2048), (1030, 2560), (1027, 4096), (1026, 4104), (4, 9728),
                                       (3, 10248), (2, 16384), (2, 16392), (3, 40000)])
def test_row_codes(rows, cols):
    x = acts(rows, cols, rows + cols, ld=cols + 8)
    same_codes(ops.i8_quant(dev(x, cols + 8)), x)


@pytest.mark.parametrize("rows,cols", [(1, 8), (7, 72), (16, 64), (127, 136), (128, 64), (129, 1000), (512, 200),
                                       (513, 200), (700, 64), (1000, 72), (4096, 264), (1, 2560), (300, 9728)])
def test_column_codes(rows, cols):
    x = acts(rows, cols, rows + 3 * cols, ld=cols + 8)
    same_codes(ops.i8_quant(dev(x, cols + 8), ops.AXIS_COL), x.t().contiguous())


def test_column_codes_leave_the_rest():
    x = acts(600, 64, 5).cuda()
    for rows in (33, 600):
        q = torch.full((64, 640), 77, dtype=torch.int8, device="cuda")
        s = torch.empty(64, device="cuda")
        ops.i8_quant(x[:rows], ops.AXIS_COL, (q[:, :(rows + 15) // 16 * 16], s))
        assert (q[:, (rows + 15) // 16 * 16:] == 77).all()


def special_rows(cols):
    """Ties, the range's ends, zeros, signed zeros, subnormals, infinities, NaN."""
    x = torch.zeros(13, cols)
    k = torch.arange(cols, dtype=torch.float32)
    x[0] = (k % 255 - 127) / 2                # S = 0.5 once 63.5 is there: ties at every odd half
    x[0, 0] = 63.5
    x[1] = (k % 127) + 0.5
    x[1, 0] = 127.0                          # S = 1: ties k + 1/2
    x[2] = -0.0
    x[3] = torch.finfo(BF).max * (1 - 2 * (k % 2))
    x[4] = 2.0 ** -133 * (k % 128)           # bf16's subnormals
    x[5] = 2.0 ** -120 * (k % 128 + 1)
    x[6] = 1e-30
    x[6, 1] = -1.0
    x[7, 2] = torch.inf
    x[8, 3] = -torch.inf
    x[9, 4] = torch.nan
    x[10] = torch.inf
    x[11] = torch.nan
    x[11, 5] = torch.inf
    x[12, cols - 1] = -3.0
    return x.to(BF)


@pytest.mark.parametrize("cols", [136, 1000])
def test_special_rows_and_columns(cols):
    x = special_rows(cols)
    same_codes(ops.i8_quant(x.cuda()), x)
    xt = torch.zeros(cols, 16, dtype=BF)
    xt[:, :13] = x.t()
    same_codes(ops.i8_quant(xt.cuda(), ops.AXIS_COL), xt.t().contiguous())


def test_every_quotient_near_a_half():
    """All bf16 significands against scales of all bf16 maxima: 128 rows of one
    maximum each, columns over eight binades."""
    m = torch.arange(128, dtype=torch.float32)
    vals = torch.cat([(128 + m) * 2.0 ** -e for e in range(1, 9)])
    x = vals.repeat(128, 1)
    x[:, 0] = 128 + m
    x = x.to(BF)
    same_codes(ops.i8_quant(x.cuda()), x)


# ------------------------------------------------------------------ products
def operands(M, N, K, seed, full=False):
    g = torch.Generator().manual_seed(seed)
    lo, hi = (-128, 128) if full else (-127, 128)
    a = torch.randint(lo, hi, (M, K), generator=g, dtype=torch.int8)
    b = torch.randint(lo, hi, (N, K), generator=g, dtype=torch.int8)
    return a, torch.rand(M, generator=g) + 0.01, b, torch.rand(N, generator=g) * 0.1 + 0.001


SHAPES = [(1, 8, 16), (1, 9728, 2560), (1, 1536, 1008), (2, 24, 32), (15, 136, 64), (16, 128, 128), (17, 72, 80),
          (33, 264, 144), (64, 2560, 9728), (64, 40, 48), (65, 64, 128), (100, 1512, 1008), (128, 128, 256),
          (129, 136, 272), (200, 8, 4096), (333, 1512, 1008), (256, 256, 1152), (700, 520, 112), (1030, 2056, 240),
          (2048, 4096, 1040), (4100, 2568, 400)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", [BF, F32])
def test_product(M, N, K, out):
    a, sa, b, sb = operands(M, N, K, M + N + K)
    c = ops.i8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out)
    R.check_product(c, R.product(a, sa, b, sb))


@pytest.mark.parametrize("M,N,K", [(3, 136, 80), (40, 264, 336), (150, 200, 336), (2000, 2304, 144)])
def test_product_strides(M, N, K):
    a, sa, b, sb = operands(M, N, K, 7 * M)
    store = torch.full((M, N + 24), 5.0, dtype=BF, device="cuda")
    ops.i8_gemm(dev(a, K + 16), sa.cuda(), dev(b, K + 48), sb.cuda(), BF, store[:, :N])
    R.check_product(store[:, :N], R.product(a, sa, b, sb))
    assert (store[:, N:] == 5).all()


@pytest.mark.parametrize("M", [1, 20, 100, 2100])
def test_product_extremes(M):
    """The largest sum 32 bits hold (K 131056 codes of -128), and no sum at all."""
    N, K = (2304, 0) if M > 2000 else (72, 131056)
    a = torch.full((M, K), -128, dtype=torch.int8)
    b = torch.full((N, K), -128, dtype=torch.int8)
    sa, sb = torch.full((M,), 0.5), torch.arange(N) + 1.0
    c = ops.i8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), F32)
    ref = (16384.0 * K) * 0.5 * sb.double()[None, :].expand(M, N)
    R.check_product(c, ref)


@pytest.mark.parametrize("M", [5, 90, 2100])
def test_bad_rows_stay_in_their_rows(M):
    N, K = (2304, 256) if M > 2000 else (64, 256)
    x, w = acts(M, K, 3), acts(N, K, 4)
    x[2, 7], x[4, 9], w[11, 3] = torch.nan, torch.inf, -torch.inf
    qa, sa = ops.i8_quant(x.cuda())
    qb, sb = ops.i8_quant(w.cuda())
    c = ops.i8_gemm(qa, sa, qb, sb).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[2], bad[4], bad[:, 11] = True, True, True
    assert torch.equal(torch.isnan(c), bad) and torch.isfinite(c[~bad]).all()


@pytest.mark.parametrize("rows,cols,out", [(1, 2560, 9728), (1, 8, 8), (2, 1000, 1512), (64, 9728, 2560),
                                           (333, 1000, 1512), (1500, 264, 72), (4, 16392, 64)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_linear(rows, cols, out, dt):
    x, w = acts(rows, cols, 11 + rows, ld=cols + 8), acts(out, cols, 12 + rows)
    qw, sw = ops.i8_quant(w.cuda())
    xd = dev(x, cols + 8)
    r = ops.i8_linear(xd, qw, sw, dt)
    (qx, sx), (qr, sr) = R.codes(x), R.codes(w)
    R.check_product(r.y, R.product(qx, sx, qr, sr))
    qa, sa = ops.i8_quant(xd)                 # the two calls by themselves give the same bits
    assert torch.equal(r.y, ops.i8_gemm(qa, sa, qw, sw, dt))
    again = ops.i8_linear(xd, qw, sw, dt, out=r)
    assert again.y is r.y


@pytest.mark.parametrize("T,I,O", [(1, 8, 8), (16, 64, 128), (205, 1000, 1512), (513, 264, 136), (1024, 512, 2048),
                                   (0, 64, 128)])
def test_linear_backward(T, I, O):
    x, w, dy = acts(T, I, 21), acts(O, I, 22), acts(T, O, 23)
    y, saved = ops.i8_linear_forward(x.cuda(), w.cuda())
    g = ops.i8_linear_backward(dy.cuda(), saved)
    assert y.shape == (T, O) and g.dx.shape == (T, I) and g.dw.shape == (O, I)
    if T == 0:
        assert (g.dw == 0).all()
        return
    (qd, sd), (qw, sw) = R.codes(dy), R.codes(w.t().contiguous())
    R.check_product(g.dx, R.product(qd, sd, qw, sw))
    (qd, sd), (qx, sx) = R.codes(dy.t().contiguous()), R.codes(x.t().contiguous())
    R.check_product(g.dw, R.product(qd, sd, qx, sx))
    r = ops.i8_linear_backward(dy.cuda(), saved, out=g)
    assert r.dx is g.dx and r.dw is g.dw


@pytest.mark.parametrize("T,I,O", [(48, 128, 96), (640, 256, 160)])
def test_linear_backward_against_differences(T, I, O):
    """<dY, Y(x, w)> of the unrounded layer is linear in each operand, so its
    difference quotients are its gradients up to 64-bit rounding; the integer
    gradient is off by its codes: each operand by at most S / 2 a value, so
    |dx - ref| <= sum_o (|dy| S_w / 2 + |w| S_dy / 2 + S_dy S_w / 4)."""
    x, w, dy = acts(T, I, 31), acts(O, I, 32), acts(T, O, 33)
    g = ops.i8_linear_backward(dy.cuda(), ops.i8_linear_forward(x.cuda(), w.cuda())[1])
    X, W, D = x.double(), w.double(), dy.double()
    f = lambda X, W: (D * (X @ W.t())).sum()

    def bound(a, b):                          # rows of a against rows of b
        sa, sb = R.codes(a)[1], R.codes(b)[1]
        n = a.shape[1]
        return (a.double().abs().sum(1)[:, None] * sb / 2 + sa[:, None] * b.double().abs().sum(1) / 2 +
                n * sa[:, None] * sb / 4) * 1.001 + 1e-9

    bx, bw = bound(dy, w.t().contiguous()), bound(dy.t().contiguous(), x.t().contiguous())
    gen = torch.Generator().manual_seed(1)
    for _ in range(40):
        t, i, o = (int(torch.randint(0, n, (), generator=gen)) for n in (T, I, O))
        e = torch.zeros_like(X)
        e[t, i] = 1.0
        assert abs(float((f(X + e, W) - f(X - e, W)) / 2) - float(g.dx[t, i])) <= float(bx[t, i])
        e = torch.zeros_like(W)
        e[o, i] = 1.0
        assert abs(float((f(X, W + e) - f(X, W - e)) / 2) - float(g.dw[o, i])) <= float(bw[o, i])


# ------------------------------------------------------------------ experts
def groups_of(counts, T, seed):
    g = torch.Generator().manual_seed(seed)
    offsets = torch.zeros(len(counts) + 1, dtype=torch.int32)
    offsets[1:] = torch.tensor(counts, dtype=torch.int32).cumsum(0)
    return offsets, torch.randint(0, T, (int(offsets[-1]),), generator=g, dtype=torch.int32)


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 1], [5, 16, 17, 0, 33], [64, 0, 65, 1, 130, 0], [0, 0],
                                    [300, 7, 513, 0, 256], [2] * 130, [700, 900, 0, 1200, 800, 1, 600, 640]])
@pytest.mark.parametrize("N,K", [(128, 256), (1512, 80)])
@pytest.mark.parametrize("gather", [True, False])
def test_grouped_product(counts, N, K, gather):
    offsets, rows = groups_of(counts, 50, len(counts) + N)
    n, G, behind = int(offsets[-1]), len(counts), 5
    T = 50 if gather else n + behind
    a, sa, b, sb = operands(T, G * N, K, 9)
    token = torch.cat([rows, torch.zeros(behind, dtype=torch.int32)])
    c = torch.full((n + behind, N), 3.0, dtype=BF, device="cuda")
    ops.i8_grouped_gemm(a.cuda(), sa.cuda(), b.view(G, N, K).cuda(), sb.view(G, N).cuda(), offsets.cuda(),
                        token.cuda() if gather else None, out=c)
    assert (c[n:] == 3).all(), "rows behind the last group"
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        at = rows[lo:hi].long() if gather else torch.arange(lo, hi)
        R.check_product(c[lo:hi], R.product(a[at], sa[at], b[g * N:(g + 1) * N], sb[g * N:(g + 1) * N]))


@pytest.mark.parametrize("rows,I", [(1, 8), (5, 768), (1025, 136), (130, 2568), (3, 4104), (2, 16392)])
def test_silu_mul_codes(rows, I):
    gu = (acts(rows, 2 * I, 41).float() * 2).to(BF)
    gu[:, ::7] *= 4
    gu[0, 0] = -70.0
    same_codes(ops.i8_silu_mul_quant(gu.cuda()), R.silu_h(gu))
    h = torch.empty(rows, I, dtype=BF, device="cuda")
    q = torch.empty(rows, (I + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    ops.int8_silu_mul_quant(gu.cuda(), rows, I, 2 * I, None, q, q.shape[1], s, h, I)
    assert torch.equal(h.cpu(), R.silu_h(gu))


@pytest.mark.parametrize("rows,live", [(9, 4), (9, 0), (9, 9), (2000, 1333), (9, 100)])
def test_silu_mul_codes_of_live_rows(rows, live):
    gu = acts(rows, 2 * 72, 43).cuda()
    gu[live:] = torch.nan
    q = torch.full((rows, 80), 99, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), 9.0, device="cuda")
    ops.i8_silu_mul_quant(gu, torch.tensor(live, dtype=torch.int32, device="cuda"), (q, s))
    assert (q[live:] == 99).all() and (s[live:] == 9).all()
    n = min(rows, live)
    same_codes((q[:n], s[:n]), R.silu_h(gu[:n].cpu()))


@pytest.mark.parametrize("T,H,I,G,k", [(1, 128, 64, 4, 2), (32, 256, 96, 16, 4), (700, 272, 160, 8, 3)])
def test_moe_forward(T, H, I, G, k):
    """The chain of calls as one, against the chain of references (each rounding of
    the definition in its place).  y is held in bf16 and combined in fp32."""
    x, wgu, wd = acts(T, H, 51), acts(G * 2 * I, H, 52), acts(G * H, I, 53)
    logits = torch.randn(T, G, generator=torch.Generator().manual_seed(5))
    mask = torch.ones(T, dtype=torch.bool)
    mask[T // 2:T // 2 + T // 5] = False
    r = ops.moe_route(logits.cuda(), k, mask=mask.cuda())
    (qgu, sgu), (qd, sd) = ops.i8_quant(wgu.cuda()), ops.i8_quant(wd.cuda())
    out = ops.i8_moe_forward(x.cuda(), qgu.view(G, 2 * I, H), sgu.view(G, 2 * I), qd.view(G, H, I), sd.view(G, H),
                             r.offsets, r.row_token, r.token_rows, r.weights, F32).cpu()
    off, token, pos, w = r.offsets.cpu(), r.row_token.cpu().long(), r.token_rows.cpu(), r.weights.cpu().double()
    (qx, sx), (qgu, sgu), (qd, sd) = R.codes(x), R.codes(wgu), R.codes(wd)
    n = int(off[-1])
    y = torch.zeros(n, H, dtype=torch.float64)
    for g in range(G):
        lo, hi = int(off[g]), int(off[g + 1])
        at = token[lo:hi]
        e = slice(g * 2 * I, (g + 1) * 2 * I)
        f32 = ((qx[at] @ qgu[e].t()).float() * sx[at].float()[:, None]) * sgu[e].float()[None, :]
        qh, sh = R.codes(R.silu_h(f32.to(BF)))
        e = slice(g * H, (g + 1) * H)
        y[lo:hi] = R.product(qh, sh, qd[e], sd[e])
    ref, mag = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0)[:, 0]
        ref[t] += w[t, j, None] * y[pos[t, j].long()]
        mag[t] += w[t, j, None] * y[pos[t, j].long()].abs()
    assert ((out.double() - ref).abs() <= mag * (2.0 ** -8 * 1.01 + (k + 3) * R.U) + 1e-30).all()
    assert (out[~mask] == 0).all()


# ------------------------------------------------------------------ use
def test_streams_and_graph():
    """On another stream, and captured: replays give the eager bits for new inputs
    in the same tensors."""
    x, w, dy = acts(1000, 512, 61).cuda(), acts(640, 512, 62).cuda(), acts(1000, 640, 63).cuda()
    qw, sw = ops.i8_quant(w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, grads = ops.i8_linear(x, qw, sw), ops.i8_linear_backward(dy, (w, x))
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ops.i8_linear(x, qw, sw, out=out)
        ops.i8_linear_backward(dy, (w, x), out=grads)
    for i in range(3):
        x.copy_(acts(1000, 512, 70 + i))
        dy.copy_(acts(1000, 640, 80 + i))
        out.y.zero_(), grads.dx.zero_(), grads.dw.zero_()
        torch.cuda.synchronize()
        g.replay()
        eager, eg = ops.i8_linear(x, qw, sw), ops.i8_linear_backward(dy, (w, x))
        torch.cuda.synchronize()
        assert torch.equal(out.y, eager.y) and torch.equal(grads.dx, eg.dx) and torch.equal(grads.dw, eg.dw)
