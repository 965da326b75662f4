"""Integer products and gradients around the sizes at which another kernel takes over,
with the exact results of the other tests: sums of integers do not depend on the way."""
import pytest
import torch

import int8_ref as R
from fp8_block_scaled_x128_amd import ops
from test_gpu_int8 import BF, F32, acts, dev, groups_of, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K", [16, 112, 896, 912, 1024, 2560, 2576, 5120, 5136, 10256])
@pytest.mark.parametrize("N", [8, 200])
def test_few_rows(N, K):
    """One or two rows, up to 16, 32 and 64, and one more; a second pass of rows."""
    for M in (1, 2, 3, 16, 17, 32, 33, 64, 65, 100):
        a, sa, b, sb = operands(M, N, K, M + N + K, full=True)
        for out in (BF, F32):
            c = ops.i8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), out)
            R.check_product(c, R.product(a, sa, b, sb))


@pytest.mark.parametrize("M,N,K", [(17, 4000, 9728), (64, 2560, 9744), (130, 1000, 5136), (512, 136, 9760), (200, 520, 65552)])
@pytest.mark.parametrize("out", [BF, F32])
def test_ranges_of_k(M, N, K, out):
    """With a workspace K is split; without one it is not, and the bits are the same."""
    need = ops.int8_gemm_ws_size(M, N, K)
    assert need > 0 and need % (M * N * 4) == 0
    a, sa, b, sb = (t.cuda() for t in operands(M, N, K, 3 * M))
    store = torch.full((M + 1, N + 8), 7.0, dtype=out, device="cuda")
    split = ops.i8_gemm(a, sa, b, sb, out, store[:M, :N])
    whole = torch.empty((M, N), dtype=out, device="cuda")
    ops.int8_gemm(M, N, K, a, K, sa, b, K, sb, whole, N, int(out == F32), None, 0)
    assert torch.equal(split, whole) and (store[M] == 7).all() and (store[:, N:] == 7).all()
    R.check_product(whole, R.product(a, sa, b, sb))


@pytest.mark.parametrize("cols", [8, 24, 1016, 1024, 5112, 5128, 16376, 16384, 16392])
@pytest.mark.parametrize("N", [8, 136])
def test_one_row_of_a_linear_layer(cols, N):
    """The row that every workgroup quantizes for itself gives the two calls' bits."""
    w = acts(N, cols, 5)
    qw, sw = ops.i8_quant(w.cuda())
    for k, x in enumerate((acts(1, cols, 6), torch.zeros(1, cols, dtype=BF), acts(1, cols, 8))):
        if k == 2:
            x[0, cols // 2] = torch.inf
        y = ops.i8_linear(x.cuda(), qw, sw, F32).y
        q, s = ops.i8_quant(x.cuda())
        two = ops.i8_gemm(q, s, qw, sw, F32)
        assert torch.equal(y.view(torch.int32) & 0x7fffffff, two.view(torch.int32) & 0x7fffffff) or k == 2
        if k == 2:
            assert torch.isnan(y).all() and torch.isnan(two).all()
        else:
            R.check_product(y, R.product(*R.codes(x), *R.codes(w)))


@pytest.mark.parametrize("counts", [[3, 4, 5, 4, 0, 4], [6, 0, 9, 1, 64, 65], [33, 32, 31, 0, 100, 2], [100, 0, 129, 64],
                                    [129, 300, 0, 255, 1, 257], [0, 0, 0, 40], [1] * 70])
@pytest.mark.parametrize("N,K", [(8, 16), (136, 1152), (520, 5136)])
def test_groups(counts, N, K):
    offsets, rows = groups_of(counts, 90, sum(counts))
    n, G = int(offsets[-1]), len(counts)
    a, sa, b, sb = operands(90, G * N, K, 19)
    c = torch.full((n + 3, N), 3.0, dtype=F32, device="cuda")
    token = torch.cat([rows, torch.zeros(3, dtype=torch.int32)])
    ops.i8_grouped_gemm(a.cuda(), sa.cuda(), b.view(G, N, K).cuda(), sb.view(G, N).cuda(), offsets.cuda(), token.cuda(),
                        F32, out=c)
    assert (c[n:] == 3).all()
    for g in range(G):
        lo, hi = int(offsets[g]), int(offsets[g + 1])
        at = rows[lo:hi].long()
        R.check_product(c[lo:hi], R.product(a[at], sa[at], b[g * N:(g + 1) * N], sb[g * N:(g + 1) * N]))


@pytest.mark.parametrize("M,K", [(70000, 16), (70000, 912)])
def test_outputs_past_four_gigabytes(M, K):
    """Rows of a view whose storage passes 2^32 bytes."""
    N, ld = 8, 16384
    a, sa, b, sb = operands(M, N, K, 23)
    store = torch.empty((M, ld), dtype=F32, device="cuda")
    ops.i8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), F32, store[:, :N])
    R.check_product(store[:, :N], R.product(a, sa, b, sb))


@pytest.mark.parametrize("T,I,O", [(1, 16, 8), (17, 24, 1000), (255, 72, 264), (257, 520, 72), (8300, 16, 24), (24, 16, 8304),
                                   (100, 1000, 6600), (2100, 2056, 5000), (5000, 2056, 2096)])
def test_gradient(T, I, O):
    """Runs of rows for the maxima, K ranges, and both products in one launch in
    either order; rows of strided inputs."""
    x, w, dy = acts(T, I, 41), acts(O, I, 42), acts(T, O, 43)
    x[:, I // 2] = 0
    g = ops.i8_linear_backward(dev(dy, O + 8), (dev(w, I + 16), dev(x, I + 8)))
    R.check_product(g.dx, R.product(*R.codes(dy), *R.codes(w.t().contiguous())))
    R.check_product(g.dw, R.product(*R.codes(dy.t().contiguous()), *R.codes(x.t().contiguous())))
    assert (g.dw[:, I // 2] == 0).all()


def test_gradient_of_nothing():
    x, w, dy = (torch.empty(s, dtype=BF, device="cuda") for s in ((5, 16), (0, 16), (5, 0)))
    g = ops.i8_linear_backward(dy, (w, x))
    assert g.dw.shape == (0, 16) and (g.dx == 0).all()


def test_gradient_keeps_bad_values_in_their_lines():
    """A NaN of dY reaches its token's dX and its output's dW and nothing else; one of X
    its input's dW."""
    T, I, O = 600, 64, 48
    x, w, dy = acts(T, I, 51), acts(O, I, 52), acts(T, O, 53)
    dy[500, 7], x[3, 9], w[40, 11] = torch.nan, torch.inf, -torch.inf
    g = ops.i8_linear_backward(dy.cuda(), (w.cuda(), x.cuda()))
    dx, dw = torch.zeros(T, I, dtype=torch.bool), torch.zeros(O, I, dtype=torch.bool)
    dx[500], dx[:, 11], dw[7], dw[:, 9] = True, True, True, True
    assert torch.equal(torch.isnan(g.dx.cpu()), dx) and torch.equal(torch.isnan(g.dw.cpu()), dw)


def test_two_streams_and_replays():
    """Two calls at once with workspaces of their own, and two captured calls that share
    one, replayed with eager calls between."""
    w = acts(2560, 9728, 3).cuda()
    qw, sw = ops.i8_quant(w)
    xs = [acts(64, 9728, 4 + i).cuda() for i in range(2)]
    want = [ops.i8_linear(x, qw, sw).y.clone() for x in xs]
    outs = [ops.i8_linear(x, qw, sw) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, o, s in zip(xs, outs, streams):
            with torch.cuda.stream(s):
                ops.i8_linear(x, qw, sw, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o.y, v) for o, v in zip(outs, want))
    shared = [ops.I8Linear(torch.zeros_like(v), outs[0].ws) for v in want]
    graphs = []
    for x, o in zip(xs, shared):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.i8_linear(x, qw, sw, out=o)
        graphs.append(g)
    for _ in range(3):
        for o in shared:
            o.y.zero_()
        for g in graphs:
            g.replay()
        eager = ops.i8_linear(xs[0], qw, sw, out=outs[0])       # the same workspace, behind both
        torch.cuda.synchronize()
        assert all(torch.equal(o.y, v) for o, v in zip(shared, want)) and torch.equal(eager.y, want[0])
