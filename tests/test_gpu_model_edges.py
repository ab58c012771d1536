"""Model operators on the GPU where they can go wrong: graphs, streams, far strides, empty sums, NaN, many tokens;
gradients against differences, and all of them together as a step uses them."""
import math

import pytest

torch = pytest.importorskip("torch")

import model_util as mu  # noqa: E402
import stack_util as su  # noqa: E402
from test_gpu_model import BF16, DEV, E4M3, F16, F32, M, dgrad, encode, gen, linear, operand, wgrad, workspace  # noqa: E402,F401

pytestmark = pytest.mark.gpu


class Layer:
    """One linear layer's tensors, an embedding before it, and every call on them."""

    def __init__(self, M, n, rows, cols, outs, seed):
        g = gen(seed)
        self.M = M
        self.ids = torch.randint(-2, rows, (n,), generator=g).to(DEV)
        self.table, self.table_s = (t.to(DEV) for t in encode(torch.randn(rows, cols, generator=g)))
        self.e = torch.empty(n, cols, dtype=BF16, device=DEV)
        self.q = torch.empty(n, cols, dtype=E4M3, device=DEV)
        self.qs = torch.empty(n, -(-cols // 32), dtype=torch.uint8, device=DEV)
        self.w, self.ws = (t.to(DEV) for t in encode(0.05 * torch.randn(outs, cols, generator=g)))
        self.y = torch.empty(n, outs, dtype=BF16, device=DEV)
        self.dx = torch.empty(n, cols, dtype=F32, device=DEV)
        self.gw = torch.zeros(outs, cols, device=DEV)
        self.gt = torch.zeros(rows, cols, device=DEV)

    def bytes(self):
        m = self.M
        return max(m.hpo_mx8_linear_workspace(self.q, self.w), m.hpo_mx8_dgrad_workspace(self.y, self.w),
                   m.hpo_mx8_wgrad_workspace(self.y, self.q), m.hpo_embedding_grad_workspace(self.ids, self.gt))

    def run(self, ws):
        """The forward pass with dY = Y, and the gradients."""
        m = self.M
        m.hpo_embedding(self.ids, self.table, self.e, scales=self.table_s, scale=1.5)
        m.hpo_mx8_save(self.e, self.q, self.qs)
        m.hpo_mx8_linear(self.q, self.qs, self.w, self.ws, self.y, ws)
        m.hpo_mx8_dgrad(self.y, self.w, self.ws, self.dx, ws)
        m.hpo_mx8_wgrad(self.y, self.q, self.qs, self.gw, ws, scale=0.5)
        m.hpo_embedding_grad(self.ids, self.dx, self.gt, ws, scale=1.5)

    def bits(self):
        return [su.bits(t).clone() for t in (self.e, self.q, self.qs, self.y, self.dx, self.gw, self.gt)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_graphs_that_share_a_workspace(M):
    """Two captured steps with one workspace, replayed in turn, with eager work and other tokens in between: each
    replay gives what eager calls give."""
    shapes = [(2000, 200, 512, 320, 1), (3000, 77, 256, 256, 2)]
    layers, refs = [Layer(M, *s) for s in shapes], [Layer(M, *s) for s in shapes]
    assert all(M.hpo_mx8_wgrad_workspace(x.y, x.q) > 0 for x in layers), "a sum in parts belongs here"
    ws, other = workspace(max(x.bytes() for x in layers)), workspace(max(x.bytes() for x in layers))
    for x, r in zip(layers, refs):   # modules loaded before a capture
        x.run(ws), r.run(other)
    torch.cuda.synchronize()
    graphs = []
    for x in layers:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x.run(ws)
        graphs.append(graph)
    for k in range(5):
        for x, r, graph in zip(layers, refs, graphs):
            ids = torch.randint(-1, x.table.shape[0], x.ids.shape, generator=gen(k)).to(DEV)
            x.ids.copy_(ids), r.ids.copy_(ids)
            graph.replay()
            junk = torch.randn(512, 512, device=DEV) @ torch.randn(512, 512, device=DEV)
            r.run(other)
            if k % 2:
                torch.cuda.synchronize()
            assert same(x.bits(), r.bits()), k
            del junk


def test_calls_at_once_on_two_streams(M):
    shapes = [(700, 300, 1024, 512, 5), (9, 40, 96, 1000, 6)]
    layers, refs = [Layer(M, *s) for s in shapes], [Layer(M, *s) for s in shapes]
    spaces = [workspace(x.bytes(), 0x3C) for x in layers]
    for r, w in zip(refs, spaces):
        for _ in range(6):
            r.run(w)
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        for x, s, w in zip(layers, streams, spaces):
            with torch.cuda.stream(s):
                x.run(w)
    torch.cuda.synchronize()
    for x, r in zip(layers, refs):
        assert same(x.bits(), r.bits())


def test_explicit_stream(M):
    """stream= names the stream; the current one may be another."""
    x = Layer(M, 64, 30, 128, 96, 9)
    ws = workspace(x.bytes())
    x.run(ws)
    y = torch.empty_like(x.y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    M.hpo_mx8_linear(x.q, x.qs, x.w, x.ws, y, ws, stream=s)
    s.synchronize()
    assert torch.equal(su.bits(y), su.bits(x.y))


# --------------------------------------------------------------------------
# offsets behind 2^31 and 2^32
# --------------------------------------------------------------------------
def far(value, rs, bs=0):
    """`value` in a buffer whose rows lie rs elements apart and whose matrices bs elements."""
    b, r, c = value.shape
    n = (b - 1) * bs + (r - 1) * rs + c
    buf = torch.empty(n * value.element_size(), dtype=torch.uint8, device=DEV)
    view = buf.view(value.dtype).as_strided((b, r, c), (bs, rs, 1))
    view.copy_(value.to(DEV))
    return view


def test_far_rows_of_a_table(M):
    g = gen(4)
    ids = torch.tensor([2, 0, 1, 5, 2]).to(DEV)
    w = torch.randn(1, 3, 72, generator=g).to(BF16)
    W = far(w, 2 ** 31 + 8)[0]
    out = torch.empty(5, 72, device=DEV)
    M.hpo_embedding(ids, W, out)
    assert torch.equal(out.cpu(), mu.embedding(ids.cpu(), w[0].float(), 1.0, 0))
    del W
    q, byte = encode(w.float())
    W = far(q, 2 ** 32 + 16)[0]
    M.hpo_embedding(ids, W, out, scales=byte.to(DEV))
    assert torch.equal(out.cpu(), mu.embedding(ids.cpu(), mu.mx_values(q, byte)[0].float(), 1.0, 0))
    del W
    dy = torch.randn(1, 5, 72, generator=g)
    D, G = far(dy, 2 ** 30 + 4)[0], far(torch.ones(1, 3, 72), 2 ** 31 + 4)[0]
    M.hpo_embedding_grad(ids, D, G, workspace(M.hpo_embedding_grad_workspace(ids, G)))
    want, tol, _ = mu.embedding_grad(ids.cpu(), dy[0], torch.ones(3, 72), 1.0, 0)
    mu.check(G, want, tol, "far")


@pytest.mark.parametrize("cols", [96, 100])
def test_far_rows_of_products(M, cols):
    g = gen(cols)
    t, r, rs, bs = 3, 2, 2 ** 31 + 64, 2 ** 32 + 2 ** 31 + 128
    x, xs = encode(torch.randn(2, t, cols, generator=g))
    w, ws = encode(torch.randn(2, r, cols, generator=g))
    dy = torch.randn(2, t, r, generator=g).to(BF16)
    X = far(x, rs, bs)
    Y = torch.empty(2, t, r, dtype=F16, device=DEV)
    M.hpo_mx8_linear(X, xs.to(DEV), w.to(DEV), ws.to(DEV), Y, workspace(M.hpo_mx8_linear_workspace(X, w)))
    a, b = mu.mx_values(x, xs), mu.mx_values(w, ws)
    want, size = mu.matmul64(a, b.mT)
    cut = mu.aligned_cut(a, b)
    mu.check(Y, want, mu.product_tolerance(size + cut, cols, want, F16) + cut, "far x")
    G = torch.zeros(2, r, cols, device=DEV)
    M.hpo_mx8_wgrad(dy.to(DEV), X, xs.to(DEV), G, workspace(M.hpo_mx8_wgrad_workspace(dy, X)))
    want, size = mu.matmul64(dy.mT, a)
    mu.check(G, want, mu.product_tolerance(size, t, want, F32), "far x, wgrad")
    del X
    D = far(dy, 2 ** 30 + 32, 2 ** 32)
    dx = torch.empty(2, t, cols, device=DEV)
    M.hpo_mx8_dgrad(D, w.to(DEV), ws.to(DEV), dx, workspace(M.hpo_mx8_dgrad_workspace(D, w)))
    want2, size2 = mu.matmul64(dy, b)
    mu.check(dx, want2, mu.product_tolerance(size2, r, want2, F32), "far dy")
    M.hpo_mx8_wgrad(D, x.to(DEV), xs.to(DEV), G, workspace(M.hpo_mx8_wgrad_workspace(D, x)), accumulate=False)
    mu.check(G, want, mu.product_tolerance(size, t, want, F32), "far dy, wgrad")
    del D
    G = far(torch.ones(2, r, cols), 2 ** 31 + 4, 2 ** 32)
    M.hpo_mx8_wgrad(dy.to(DEV), x.to(DEV), xs.to(DEV), G, workspace(M.hpo_mx8_wgrad_workspace(dy, x)))
    ones = torch.ones(2, r, cols, dtype=torch.float64)
    mu.check(G, want + 1, mu.product_tolerance(size, t, want + 1, F32, 1.0, ones), "far grad")


@pytest.mark.parametrize("log", [21, 22, 23, 24])
def test_rows_about_the_reach_of_32_bit_offsets(M, log):
    """Rows so far apart that a tile's 64 or 128 of them end before 2^30 bytes or behind them."""
    g, rs, n = gen(log), 2 ** log, 130
    x, xs = encode(torch.randn(1, n, 256, generator=g))
    w, ws = encode(torch.randn(1, 144, 256, generator=g))
    dy = torch.randn(1, n, 144, generator=g).to(BF16)
    a, b = mu.mx_values(x, xs), mu.mx_values(w, ws)
    X = far(x, rs)
    Y = torch.empty(1, n, 144, dtype=BF16, device=DEV)
    M.hpo_mx8_linear(X, xs.to(DEV), w.to(DEV), ws.to(DEV), Y, workspace(M.hpo_mx8_linear_workspace(X, w)))
    want, size = mu.matmul64(a, b.mT)
    cut = mu.aligned_cut(a, b)
    mu.check(Y, want, mu.product_tolerance(size + cut, 256, want, BF16) + cut, "x")
    want, size = mu.matmul64(dy.mT, a)
    tol = mu.product_tolerance(size, n, want, F32)
    for d, xx in ((dy.to(DEV), X), (far(dy, rs), x.to(DEV))):
        G = torch.empty(1, 144, 256, device=DEV)
        M.hpo_mx8_wgrad(d, xx, xs.to(DEV), G, workspace(M.hpo_mx8_wgrad_workspace(d, xx)), accumulate=False)
        mu.check(G, want, tol, "wgrad")
    del X, xx
    want, size = mu.matmul64(dy, b)
    tol = mu.product_tolerance(size, 144, want, F32)
    for dd, ww in ((d, w.to(DEV)), (dy.to(DEV), far(w, rs))):
        dx = torch.empty(1, n, 256, device=DEV)
        M.hpo_mx8_dgrad(dd, ww, ws.to(DEV), dx, workspace(M.hpo_mx8_dgrad_workspace(dd, ww)))
        mu.check(dx, want, tol, "dgrad")


# --------------------------------------------------------------------------
# nothing to add, and values that are none
# --------------------------------------------------------------------------
def test_sums_of_nothing(M):
    def e4(*s):
        return torch.empty(*s, dtype=E4M3, device=DEV), torch.empty(*s[:-1], -(-s[-1] // 32), dtype=torch.uint8, device=DEV)
    x, xs = e4(5, 0)
    w, ws = e4(7, 0)
    y = torch.full((5, 7), math.nan, dtype=BF16, device=DEV)
    M.hpo_mx8_linear(x, xs, w, ws, y)
    assert torch.equal(su.bits(y), torch.zeros_like(su.bits(y)))
    w, ws = e4(0, 40)
    dx = torch.full((5, 40), math.nan, device=DEV)
    M.hpo_mx8_dgrad(torch.empty(5, 0, dtype=BF16, device=DEV), w, ws, dx)
    assert torch.equal(dx, torch.zeros_like(dx))
    x, xs = e4(0, 40)
    dy = torch.empty(0, 6, dtype=F16, device=DEV)
    for gt in (F32, BF16):
        grad = torch.randn(6, 40, device=DEV).to(gt)
        kept = grad.clone()
        M.hpo_mx8_wgrad(dy, x, xs, grad, scale=3.0)
        assert torch.equal(grad, kept)
        M.hpo_mx8_wgrad(dy, x, xs, grad, accumulate=False)
        assert torch.equal(grad, torch.zeros_like(grad))
    # no tokens: nothing to write
    w, ws = e4(6, 40)
    M.hpo_mx8_linear(x, xs, w, ws, torch.empty(0, 6, dtype=BF16, device=DEV))
    M.hpo_mx8_save(torch.empty(0, 40, device=DEV), x, xs)
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    M.hpo_embedding(ids, torch.randn(3, 8, device=DEV), torch.empty(0, 8, device=DEV))
    grad = torch.randn(3, 8, device=DEV)
    kept = grad.clone()
    M.hpo_embedding_grad(ids, torch.empty(0, 8, device=DEV), grad, workspace(M.hpo_embedding_grad_workspace(ids, grad)))
    assert torch.equal(grad, kept)


# sizes of every tile, aligned and not
@pytest.mark.parametrize("t,c,r", [(40, 96, 50), (50, 100, 33), (600, 1024, 600), (2304, 512, 2304), (601, 515, 603)])
def test_nan_and_infinity_stay_where_they_enter(M, t, c, r):
    """NaN blocks and infinite gradients reach the results that read them, and no other: not a neighbour row, not
    what a tile reads behind an edge."""
    g = gen(t + c + r)
    x = operand(g, t, c)
    x[1, c - 1] = math.nan       # one block of row 1
    x[t - 1, 0] = math.inf       # as is an infinity
    w = 0.05 * torch.randn(r, c, generator=g)
    w[r - 1, 3] = math.nan
    (xq, xs), (wq, ws) = encode(x), encode(w)
    assert int(xs[1, -1]) == 255 and int(xs[t - 1, 0]) == 255
    dev = [v.to(DEV) for v in (xq, xs, wq, ws)]
    y = torch.empty(t, r, dtype=BF16, device=DEV)
    M.hpo_mx8_linear(*dev, y, workspace(M.hpo_mx8_linear_workspace(xq, wq)))
    bad = torch.zeros(t, r, dtype=torch.bool)
    bad[1] = bad[t - 1] = bad[:, r - 1] = True
    assert torch.equal(y.isnan().cpu(), bad) and not bool(y.isinf().any())
    dy = torch.randn(t, r, generator=g).to(BF16)
    dy[2, r // 2] = math.inf
    dy[t // 2, 0] = math.nan
    d = dy.to(DEV)
    dx = torch.empty(t, c, device=DEV)
    M.hpo_mx8_dgrad(d, dev[2], dev[3], dx, workspace(M.hpo_mx8_dgrad_workspace(d, wq)))
    bad = torch.zeros(t, c, dtype=torch.bool)
    bad[t // 2] = True
    bad[:, :32] = True           # the NaN block of W's last row meets every dY
    got = dx.cpu()
    assert bool(got[t // 2].isnan().all()) and bool(got[:, :32].isnan().all())
    inf = torch.zeros(t, c, dtype=torch.bool)
    inf[2, 32:] = True           # infinity times W's row: infinite, or NaN where an element of W is 0
    assert torch.equal(~got.isfinite() & ~bad, inf & ~bad)
    G = torch.zeros(r, c, device=DEV)
    M.hpo_mx8_wgrad(d, dev[0], dev[1], G, workspace(M.hpo_mx8_wgrad_workspace(d, xq)))
    bad = torch.zeros(r, c, dtype=torch.bool)
    bad[0] = bad[r // 2] = True
    bad[:, (c - 1) // 32 * 32:] = True
    bad[:, :32] = True
    assert torch.equal(~G.isfinite().cpu(), bad)


@pytest.mark.parametrize("n", [100, 5000, 70000])
def test_rows_of_padding_are_not_read(M, n):
    """dY is NaN and infinite where an id has no row: no gradient sees it.  A table without rows gives zeros."""
    g = gen(n)
    rows, cols = 37, 40
    ids = torch.randint(-30, rows + 30, (n,), generator=g)
    out = (ids < 0) | (ids >= rows)
    assert 0 < int(out.sum()) < n
    dy = torch.randn(n, cols, generator=g)
    dy[out] = torch.where(torch.rand(int(out.sum()), 1, generator=g) < 0.5, math.nan, math.inf)
    grad = torch.randn(rows, cols, generator=g)
    G = grad.to(DEV)
    M.hpo_embedding_grad(ids.to(DEV), dy.to(DEV), G, workspace(M.hpo_embedding_grad_workspace(ids, grad)))
    want, tol, _ = mu.embedding_grad(ids[~out], dy[~out], grad, 1.0, 0)
    mu.check(G, want, tol, f"{n}")
    none = torch.full((n, cols), math.nan, device=DEV)
    M.hpo_embedding(ids.to(DEV), torch.empty(0, cols, device=DEV), none)
    assert not bool(none.any())


# --------------------------------------------------------------------------
# large tiles with ragged edges, and sums in parts of unequal lengths
# --------------------------------------------------------------------------
@pytest.mark.parametrize("b,t,c,r", [(1, 1000, 40000, 912), (1, 1040, 1008, 30000), (1, 12000, 1040, 1000), (2, 500, 6000, 1000)])
@pytest.mark.parametrize("layout", ["dense", "aligned"])
def test_products_in_parts(M, b, t, c, r, layout):
    linear(M, b, t, c, r, BF16, layout, dev=DEV)
    dgrad(M, b, t, c, r, F16, BF16, layout, dev=DEV)
    dgrad(M, b, t, c, r, BF16, F32, layout, dev=DEV)
    wgrad(M, b, t, c, r, BF16, BF16, layout, True, dev=DEV)
    wgrad(M, b, t, c, r, F16, F32, layout, False, dev=DEV)


@pytest.mark.parametrize("layout", ["dense", "aligned", "padded"])
def test_linear_in_parts_of_large_tiles(M, layout):
    linear(M, 1, 1010, 50000, 1000, BF16, layout, dev=DEV)


# --------------------------------------------------------------------------
# many tokens
# --------------------------------------------------------------------------
@pytest.mark.parametrize("n,rows,cols,kind", [(65536, 1000, 24, "any"), (65537, 40000, 16, "any"), (70001, 9, 40, "any"),
                                              (66000, 300, 20, "same"), (131072, 128256, 8, "any"), (100000, 50, 8, "none"),
                                              (200003, 70000, 3, "padded")])
def test_embedding_grad_of_many_tokens(M, n, rows, cols, kind):
    g = gen(n)
    ids = {"any": torch.randint(-3, rows + 3, (n,), generator=g), "same": torch.full((n,), 17), "none": torch.full((n,), -1),
           "padded": torch.where(torch.rand(n, generator=g) < 0.8, rows, torch.randint(0, rows, (n,), generator=g))}[kind]
    dy = torch.randn(n, cols, generator=g).to(BF16)
    grad = torch.randn(rows, cols, generator=g)
    G = grad.to(DEV)
    M.hpo_embedding_grad(ids.to(DEV), dy.to(DEV), G, workspace(M.hpo_embedding_grad_workspace(ids, grad)), scale=-2.0)
    want, tol, some = mu.embedding_grad(ids, dy, grad, -2.0, 0)
    mu.check(G, want, tol, f"{n} {kind}")
    assert torch.equal(su.bits(G)[~some], su.bits(grad)[~some])


@pytest.mark.parametrize("n,rows,cols", [(2 ** 21, 2 ** 21, 3), (60000, 2 ** 21, 5), (128, 2 ** 21, 9), (200, 3, 2 ** 21)])
def test_embedding_at_the_largest_sizes(M, n, rows, cols):
    g = gen(n + cols)
    ids = torch.randint(-2, rows + 2, (n,), generator=g)
    ids[:2] = torch.tensor([rows - 1, 0])
    dy = torch.randn(n, cols, generator=g).to(BF16)
    grad = torch.randn(rows, cols, generator=g)
    G = grad.to(DEV)
    M.hpo_embedding_grad(ids.to(DEV), dy.to(DEV), G, workspace(M.hpo_embedding_grad_workspace(ids, grad)))
    want, tol, some = mu.embedding_grad(ids, dy, grad, 1.0, 0)
    mu.check(G, want, tol, f"{n} {rows} {cols}")
    assert torch.equal(su.bits(G)[~some], su.bits(grad)[~some])
    out = torch.empty(n, cols, device=DEV)
    M.hpo_embedding(ids.to(DEV), grad.to(DEV), out)
    assert torch.equal(out.cpu(), mu.embedding(ids, grad, 1.0, 0))


@pytest.mark.parametrize("b,t,c,r", [(65535, 2, 33, 3), (1, 2 ** 21, 40, 4), (1, 2, 2 ** 21, 3), (1, 2, 2 ** 21 - 1, 3),
                                     (1, 3, 40, 2 ** 21), (1, 3, 36, 2 ** 21 - 5)])
def test_products_at_the_largest_sizes(M, b, t, c, r):
    linear(M, b, t, c, r, BF16, "dense", dev=DEV)
    dgrad(M, b, t, c, r, BF16, F32, "dense", dev=DEV)
    wgrad(M, b, t, c, r, F16, F32, "dense", True, dev=DEV)


# --------------------------------------------------------------------------
# gradients against differences
# --------------------------------------------------------------------------
def small(g, *shape):
    """Values of two bits at scale 1: with up to 64 of them in a sum every result here is exact in fp16."""
    vals = torch.tensor([0.0, 1.0, -1.0, 1.5, -1.5, 2.0])
    v = vals[torch.randint(0, 6, shape, generator=g)]
    return v, v.to(E4M3).to(DEV), torch.full((*shape[:-1], -(-shape[-1] // 32)), 127, dtype=torch.uint8, device=DEV)


def test_gradients_against_differences(M):
    """<dY, Y(X + D) - Y(X)> = <dX, D> and the same for W: the layer is linear and nothing here rounds."""
    b, t, c, r = 2, 45, 64, 50
    g = gen(8)
    (x, xq, xs), (x2, x2q, _) = small(g, b, t, c), small(g, b, t, c)
    (w, wq, ws), (w2, w2q, _) = small(g, b, r, c), small(g, b, r, c)
    dy = torch.randint(-2, 3, (b, t, r), generator=g).to(F16).to(DEV)

    def forward(a, v):
        y = torch.empty(b, t, r, dtype=F16, device=DEV)
        M.hpo_mx8_linear(a, xs, v, ws, y, workspace(M.hpo_mx8_linear_workspace(a, v)))
        return y.double()
    dx = torch.empty(b, t, c, dtype=F32, device=DEV)
    M.hpo_mx8_dgrad(dy, wq, ws, dx, workspace(M.hpo_mx8_dgrad_workspace(dy, wq)))
    G = torch.zeros(b, r, c, device=DEV)
    M.hpo_mx8_wgrad(dy, xq, xs, G, workspace(M.hpo_mx8_wgrad_workspace(dy, xq)))
    y = forward(xq, wq)
    assert float((dy.double() * (forward(x2q, wq) - y)).sum()) == float((dx.double().cpu() * (x2 - x).double()).sum())
    assert float((dy.double() * (forward(xq, w2q) - y)).sum()) == float((G.double().cpu() * (w2 - w).double()).sum())


def test_embedding_gradient_against_differences(M):
    g = gen(6)
    ids = torch.randint(-2, 23, (200,), generator=g).to(DEV)
    table, step = (torch.randint(-3, 4, (20, 33), generator=g).float().to(DEV) for _ in range(2))
    dy = torch.randint(-3, 4, (200, 33), generator=g).float().to(DEV)
    a, b, G = torch.empty_like(dy), torch.empty_like(dy), torch.zeros_like(table)
    M.hpo_embedding(ids, table, a, scale=2.0)
    M.hpo_embedding(ids, table + step, b, scale=2.0)
    M.hpo_embedding_grad(ids, dy, G, workspace(M.hpo_embedding_grad_workspace(ids, G)), scale=2.0)
    assert float((dy * (b - a)).double().sum()) == float((G * step).double().sum())


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------
def test_a_training_step_of_a_layer_behind_an_embedding(M):
    """Tokens -> table in 8 bits -> kept activation -> layer, both gradients added to main grads over two
    micro-batches, then the optimizers' steps, which write the 8-bit weights the next forward pass reads.  Each result is
    checked against binary64 from the operands that the call read."""
    from mixed_precision_optimizer_amd.optimizer import StackMuon
    g = gen(12)
    n, vocab, cols, outs = 333, 97, 160, 224
    master_e, master_w = torch.randn(vocab, cols, generator=g), 0.1 * torch.randn(outs, cols, generator=g)
    (eq, es), (wq, ws) = encode(master_e), encode(master_w)
    eq, es, wq, ws, master_e, master_w = (v.to(DEV) for v in (eq, es, wq, ws, master_e, master_w))
    opt_e = StackMuon(master_e, eq, es, lr=0.1)
    opt_w = StackMuon(master_w, wq, ws, lr=0.1)
    e = torch.empty(n, cols, dtype=BF16, device=DEV)
    q, qs = torch.empty(n, cols, dtype=E4M3, device=DEV), torch.empty(n, cols // 32, dtype=torch.uint8, device=DEV)
    y, dx = torch.empty(n, outs, dtype=BF16, device=DEV), torch.empty(n, cols, dtype=BF16, device=DEV)
    for step in range(2):
        ge, gw = torch.zeros(vocab, cols, device=DEV), torch.zeros(outs, cols, device=DEV)
        we, wt = torch.zeros(vocab, cols, dtype=torch.float64), torch.zeros(outs, cols, dtype=torch.float64)
        te, tt = torch.zeros_like(we), torch.zeros_like(wt)
        before = su.bits(wq).clone()
        for micro in range(2):
            ids = torch.randint(-1, vocab, (n,), generator=g)
            M.hpo_embedding(ids.to(DEV), eq, e, scales=es, scale=math.sqrt(cols))
            want = mu.embedding(ids, mu.mx_values(eq, es).float(), math.sqrt(cols), 0).to(BF16)
            assert torch.equal(su.bits(e), su.bits(want))
            M.hpo_mx8_save(e, q, qs)
            ref, byte = su.mx_reference(want.float())
            assert torch.equal(qs.cpu(), byte)
            M.hpo_mx8_linear(q, qs, wq, ws, y, workspace(M.hpo_mx8_linear_workspace(q, wq)))
            a, b = mu.mx_values(q, qs), mu.mx_values(wq, ws)
            want, size = mu.matmul64(a, b.mT)
            cut = mu.aligned_cut(a, b)
            mu.check(y, want, mu.product_tolerance(size + cut, cols, want, BF16) + cut, f"y {step}")
            dy = torch.randn(n, outs, generator=g).to(BF16)
            d = dy.to(DEV)
            M.hpo_mx8_dgrad(d, wq, ws, dx, workspace(M.hpo_mx8_dgrad_workspace(d, wq)))
            want, size = mu.matmul64(dy, b)
            mu.check(dx, want, mu.product_tolerance(size, outs, want, BF16), f"dx {step}")
            was = gw.cpu().double()
            M.hpo_mx8_wgrad(d, q, qs, gw, workspace(M.hpo_mx8_wgrad_workspace(d, q)), scale=0.5)
            part, size = mu.matmul64(dy.mT, a)
            wt, tt = wt + 0.5 * part, tt + mu.product_tolerance(size, n, was + 0.5 * part, F32, 0.5, was)
            was = ge.cpu()
            M.hpo_embedding_grad(ids.to(DEV), dx, ge, workspace(M.hpo_embedding_grad_workspace(ids, ge)), scale=math.sqrt(cols))
            want, tol, _ = mu.embedding_grad(ids, dx.cpu(), was, math.sqrt(cols), 0)
            mu.check(ge, want, tol, f"table's gradient {step}")
        mu.check(gw, wt, tt, f"weight's gradient {step}")
        opt_w.step(gw)
        opt_e.step(ge)
        for wt8, sc, master in ((wq, ws, master_w), (eq, es, master_e)):
            ref, byte = su.mx_reference(master.cpu())
            assert torch.equal(sc.cpu(), byte)
            got = su.bits(wt8)
            assert bool(((got == ref) | (((got | ref) & 0x7F) == 0)).all())
        assert not torch.equal(su.bits(wq), before)
