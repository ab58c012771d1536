"""Model operators on the GPU against binary64 references (model_util.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

import model_util as mu  # noqa: E402
import stack_util as su  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, F16, E4M3 = torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def M():
    from mixed_precision_optimizer_amd import hpo_model
    assert torch.cuda.is_available()
    hpo_model.load()
    return hpo_model


def gen(seed):
    return torch.Generator().manual_seed(seed)


def workspace(n, fill=0xA5):
    """A workspace that holds nothing useful: calls must not read what they did not write."""
    return torch.full((max(n, 1),), fill, dtype=torch.uint8, device=DEV)


class Guarded:
    """A strided device view inside a buffer whose other elements must stay as they are."""

    def __init__(self, value, layout="dense", fill=True):
        shape, dtype = value.shape, value.dtype
        b = shape[0] if len(shape) == 3 else 1
        r, c = shape[-2:]
        if layout == "dense":
            self.buf = torch.empty(b, r, c, dtype=dtype, device=DEV)
            view = self.buf
        elif layout == "padded":
            self.buf = torch.empty(b, r + 1, c + 5, dtype=dtype, device=DEV)
            view = self.buf[:, :r, :c]
        elif layout == "aligned":   # rows of whole 16-byte pieces, longer than the matrix's
            self.buf = torch.empty(b, r, (c + 31) // 16 * 16, dtype=dtype, device=DEV)
            view = self.buf[:, :, :c]
        elif layout == "offset":
            self.buf = torch.empty(b * r * c + 1, dtype=dtype, device=DEV)
            view = self.buf[1:].view(b, r, c)
        else:   # "rows": the matrices lie side by side in every row
            self.buf = torch.empty(r, b, c, dtype=dtype, device=DEV)
            view = self.buf.transpose(0, 1)
        # what lies around the matrix is NaN: nothing of it may reach a result
        if dtype == E4M3:
            self.buf.view(torch.uint8).fill_(0x7F)
        else:
            self.buf.fill_(math.nan)
        self.view = view if len(shape) == 3 else view[0]
        self.view.copy_(value.to(DEV))
        self.before = su.bits(self.buf).clone()

    def untouched_outside(self):
        mask = torch.ones(self.buf.shape, dtype=torch.uint8, device=DEV)
        mask.as_strided(self.view.shape, self.view.stride(), self.view.storage_offset()).zero_()
        keep = mask.cpu().bool()
        assert torch.equal(su.bits(self.buf)[keep], self.before[keep]), "elements outside the matrix changed"


def blank(shape, dtype, layout="dense"):
    return Guarded(torch.full(shape, 7.0).to(dtype), layout)


def encode(x):
    q, byte = su.mx_reference(x)
    return q.view(E4M3), byte


# --------------------------------------------------------------------------
# hpo_embedding
# --------------------------------------------------------------------------
def draw_ids(g, n, rows, first, dtype):
    ids = torch.randint(first - rows // 4 - 2, first + rows + rows // 4 + 2, (n,), generator=g)
    if n > 4:
        ids[1], ids[2], ids[3] = first, first + rows - 1, -1
    return ids.to(dtype)


@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (1, 7, 64), (5, 3, 8), (17, 1000, 333), (64, 50, 65), (300, 20, 512),
                                         (33, 900, 2048), (9, 40, 4100), (2000, 17, 31)])
@pytest.mark.parametrize("weight", [BF16, F16, F32, E4M3])
def test_embedding(M, n, rows, cols, weight):
    for k, (out, ids_t, layout, first) in enumerate([(BF16, torch.int64, "dense", 0), (F16, torch.int32, "padded", 11),
                                                     (F32, torch.int64, "offset", 5)]):
        g = gen(n + rows + cols + k)
        ids = draw_ids(g, n, rows, first, ids_t)
        w = 0.02 * torch.randn(rows, cols, generator=g)
        scale = math.sqrt(cols)
        if weight == E4M3:
            q, byte = encode(w)
            ref = mu.mx_values(q, byte).float()
            src, sc = Guarded(q, layout), byte.to(DEV)
        else:
            ref = w.to(weight).float()
            src, sc = Guarded(w.to(weight), layout), None
        dst = blank((n, cols), out, layout)
        M.hpo_embedding(ids.to(DEV), src.view, dst.view, scales=sc, scale=scale, first=first)
        want = mu.embedding(ids, ref, scale, first).to(out)
        assert torch.equal(su.bits(dst.view), su.bits(want)), (out, layout)
        dst.untouched_outside()


def test_embedding_of_far_ids_and_extreme_scales(M):
    """64-bit ids far outside, scale bytes at both ends, a block of NaN."""
    q = torch.full((4, 64), 448.0).to(E4M3)
    byte = torch.tensor([[0, 1], [126, 127], [253, 254], [255, 100]], dtype=torch.uint8)
    q.view(torch.uint8)[3, :32] = 0x7F
    q.view(torch.uint8)[0, :8] = torch.arange(1, 9, dtype=torch.uint8)   # subnormals at the smallest scale
    ids = torch.tensor([0, 1, 2, 3, -2 ** 63, 2 ** 63 - 1, 2 ** 32, 4])
    out = torch.empty(8, 64, device=DEV)
    M.hpo_embedding(ids.to(DEV), q.to(DEV), out, scales=byte.to(DEV))
    with torch.no_grad():
        want = mu.embedding(ids, mu.mx_values(q, byte).float(), 1.0, 0)
    got = out.cpu()
    assert torch.equal(torch.nan_to_num(got, nan=-1.0, posinf=-2.0), torch.nan_to_num(want, nan=-1.0, posinf=-2.0))


# --------------------------------------------------------------------------
# hpo_embedding_grad
# --------------------------------------------------------------------------
def run_embedding_grad(M, ids, dy, grad, scale, first, layout="dense", tag=""):
    G, D = Guarded(grad, layout), Guarded(dy, layout)
    ws = workspace(M.hpo_embedding_grad_workspace(ids, grad))
    M.hpo_embedding_grad(ids.to(DEV), D.view, G.view, ws, scale=scale, first=first)
    want, tol, some = mu.embedding_grad(ids, dy, grad, scale, first)
    mu.check(G.view, want, tol, tag)
    assert torch.equal(su.bits(G.view)[~some], su.bits(grad)[~some]), "rows without a token changed"
    G.untouched_outside()
    return G.view


@pytest.mark.parametrize("n,rows,cols", [(1, 1, 1), (1, 9, 70), (2, 1, 8), (100, 5, 33), (128, 1000, 512), (129, 1, 7),
                                         (129, 100, 520), (200, 3, 64), (1000, 2047, 100), (1000, 2048, 40),
                                         (4096, 64, 12), (8192, 128256, 16), (8193, 300, 24), (9000, 1500, 8),
                                         (20000, 70000, 9), (40000, 10, 65)])
def test_embedding_grad(M, n, rows, cols):
    for k, (dt, gt, it, layout, first) in enumerate([(BF16, F32, torch.int64, "dense", 0),
                                                     (F16, BF16, torch.int32, "padded", 3),
                                                     (F32, F32, torch.int32, "offset", 2 ** 31 - 2 ** 18)]):
        g = gen(n * 7 + rows + cols + k)
        ids = draw_ids(g, n, rows, first, it)
        dy = torch.randn(n, cols, generator=g).to(dt)
        grad = torch.randn(rows, cols, generator=g).to(gt)
        run_embedding_grad(M, ids, dy, grad, 0.37, first, layout, f"{n}x{rows}x{cols} {dt} {gt}")


@pytest.mark.parametrize("n", [60, 128, 129, 5000, 8192, 30000])
@pytest.mark.parametrize("kind", ["same", "two", "sorted", "none", "padded"])
def test_embedding_grad_runs(M, n, kind):
    """One token all along, two halves, sorted tokens, no token inside, mostly padding."""
    g = gen(n)
    rows, cols = 500, 72
    ids = {"same": torch.full((n,), 77), "two": torch.where(torch.arange(n) < n // 2 + 3, 8, 3),
           "sorted": torch.arange(n) * rows // n, "none": torch.full((n,), -1),
           "padded": torch.where(torch.rand(n, generator=g) < 0.9, -100, torch.randint(0, rows, (n,), generator=g))}[kind]
    dy = torch.randn(n, cols, generator=g).to(BF16)
    run_embedding_grad(M, ids, dy, torch.randn(rows, cols, generator=g), 1.0, 0, tag=f"{kind} {n}")


def test_embedding_grad_is_the_same_twice_and_on_another_stream(M):
    g = gen(3)
    ids = torch.randint(0, 40, (12000,), generator=g).to(DEV)
    dy = torch.randn(12000, 264, generator=g).to(BF16).to(DEV)
    outs = []
    for k in range(3):
        grad = torch.zeros(50, 264, device=DEV)
        ws = workspace(M.hpo_embedding_grad_workspace(ids, grad), 0x11 * (k + 1))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            M.hpo_embedding_grad(ids, dy, grad, ws)
        torch.cuda.current_stream().wait_stream(s)
        outs.append(su.bits(grad))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_embedding_grad_keeps_nan_to_its_row(M):
    ids = torch.tensor([3, 1, 3, 0, 1])
    dy = torch.ones(5, 20)
    dy[2, 4] = math.nan
    dy[3, 6] = math.inf
    grad = torch.zeros(6, 20)
    G = grad.to(DEV)
    M.hpo_embedding_grad(ids.to(DEV), dy.to(DEV), G, None)
    want = torch.zeros(6, 20)
    want.index_add_(0, ids, dy)
    assert torch.equal(G.cpu().nan_to_num(-5, -6), want.nan_to_num(-5, -6))


# --------------------------------------------------------------------------
# hpo_mx8_save
# --------------------------------------------------------------------------
@pytest.mark.parametrize("b,r,c", [(1, 1, 1), (1, 1, 31), (2, 3, 32), (1, 5, 33), (3, 43, 257), (2, 9, 64), (1, 300, 72),
                                   (1, 3, 2048), (1, 2, 5000), (4, 1, 129)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_mx8_save(M, b, r, c, dtype):
    for layout in ("dense", "padded", "offset", "rows"):
        g = gen(b * 1000 + r * 10 + c)
        x = (torch.randn(b, r, c, generator=g) * torch.exp(3 * torch.randn(b, r, 1, generator=g))).to(dtype)
        if r > 2 and c > 40:
            x[0, 1, :32] = 0.0
            x[0, 2, 33] = math.inf
            x[-1, -1, 0] = math.nan
        src, dst = Guarded(x, layout), blank((b, r, c), E4M3, layout)
        sc = torch.full((b, r, -(-c // 32)), 9, dtype=torch.uint8, device=DEV)
        M.hpo_mx8_save(src.view, dst.view, sc)
        q, byte = su.mx_reference(x.float())
        assert torch.equal(sc.cpu(), byte), layout
        got = su.bits(dst.view)
        same = (got == q) | (((got | q) & 0x7F) == 0)   # -0 and 0 stand for the same
        assert bool(same.all()), (layout, int((~same).sum()))
        dst.untouched_outside()


def test_mx8_save_of_extremes(M):
    """Ties, saturation, subnormal blocks, the ends of fp32."""
    v = [0.0, 1e-45, 1.1754944e-38, 2.0 ** -118, 2.0 ** -119, 3.4028235e38, 448.0, 449.0, 464.0, 480.0, 1.0625, 1.1875, 17.0,
         2.0 ** -9, 2.0 ** -10, -2.0 ** -10]
    x = torch.tensor(v).repeat(32, 1).T.contiguous()
    y = torch.tensor(v).repeat(2).view(1, 32) * torch.linspace(0.5, 1.0, 32)
    x = torch.cat([x, y, y * 1e-30, y * 1e-37])
    q, byte = su.mx_reference(x)
    got, sc = torch.empty(x.shape, dtype=E4M3, device=DEV), torch.empty(x.shape[0], 1, dtype=torch.uint8, device=DEV)
    M.hpo_mx8_save(x.to(DEV), got, sc)
    assert torch.equal(sc.cpu(), byte)
    b = su.bits(got)
    assert bool(((b == q) | (((b | q) & 0x7F) == 0)).all())


# --------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------
# (batch, tokens, cols, rows): every tile, cuts of the depth, odd sizes, one token, few of everything
SHAPES = [(1, 1, 1, 1), (1, 1, 128, 256), (1, 3, 33, 5), (2, 5, 16, 31), (1, 64, 64, 64), (1, 65, 129, 63),
          (3, 37, 200, 96), (1, 128, 512, 128), (2, 130, 260, 300), (1, 1, 4096, 1000), (1, 300, 1024, 17),
          (1, 16, 3000, 700), (1, 2000, 48, 80), (5, 257, 255, 257), (1, 512, 544, 4096), (1, 9000, 64, 72)]
LARGE = [(1, 2560, 528, 3000), (1, 4096, 4096, 4096), (12, 700, 384, 1100), (1, 30000, 256, 512), (1, 2500, 2100, 2600)]


def operand(g, *shape, outliers=True):
    x = torch.randn(*shape, generator=g)
    return x * torch.exp(torch.randn(shape[-1], generator=g)) if outliers else x


def linear(M, b, t, c, r, out, layout, seed=0, tag="", dev="cpu"):
    g = gen(seed + b + 3 * t + 5 * c + 7 * r)
    xq, xs = encode(operand(g, b, t, c))
    wq, ws = encode(0.05 * operand(g, b, r, c, outliers=False))
    X, W, Y = Guarded(xq, layout), Guarded(wq, layout), blank((b, t, r), out, layout)
    work = workspace(M.hpo_mx8_linear_workspace(X.view, W.view))
    M.hpo_mx8_linear(X.view, xs.to(DEV), W.view, ws.to(DEV), Y.view, work)
    x, w = mu.mx_values(xq, xs).to(dev), mu.mx_values(wq, ws).to(dev)
    want, size = mu.matmul64(x, w.mT)
    tol = mu.product_tolerance(size + mu.aligned_cut(x, w), c, want, out) + mu.aligned_cut(x, w)
    mu.check(Y.view, want, tol, f"linear {b}x{t}x{c}x{r} {out} {layout} {tag}")
    Y.untouched_outside()


def linear_exact(M, b, t, c, r, out, layout, dev="cpu"):
    """Values of two bits at scales that differ by up to four: no product lies 13 bits below another and every
    sum is a multiple of 2^-8 under 2^16, so the matrix cores lose nothing and the result is the sum's one
    rounding, bit for bit."""
    g = gen(31 + b + 3 * t + 5 * c + 7 * r)
    vals = torch.tensor([0.0, 1.0, -1.0, 1.5, -1.5, 2.0])

    def small(*shape):
        nb = -(-shape[-1] // 32)
        return (vals[torch.randint(0, 6, shape, generator=g)].to(E4M3),
                torch.randint(125, 128, (*shape[:-1], nb), generator=g).to(torch.uint8))
    (xq, xs), (wq, ws) = small(b, t, c), small(b, r, c)
    X, W, Y = Guarded(xq, layout), Guarded(wq, layout), blank((b, t, r), out, layout)
    M.hpo_mx8_linear(X.view, xs.to(DEV), W.view, ws.to(DEV), Y.view, workspace(M.hpo_mx8_linear_workspace(X.view, W.view)))
    want, size = mu.matmul64(mu.mx_values(xq, xs).to(dev), mu.mx_values(wq, ws).mT.to(dev))
    assert float(size.max()) < 2 ** 16
    assert torch.equal(su.bits(Y.view + 0.0), su.bits(want.float().to(out) + 0.0)), (b, t, c, r, out, layout)
    Y.untouched_outside()


def dgrad(M, b, t, c, r, dt, out, layout, tag="", dev="cpu"):
    g = gen(11 + b + 3 * t + 5 * c + 7 * r)
    dy = operand(g, b, t, r, outliers=False).to(dt)
    wq, ws = encode(0.05 * operand(g, b, r, c, outliers=False))
    D, W, X = Guarded(dy, layout), Guarded(wq, layout), blank((b, t, c), out, layout)
    work = workspace(M.hpo_mx8_dgrad_workspace(D.view, W.view))
    M.hpo_mx8_dgrad(D.view, W.view, ws.to(DEV), X.view, work)
    w = mu.mx_values(wq, ws)
    if dt == F16:
        w = w.half().double()   # as documented: in dy's type
    want, size = mu.matmul64(dy.to(dev), w.to(dev))
    mu.check(X.view, want, mu.product_tolerance(size, r, want, out), f"dgrad {b}x{t}x{c}x{r} {dt} {out} {layout} {tag}")
    X.untouched_outside()


def wgrad(M, b, t, c, r, dt, gt, layout, accumulate, scale=0.3, tag="", dev="cpu"):
    g = gen(23 + b + 3 * t + 5 * c + 7 * r)
    dy = operand(g, b, t, r, outliers=False).to(dt)
    xq, xs = encode(operand(g, b, t, c).to(dt).float())
    grad = torch.randn(b, r, c, generator=g).to(gt)
    D, X = Guarded(dy, layout), Guarded(xq, layout)
    G = Guarded(grad if accumulate else torch.full_like(grad, math.nan), layout)
    work = workspace(M.hpo_mx8_wgrad_workspace(D.view, X.view))
    M.hpo_mx8_wgrad(D.view, X.view, xs.to(DEV), G.view, work, scale=scale, accumulate=accumulate)
    s = float(torch.tensor(scale, dtype=F32))
    want, size = mu.matmul64(dy.mT.to(dev), mu.mx_values(xq, xs).to(dev))
    want = s * want + (grad.double().to(dev) if accumulate else 0.0)
    tol = mu.product_tolerance(size, t, want, gt, s, grad.double().to(dev) if accumulate else None)
    mu.check(G.view, want, tol, f"wgrad {b}x{t}x{c}x{r} {dt} {gt} {layout} {accumulate} {tag}")
    G.untouched_outside()


@pytest.mark.parametrize("b,t,c,r", SHAPES)
def test_mx8_linear(M, b, t, c, r):
    for out, layout in ((F16, "dense"), (BF16, "aligned"), (F16, "padded"), (F16, "offset"), (BF16, "rows")):
        linear(M, b, t, c, r, out, layout)
        linear_exact(M, b, t, c, r, out, layout)


@pytest.mark.parametrize("b,t,c,r", SHAPES)
def test_mx8_dgrad(M, b, t, c, r):
    for dt, out, layout in ((BF16, F32, "dense"), (BF16, BF16, "aligned"), (F16, F16, "padded"), (F16, F32, "offset"),
                            (BF16, BF16, "rows"), (F16, F32, "aligned")):
        dgrad(M, b, t, c, r, dt, out, layout)


@pytest.mark.parametrize("b,t,c,r", SHAPES)
def test_mx8_wgrad(M, b, t, c, r):
    for dt, gt, layout, acc in ((BF16, F32, "dense", True), (BF16, BF16, "aligned", False), (F16, F32, "padded", True),
                                (F16, BF16, "offset", True), (BF16, F32, "rows", False), (F16, F32, "aligned", True)):
        wgrad(M, b, t, c, r, dt, gt, layout, acc)


@pytest.mark.parametrize("b,t,c,r", LARGE)
def test_mx8_products_of_large_tiles(M, b, t, c, r):
    """The reference's products run on the GPU, in binary64."""
    for layout in ("dense", "padded"):
        linear(M, b, t, c, r, F16, layout, dev=DEV)
        linear_exact(M, b, t, c, r, BF16, layout, dev=DEV)
        dgrad(M, b, t, c, r, BF16, F32, layout, dev=DEV)
        wgrad(M, b, t, c, r, BF16, F32, layout, True, dev=DEV)
