"""Stack operators on the GPU against binary64 references (stack_util.py)."""
import math

import pytest

torch = pytest.importorskip("torch")

import stack_util as su  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = math.inf


@pytest.fixture(scope="module")
def S():
    from mixed_precision_optimizer_amd import hpo_stack
    assert torch.cuda.is_available()
    hpo_stack.load()
    return hpo_stack


def gen(seed):
    return torch.Generator().manual_seed(seed)


def workspace(n, fill=0xA5):
    """A workspace that holds nothing useful: calls must not read what they did not write."""
    return torch.full((max(n, 1),), fill, dtype=torch.uint8, device=DEV)


class Guarded:
    """A strided device view inside a buffer whose other elements must stay as they are."""

    def __init__(self, shape, dtype, layout, fill=None):
        b, r, c = shape
        if layout == "dense":
            self.buf = torch.empty(b, r, c + 0, dtype=dtype, device=DEV)
            self.view = self.buf
        elif layout == "padded":
            self.buf = torch.empty(b, r + 1, c + 5, dtype=dtype, device=DEV)
            self.view = self.buf[:, :r, :c]
        elif layout == "offset":
            self.buf = torch.empty(b * r * c + 1, dtype=dtype, device=DEV)
            self.view = self.buf[1:].view(b, r, c)
        else:   # "rows": the matrices lie side by side in every row
            self.buf = torch.empty(r, b, c, dtype=dtype, device=DEV)
            self.view = self.buf.transpose(0, 1)
        self.buf.view(torch.uint8).random_(0, 256) if dtype == torch.float8_e4m3fn else self.buf.fill_(7.0)
        if fill is not None:
            self.view.copy_(fill)
        self.before = su.bits(self.buf).clone()

    def untouched_outside(self):
        mask = torch.ones_like(self.buf, dtype=torch.uint8)
        at = mask.as_strided(self.view.shape, self.view.stride(), self.view.storage_offset())
        at.zero_()
        keep = mask.cpu().bool()
        assert torch.equal(su.bits(self.buf)[keep], self.before[keep]), "elements outside the stack changed"

    def unchanged(self):
        assert torch.equal(su.bits(self.buf), self.before)


# --------------------------------------------------------------------------
# hpo_orthogonalize
# --------------------------------------------------------------------------
def gradient(seed, b, r, c, noise=0.3):
    g = gen(seed)
    k = max(1, min(r, c) // 16)
    return (torch.randn(b, r, k, generator=g) @ torch.randn(b, k, c, generator=g) / math.sqrt(k)
            + noise * torch.randn(b, r, c, generator=g)) * 1e-3


def ortho(S, G, M=None, out=None, cfg=None, ws=None, **kw):
    cfg = cfg or S.hpo.make_muon_cfg()
    out = torch.full(G.shape, 9.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    ws = workspace(S.hpo_orthogonalize_workspace(G)) if ws is None else ws
    S.hpo_orthogonalize(G, out, cfg, ws, momentum=M, **kw)
    return out


def check_ortho(got, g64, steps=5, coeffs=None, eps=1e-7, tag=""):
    got = got.detach().double().cpu()
    for z in range(g64.shape[0]):
        e, tol = su.ns_tolerance(g64[z], steps, coeffs, eps)
        n = float(torch.linalg.vector_norm(e))
        d = float(torch.linalg.vector_norm(got[z] - e))
        print(f"[ortho] {tag}[{z}] rel {d / n if n else d:.2e} (allowed {tol:.2e})", flush=True)
        assert d <= tol * n, (tag, z, d, n)


@pytest.mark.parametrize("b,r,c", [(1, 1, 1), (1, 1, 300), (2, 300, 1), (3, 2, 7), (2, 2, 2), (2, 16, 16), (2, 64, 64), (2, 128, 640),
                                   (2, 640, 128), (3, 129, 257), (1, 256, 256), (2, 300, 520), (1, 520, 300),
                                   (5, 33, 1000), (4, 128, 129), (2, 96, 2048), (1, 17, 16384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize(S, b, r, c, dtype):
    G = gradient(r * 1000 + c, b, r, c).to(dtype)
    out = ortho(S, G.to(DEV))
    check_ortho(out, G.double(), tag=f"{b}x{r}x{c} {dtype}")


@pytest.mark.parametrize("b,r,c", [(400, 256, 256), (64, 512, 500), (2, 2048, 2100), (2, 2100, 2048), (1, 4000, 4100),
                                   (2, 260, 5000), (1, 1300, 9001), (1, 4096, 14336), (1, 14336, 4096), (1, 200, 20000),
                                   (64, 100, 3000), (300, 3000, 20)])
def test_orthogonalize_every_tile_and_cut(S, b, r, c):
    """Stacks that take the larger tiles and the Gram products cut in depth; the reference runs on the GPU."""
    g = torch.Generator(device=DEV).manual_seed(b + r + c)
    G = 1e-3 * torch.randn(b, r, c, generator=g, device=DEV)
    M = 1e-3 * torch.randn(b, r, c, generator=g, device=DEV)
    gt = G + 0.95 * (0.95 * M + G)
    out = ortho(S, G, M)
    for z in sorted({0, b // 2, b - 1}):
        e, tol = su.ns_tolerance(gt[z])
        d = float(torch.linalg.vector_norm(out[z].double() - e) / torch.linalg.vector_norm(e))
        print(f"[ortho] {b}x{r}x{c}[{z}] rel {d:.2e} (allowed {tol:.2e})", flush=True)
        assert d <= tol, z


@pytest.mark.parametrize("layout", ["dense", "padded", "offset", "rows"])
@pytest.mark.parametrize("r,c", [(100, 333), (260, 130), (64, 256)])
def test_orthogonalize_strides(S, layout, r, c):
    b = 3
    G = gradient(5, b, r, c)
    M = 10 * gradient(6, b, r, c)
    g, m, o = (Guarded((b, r, c), dt, layout, f) for dt, f in ((torch.float32, G), (torch.float32, M),
                                                               (torch.bfloat16, None)))
    ortho(S, g.view, m.view, o.view)
    mu = torch.tensor(0.95, dtype=torch.float32)
    M1 = mu * M + G
    assert torch.equal(m.view.cpu(), M1)
    check_ortho(o.view, (G + mu * M1).double(), tag=layout)
    g.unchanged()
    m.untouched_outside()
    o.untouched_outside()


@pytest.mark.parametrize("form", [0, 1])
@pytest.mark.parametrize("nesterov", [False, True])
def test_orthogonalize_momentum_and_clip(S, form, nesterov):
    b, r, c = 2, 150, 80
    G, M = gradient(7, b, r, c), gradient(8, b, r, c)
    cfg = S.hpo.make_muon_cfg(momentum=0.9, nesterov=nesterov, momentum_form=form)
    norm = torch.tensor([3.0], device=DEV)
    m = M.to(DEV)
    out = ortho(S, G.to(DEV), m, cfg=cfg, inv_scale=0.5, max_norm=1.5, d_norm=norm)
    f = lambda x: torch.tensor(x, dtype=torch.float32)
    g = (G * f(0.5)) * f(1.5 / (3.0 + 1e-6))
    mu, omu = f(0.9), f(1.0 - 0.9)
    M1 = mu * M + g if form == 0 else mu * M + omu * g
    gt = (g + mu * M1 if form == 0 else omu * g + mu * M1) if nesterov else M1
    assert torch.equal(m.cpu(), M1)
    check_ortho(out, gt.double(), tag=f"form {form} nesterov {nesterov}")


def test_orthogonalize_low_rank_keeps_its_small_directions(S):
    """Strong directions over a floor of 1 %: fp16 operands alone are off by 3e-2 here."""
    G = gradient(11, 2, 256, 512, noise=0.01)
    e, tol = su.ns_tolerance(G[0].double())
    assert tol < 8e-3
    check_ortho(ortho(S, G.to(DEV)), G.double(), tag="low rank")


@pytest.mark.parametrize("steps,coeffs", [(1, None), (2, None), (3, [(8.2, -23.6, 17.3), (4.1, -2.9, 0.5),
                                                                     (1.875, -1.25, 0.375)]),
                                          (4, [(1.5, -0.5, 0.0)] * 4), (1, [(0.0, 0.0, 0.0)]), (7, None)])
@pytest.mark.parametrize("r", [90, 150])
def test_orthogonalize_schedules(S, steps, coeffs, r):
    G = gradient(13, 2, r, 200)
    cfg = S.hpo.make_muon_cfg(ns_steps=steps, ns_coeffs=coeffs)
    check_ortho(ortho(S, G.to(DEV), cfg=cfg), G.double(), steps, coeffs, tag=f"{steps} steps")


def test_orthogonalize_scale_of_the_input_does_not_matter(S):
    """Powers of two of the gradient, far beyond fp16's range, give the same bits (eps 0)."""
    G = gradient(17, 1, 70, 140)
    cfg = S.hpo.make_muon_cfg(ns_eps=0.0)
    base = ortho(S, G.to(DEV), cfg=cfg)
    for e in (-80, -30, 30, 80):
        assert torch.equal(su.bits(ortho(S, (G * 2.0 ** e).to(DEV), cfg=cfg)), su.bits(base)), e


@pytest.mark.parametrize("r,c", [(40, 60), (140, 150)])
def test_orthogonalize_zero_and_non_finite(S, r, c):
    G = gradient(19, 4, r, c)
    G[0] = 0.0
    G[1, 3, 5] = math.nan
    G[2, 7, 1] = INF
    for eps in (1e-7, 0.0):
        out = ortho(S, G.to(DEV), cfg=S.hpo.make_muon_cfg(ns_eps=eps)).cpu()
        assert bool((out[0] == 0).all())
        assert bool(out[1].isnan().all()) and bool(out[2].isnan().all())
        check_ortho(out[3:], G[3:].double(), eps=eps, tag="beside NaN")


def test_orthogonalize_skips_behind_found_inf(S):
    G, M = gradient(21, 2, 40, 60).to(DEV), gradient(22, 2, 40, 60).to(DEV)
    for n in (60, 300):
        G, M = gradient(21, 2, 40, n).to(DEV), gradient(22, 2, 40, n).to(DEV)
        flag = torch.ones(1, dtype=torch.int32, device=DEV)
        M0, out = M.clone(), torch.full(G.shape, 9.0, dtype=torch.bfloat16, device=DEV)
        ortho(S, G, M, out, d_found_inf=flag)
        assert torch.equal(M, M0) and bool((out == 9.0).all())
        flag.zero_()
        ortho(S, G, M, out, d_found_inf=flag)
        assert not torch.equal(M, M0) and not bool((out == 9.0).any())


@pytest.mark.parametrize("r,c", [(96, 512), (300, 280)])
def test_orthogonalize_same_bits_again_on_a_stream_and_in_a_graph(S, r, c):
    G = gradient(23, 3, r, c).to(DEV)
    base = su.bits(ortho(S, G))
    n = S.hpo_orthogonalize_workspace(G)
    side = torch.cuda.Stream()
    out, ws = torch.zeros(G.shape, dtype=torch.bfloat16, device=DEV), workspace(n, 0x5A)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ortho(S, G, out=out, ws=ws)
    side.synchronize()
    assert torch.equal(su.bits(out), base)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ortho(S, G, out=out, ws=ws)
    for k in range(4):
        G.copy_(gradient(23 + 10 * k, 3, r, c))
        out.zero_()
        ws.fill_(k)
        g.replay()
        got = su.bits(out)
        torch.cuda.synchronize()
        assert torch.equal(got, su.bits(ortho(S, G))), k


# --------------------------------------------------------------------------
# hpo_rms_update
# --------------------------------------------------------------------------
CFG = dict(lr=0.02, weight_decay=0.1, beta2=0.95, eps=1e-8, target_rms=0.2)


def rms_inputs(seed, b, r, c, odt):
    g = gen(seed)
    O = (torch.randn(b, r, c, generator=g) * torch.exp(torch.randn(b, r, 1, generator=g)) / math.sqrt(max(r, c))).to(odt)
    return O, 0.02 * torch.randn(b, r, c, generator=g), torch.rand(b, r, generator=g) / max(r, c)


def make_param(kind, shape, layout="dense"):
    if kind == "bf16":
        return Guarded(shape, torch.bfloat16, layout), None
    if kind == "mx8":
        b, r, c = shape
        return Guarded(shape, torch.float8_e4m3fn, layout), torch.full((b, r, -(-c // 32)), 77, dtype=torch.uint8,
                                                                       device=DEV)
    return None, None


def check_rms(W, v, W0, O, v0, cfg, tag):
    cols = O.shape[-1]
    w, vv, u = su.rms_reference(O, W0, v0, cfg["lr"], cfg["weight_decay"], cfg["beta2"], cfg["eps"],
                                cfg["target_rms"])
    L = su.rms_terms(cols)
    if v is not None:
        assert bool(((v.double().cpu() - vv).abs() <= (L + 2) * su.HALF32 * vv.abs()).all()), tag
    # u: its coefficient carries the means' errors twice over (v and N) and three roundings; W two
    tol = u.abs() * (2 * L + 8) * su.HALF32 + 3 * su.HALF32 * (W0.double().abs() + w.abs())
    d = (W.double().cpu() - w).abs()
    print(f"[rms] {tag}: max error / allowed {float((d / tol.clamp(min=1e-300)).max()):.3f}", flush=True)
    assert bool((d <= tol).all()), tag


@pytest.mark.parametrize("b,r,c", [(1, 1, 1), (2, 3, 2), (1, 129, 257), (2, 64, 256), (3, 40, 1000), (2, 7, 2049),
                                   (1, 5, 9000), (1, 1500, 96), (4, 33, 31), (2, 1030, 33)])
@pytest.mark.parametrize("kind", ["none", "bf16", "mx8"])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
def test_rms_update(S, b, r, c, kind, odt):
    O, W0, v0 = rms_inputs(r * 7 + c, b, r, c, odt)
    W, v = W0.to(DEV), v0.to(DEV)
    p, s = make_param(kind, (b, r, c))
    ws = workspace(S.hpo_rms_update_workspace(W))
    S.hpo_rms_update(O.to(DEV), W, v, S.make_rms_cfg(**CFG), ws, param=p and p.view, scales=s)
    check_rms(W, v, W0, O, v0, CFG, f"{b}x{r}x{c} {kind} {odt}")
    if p:
        su.check_weight(W, p.view, s)


@pytest.mark.parametrize("layout", ["padded", "offset", "rows"])
@pytest.mark.parametrize("kind", ["bf16", "mx8"])
@pytest.mark.parametrize("c", [64, 70])
def test_rms_update_strides(S, layout, kind, c):
    b, r = 3, 50
    O, W0, v0 = rms_inputs(3, b, r, c, torch.bfloat16)
    o, w = Guarded((b, r, c), torch.bfloat16, layout, O), Guarded((b, r, c), torch.float32, layout, W0)
    p, s = make_param(kind, (b, r, c), layout)
    v = v0.to(DEV)
    S.hpo_rms_update(o.view, w.view, v, S.make_rms_cfg(**CFG), workspace(S.hpo_rms_update_workspace(w.view)),
                     param=p.view, scales=s)
    check_rms(w.view, v, W0, O, v0, CFG, layout)
    su.check_weight(w.view, p.view, s)
    o.unchanged()
    w.untouched_outside()
    p.untouched_outside()


def test_rms_update_plain_norm_without_v(S):
    """beta2 = 0 is the root-mean-square norm of each row; v is optional, and written when given."""
    O, W0, v0 = rms_inputs(4, 2, 30, 500, torch.float32)
    cfg = dict(CFG, beta2=0.0, eps=1e-3, weight_decay=0.0)
    W1, W2, v = W0.to(DEV), W0.to(DEV), v0.to(DEV)
    ws = workspace(S.hpo_rms_update_workspace(W1))
    S.hpo_rms_update(O.to(DEV), W1, None, S.make_rms_cfg(**cfg), ws)
    S.hpo_rms_update(O.to(DEV), W2, v, S.make_rms_cfg(**cfg), ws)
    assert torch.equal(W1, W2)
    check_rms(W1, v, W0, O, v0, cfg, "plain")


@pytest.mark.parametrize("rows", [20, 1100])
def test_rms_update_empty_rows_and_matrices(S, rows):
    """A zero row is left out; a zero matrix only decays, eps = 0 included."""
    O, W0, v0 = rms_inputs(5, 2, rows, 40, torch.float32)
    O[0] = 0.0
    O[1, 3] = 0.0
    v0[0] = 0.0
    v0[1, 3] = 0.0
    for eps in (0.0, 1e-8):
        cfg = dict(CFG, eps=eps)
        W, v = W0.to(DEV), v0.to(DEV)
        S.hpo_rms_update(O.to(DEV), W, v, S.make_rms_cfg(**cfg), workspace(S.hpo_rms_update_workspace(W)))
        check_rms(W, v, W0, O, v0, cfg, f"eps {eps}")
        keep = W0 * torch.tensor(1 - 0.02 * 0.1, dtype=torch.float32)
        assert torch.equal(W[0].cpu(), keep[0]) and torch.equal(W[1, 3].cpu(), keep[1, 3])


def test_mx8_edges(S):
    """Blocks at the ends of the scale's range, of zeros, with inf or NaN, values that saturate and tie."""
    rows = [torch.zeros(70), torch.full((70,), 1e-45), torch.full((70,), 3.3e38), torch.full((70,), 2.0 ** -118),
            torch.full((70,), 2.0 ** -119 * 1.5), torch.linspace(-1, 1, 70), torch.linspace(-1.999, 1.999, 70),
            torch.tensor([(1 + k / 16) for k in range(70)]), torch.tensor([2.0 ** -(k % 20) for k in range(70)])]
    nan = torch.ones(70)
    nan[40] = math.nan
    inf = torch.ones(70)
    inf[69] = -INF
    W0 = torch.stack(rows + [nan, inf]).unsqueeze(0)
    W = W0.to(DEV)
    p, s = make_param("mx8", tuple(W.shape))
    O = torch.zeros_like(W)
    S.hpo_rms_update(O, W, None, S.make_rms_cfg(0.0, beta2=0.0), workspace(S.hpo_rms_update_workspace(W)),
                     param=p.view, scales=s)
    assert torch.equal(su.bits(W), su.bits(W0))
    su.check_weight(W, p.view, s)


def test_rms_update_skip_stream_and_graph(S):
    O, W0, v0 = rms_inputs(6, 2, 100, 300, torch.bfloat16)
    O, flag = O.to(DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    cfg = S.make_rms_cfg(**CFG)

    def fresh():
        return W0.to(DEV), v0.to(DEV), make_param("mx8", (2, 100, 300))

    def call(W, v, p, s, ws):
        S.hpo_rms_update(O, W, v, cfg, ws, param=p.view, scales=s, d_found_inf=flag)

    W, v, (p, s) = fresh()
    ws = workspace(S.hpo_rms_update_workspace(W))
    call(W, v, p, s, ws)
    assert torch.equal(W.cpu(), W0) and torch.equal(v.cpu(), v0) and bool((s == 77).all())
    p.unchanged()
    flag.zero_()
    states = []
    for k in range(3):
        call(W, v, p, s, ws)
        states.append([su.bits(t) for t in (W, v, p.view, s)])
    W, v, (p, s) = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call(W, v, p, s, ws)
    for k in range(3):
        g.replay()
        torch.cuda.synchronize()
        ws.fill_(k)
        for got, want in zip((W, v, p.view, s), states[k]):
            assert torch.equal(su.bits(got), want), k


# --------------------------------------------------------------------------
# hpo_qk_max_logits
# --------------------------------------------------------------------------
def check_logits(got, q, k, scale, causal, window, dim, tag):
    best, size = su.logits_reference(q, k, scale, causal, window)
    got = got.double().cpu()
    assert torch.equal(got.isnan(), best.isnan()), (tag, got, best)
    fin = torch.isfinite(best)
    assert torch.equal(got[~fin & ~best.isnan()], best[~fin & ~best.isnan()]), (tag, got, best)
    d, tol = (got - best).abs()[fin], su.logits_tolerance(dim, size)[fin]
    print(f"[logits] {tag}: max error / allowed {float((d / tol.clamp(min=1e-300)).max()) if d.numel() else 0:.3f}",
          flush=True)
    assert bool((d <= tol).all()), (tag, got, best)


@pytest.mark.parametrize("sq,sk", [(1, 1), (1, 700), (64, 64), (65, 127), (300, 300), (257, 515), (515, 130), (128, 1)])
@pytest.mark.parametrize("causal,window", [(False, -1), (True, -1), (True, 0), (True, 100)])
def test_qk_max_masks(S, sq, sk, causal, window):
    """Lengths on both sides of a tile; more queries than keys leave rows with nothing to see."""
    g = gen(sq * 7 + sk)
    q = torch.randn(2, sq, 4, 64, generator=g).bfloat16()
    k = torch.randn(2, sk, 2, 64, generator=g).bfloat16()
    out = torch.empty(4, device=DEV)
    S.hpo_qk_max_logits(q.to(DEV), k.to(DEV), out, 0.125, causal=causal, window=window)
    check_logits(out, q, k, 0.125, causal, window, 64, f"{sq}/{sk} {causal} {window}")


@pytest.mark.parametrize("dim", [1, 7, 8, 40, 57, 64, 72, 96, 128, 130, 192, 200, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_qk_max_dims(S, dim, dtype):
    g = gen(dim)
    q = torch.randn(1, 150, 6, dim, generator=g).to(dtype)
    k = torch.randn(1, 201, 3, dim, generator=g).to(dtype)
    out = torch.empty(6, device=DEV)
    S.hpo_qk_max_logits(q.to(DEV), k.to(DEV), out, 0.3, causal=True)
    check_logits(out, q, k, 0.3, True, -1, dim, f"dim {dim} {dtype}")


def test_qk_max_every_place_counts_once(S):
    """A single large pair at each of many places is found exactly when it is seen."""
    n, dim = 200, 128
    for i, j in [(0, 0), (63, 63), (64, 0), (199, 199), (130, 131), (0, 199), (199, 0), (100, 36)]:
        q, k = torch.zeros(1, n, 1, dim), torch.zeros(1, n, 1, dim)
        q[0, i, 0, 5], k[0, j, 0, 5] = 3.0, 2.0
        out = torch.empty(1, device=DEV)
        for causal, window in ((False, -1), (True, -1), (True, 63)):
            S.hpo_qk_max_logits(q.bfloat16().to(DEV), k.bfloat16().to(DEV), out, 1.0, causal=causal, window=window)
            seen = not causal or (j <= i and (window < 0 or j >= i - window))
            assert out.item() == (6.0 if seen else 0.0), (i, j, causal, window)


@pytest.mark.parametrize("layout", ["bhsd", "fused", "odd"])
def test_qk_max_strides(S, layout):
    g = gen(31)
    b, n, h, d = 2, 190, 4, 64
    if layout == "bhsd":
        q, k = (torch.randn(b, h, n, d, generator=g).bfloat16().transpose(1, 2) for _ in range(2))
        qd, kd = q.transpose(1, 2).contiguous().to(DEV).transpose(1, 2), k.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
    else:
        w = 3 * d if layout == "fused" else 3 * d + 1
        buf = torch.randn(b, n, h, w, generator=g).bfloat16()
        dev = buf.to(DEV)
        q, k, qd, kd = buf[..., :d], buf[..., d:2 * d], dev[..., :d], dev[..., d:2 * d]
        assert qd.stride(-2) == w
    out = torch.empty(h, device=DEV)
    S.hpo_qk_max_logits(qd, kd, out, 0.125)
    check_logits(out, q, k, 0.125, True, -1, d, layout)


def test_qk_max_lengths_and_masked_values(S):
    """Values behind a sequence's end or behind the mask never count, NaN and inf among them; a seen NaN wins."""
    g = gen(37)
    b, n, h, d = 3, 140, 2, 64
    q, k = (torch.randn(b, n, h, d, generator=g).bfloat16() for _ in range(2))
    lq, lk = torch.tensor([140, 0, 77], dtype=torch.int32), torch.tensor([100, 50, 33], dtype=torch.int32)
    for z in range(b):
        q[z, lq[z]:], k[z, lk[z]:] = math.nan, INF
    out = torch.empty(h, device=DEV)
    call = lambda **kw: S.hpo_qk_max_logits(q.to(DEV), k.to(DEV), out, 0.125, seqlens_q=lq.to(DEV),
                                            seqlens_k=lk.to(DEV), **kw)
    cut = lambda t, n: [t[z, :n[z]] for z in range(b)]
    for causal in (False, True):
        call(causal=causal)
        check_logits(out, cut(q, lq), cut(k, lk), 0.125, causal, -1, d, f"lengths {causal}")
    # the first 40 queries of sequence 0 (140 queries, 100 keys) see nothing
    q[0, :40] = math.nan
    call(causal=True)
    check_logits(out, cut(q, lq), cut(k, lk), 0.125, True, -1, d, "rows that see nothing")
    q[0, 40, 1] = math.nan
    call(causal=True)
    assert not out[0].isnan() and bool(out[1].isnan())
    # lengths beyond the buffer, or negative, are cut
    S.hpo_qk_max_logits(q.to(DEV), k.to(DEV), out, 0.125, seqlens_q=torch.full((3,), -5, dtype=torch.int32, device=DEV),
                        seqlens_k=lk.to(DEV))
    assert bool((out == -INF).all())


def test_qk_max_infinities(S):
    q, k = torch.zeros(1, 3, 2, 64), torch.zeros(1, 3, 2, 64)
    q[..., 0], k[..., 0] = 1.0, -1.0
    k[0, 1, 0, 0] = -INF
    out = torch.empty(2, device=DEV)
    S.hpo_qk_max_logits(q.bfloat16().to(DEV), k.bfloat16().to(DEV), out, 2.0, causal=False)
    assert out.tolist() == [-2.0, -2.0]
    k[0, 2, 1, 0] = INF
    S.hpo_qk_max_logits(q.bfloat16().to(DEV), k.bfloat16().to(DEV), out, 2.0, causal=False)
    assert out.tolist() == [-2.0, INF]
    k[..., 0] = -INF
    S.hpo_qk_max_logits(q.bfloat16().to(DEV), k.bfloat16().to(DEV), out, 2.0, causal=False)
    assert out.tolist() == [-INF, -INF]


@pytest.mark.parametrize("hint", [None, 1, 64])
def test_qk_max_packed(S, hint):
    """Packed sequences, empty ones among them; too small a length hint changes nothing."""
    g = gen(41)
    lq, lk = [300, 0, 1, 65, 700], [300, 9, 1, 200, 650]
    q = torch.randn(sum(lq), 4, 96, generator=g).half()
    k = torch.randn(sum(lk), 2, 96, generator=g).half()
    cu = lambda n: torch.tensor([0] + n).cumsum(0).to(torch.int32)
    out = torch.empty(4, device=DEV)
    cq, ck = cu(lq), cu(lk)
    S.hpo_qk_max_logits(q.to(DEV), k.to(DEV), out, 0.1, causal=True, window=150, cu_seqlens_q=cq.to(DEV),
                        cu_seqlens_k=ck.to(DEV), max_seqlen_q=hint or 700, max_seqlen_k=hint or 650)
    check_logits(out, list(q.split(lq)), list(k.split(lk)), 0.1, True, 150, 96, f"packed {hint}")
    # offsets beyond the tokens that are there are cut
    cq[-1], ck[-1] = 10 ** 6, 2 ** 31 - 1
    S.hpo_qk_max_logits(q.to(DEV), k.to(DEV), out, 0.1, causal=True, window=150, cu_seqlens_q=cq.to(DEV),
                        cu_seqlens_k=ck.to(DEV), max_seqlen_q=700, max_seqlen_k=700)
    check_logits(out, list(q.split(lq)), list(k.split(lk)), 0.1, True, 150, 96, "cut offsets")


def test_qk_max_accumulates_over_micro_batches_in_any_order(S):
    g = gen(43)
    parts = [(torch.randn(1, n, 3, 64, generator=g).bfloat16().to(DEV), torch.randn(1, n, 3, 64, generator=g).bfloat16().to(DEV))
             for n in (10, 500, 129)]
    alone = []
    for q, k in parts:
        o = torch.full((3,), 123.0, device=DEV)
        S.hpo_qk_max_logits(q, k, o, 0.125)
        alone.append(o)
    want = torch.stack(alone).amax(0)
    for order in ([0, 1, 2], [2, 1, 0], [1, 0, 2]):
        o = torch.full((3,), -INF, device=DEV)
        for i in order:
            S.hpo_qk_max_logits(*parts[i], o, 0.125, accumulate=True)
        assert torch.equal(o, want)
    for start, stays in ((1e9, True), (-1e9, False), (math.nan, True), (0.0, False), (-0.0, False)):
        o = torch.full((3,), start, device=DEV)
        S.hpo_qk_max_logits(*parts[1], o, 0.125, accumulate=True)
        assert torch.equal(o.nan_to_num(7.0), torch.full((3,), start, device=DEV).nan_to_num(7.0) if stays else alone[1])
    o = torch.full((3,), 5.0, device=DEV)
    S.hpo_qk_max_logits(parts[0][0][:, :0], parts[0][1], o, 0.125)
    assert bool((o == -INF).all())


def test_qk_max_stream_and_graph(S):
    g = gen(47)
    q, k = (torch.randn(2, 400, 4, 128, generator=g).bfloat16().to(DEV) for _ in range(2))
    out = torch.empty(4, device=DEV)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        S.hpo_qk_max_logits(q, k, out, 0.1)
    for s in range(4):
        q.copy_(torch.randn(2, 400, 4, 128, generator=gen(50 + s)))
        gr.replay()
        got = out.clone()
        torch.cuda.synchronize()
        S.hpo_qk_max_logits(q, k, out, 0.1)
        assert torch.equal(got, out)


# --------------------------------------------------------------------------
# hpo_qk_clip
# --------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["none", "bf16", "mx8"])
@pytest.mark.parametrize("h,hk", [(8, 8), (8, 2), (1, 1)])
@pytest.mark.parametrize("d,c", [(16, 256), (7, 70)])
def test_qk_clip(S, kind, h, hk, d, c):
    g = gen(h * 10 + d)
    smax = torch.linspace(60, 140, h)
    if h == 8:
        smax[1], smax[2], smax[6] = INF, math.nan, -INF
    per = h // hk
    gamma = torch.where(torch.isfinite(smax) & (smax > 100), 100.0 / smax.double(), 1.0)
    group = gamma.view(hk, per).amin(-1)
    specs = [(h, 0.5, True), (hk, 0.5, True), (h, 1.0, False)]
    ws, refs, params = [], [], []
    for heads, power, grouped in specs:
        W0 = torch.randn(heads * d, c, generator=g)
        W = W0.to(DEV)
        p, s = make_param(kind, (heads, d, c))
        if kind == "bf16":
            p.view.copy_(W0.view(heads, d, c))
        before = (su.bits(p.buf).clone(), s.cpu().clone() if s is not None else None) if p else None
        f = (gamma if heads == h and not grouped else (group.repeat_interleave(per) if heads == h else group)) ** power
        ws.append(S.ClipWeight(W, heads, power, param=p.view if p and kind != "bf16" else (p.view.view(heads * d, c) if p else None),
                               scales=s, per_group=grouped))
        refs.append((W0.view(heads, d, c), f))
        params.append((p, s, before))
    S.hpo_qk_clip(smax.to(DEV), hk, 100.0, ws)
    for w, (W0, f), (p, s, before) in zip(ws, refs, params):
        got = w.master.view(W0.shape).double().cpu()
        want = W0.double() * f[:, None, None]
        # f is rounded once (or off by one step more, from pow), the product once
        assert bool(((got - want).abs() <= 4 * su.HALF32 * want.abs()).all())
        same = f == 1.0
        assert torch.equal(got[same], W0[same].double())
        if p:
            su.check_weight(w.master.view(W0.shape)[~same], p.view[~same], s[~same] if s is not None else None)
            assert torch.equal(su.bits(p.view)[same], before[0].view(p.view.shape)[same])
            if s is not None:
                assert torch.equal(s.cpu()[same], before[1][same])


def test_qk_clip_fused_projection_views_and_skip(S):
    """Query and key rows of a fused projection, interleaved by group, are views of one buffer; value rows stay."""
    g = gen(61)
    hk, per, d, c = 2, 2, 8, 64
    W0 = torch.randn(hk, (per + 2) * d, c, generator=g)
    W, flag = W0.to(DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    smax = torch.tensor([50.0, 400.0, 20.0, 30.0], device=DEV)
    parts = [S.ClipWeight(W[:, i * d:(i + 1) * d], hk, 0.5) for i in (0, 1, per)]
    S.hpo_qk_clip(smax, hk, 100.0, parts, d_found_inf=flag)
    assert torch.equal(W.cpu(), W0)
    flag.zero_()
    S.hpo_qk_clip(smax, hk, 100.0, parts, d_found_inf=flag)
    want = W0.clone()
    want[0, :(per + 1) * d] *= 0.5      # group 0: gamma 1/4, power 1/2
    assert torch.equal(W.cpu(), want)


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------
def test_a_muon_clip_step(S):
    """Gradient -> orthogonalised update -> row-normalised update of master and weight -> logits of
    the new weights -> clip, twice, captured and replayed against the eager run."""
    g = gen(71)
    heads, hk, d, c, n = 4, 2, 64, 256, 200
    x = torch.randn(1, n, c, generator=g).bfloat16().to(DEV)
    base = {"q": (heads, 30.0), "k": (hk, 30.0)}

    def fresh():
        st = {}
        for name, (h, size) in base.items():
            w = (torch.randn(h, d, c, generator=gen(72 + h)) * size / math.sqrt(c)).to(DEV)
            st[name] = dict(W=w, p=w.bfloat16(), M=torch.zeros_like(w), v=torch.zeros(h, d, device=DEV),
                            O=torch.zeros(h, d, c, dtype=torch.bfloat16, device=DEV),
                            G=gradient(73 + h, h, d, c).to(DEV), h=h)
            st[name]["ws"] = workspace(S.hpo_orthogonalize_workspace(w))
            st[name]["ws2"] = workspace(S.hpo_rms_update_workspace(w))
        st["smax"] = torch.empty(heads, device=DEV)
        return st

    mcfg, rcfg = S.hpo.make_muon_cfg(), S.make_rms_cfg(**CFG)

    def step(st):
        for name in base:
            t = st[name]
            S.hpo_orthogonalize(t["G"], t["O"], mcfg, t["ws"], momentum=t["M"])
            S.hpo_rms_update(t["O"], t["W"], t["v"], rcfg, t["ws2"], param=t["p"])
        q, k = ((x.float() @ st[m]["p"].float().flatten(0, 1).t()).bfloat16().view(1, n, -1, d) for m in ("q", "k"))
        S.hpo_qk_max_logits(q, k, st["smax"], 1 / 8, causal=True)
        st["q_act"], st["k_act"] = q, k
        S.hpo_qk_clip(st["smax"], hk, 100.0, [S.ClipWeight(st[m]["W"], st[m]["h"], 0.5, param=st[m]["p"]) for m in base])

    a = fresh()
    before = {m: a[m]["W"].clone() for m in base}
    M0 = {m: a[m]["M"].clone() for m in base}
    step(a)
    # each stage against its reference, from what the stage was given
    for m in base:
        t = a[m]
        Mn = 0.95 * M0[m].cpu() + t["G"].cpu()
        check_ortho(t["O"], (t["G"].cpu() + torch.tensor(0.95) * Mn).double(), tag=m)
        check_weight_after = t["W"].cpu()
        su.check_weight(t["W"], t["p"])
        w, _, u = su.rms_reference(t["O"].cpu(), before[m].cpu(), torch.zeros(t["h"], d), **{"lr": 0.02, "wd": 0.1,
                                   "beta2": 0.95, "eps": 1e-8, "target": 0.2})
        smax = a["smax"].double().cpu()
        gam = torch.where(smax > 100, 100 / smax, 1.0).view(hk, -1).amin(-1)
        f = gam.repeat_interleave(t["h"] // hk).sqrt()
        assert bool(((check_weight_after.double() - w * f[:, None, None]).abs() <= 1e-5 * (w.abs() + u.abs()) + 1e-9).all())
    check_logits(a["smax"], a["q_act"].cpu(), a["k_act"].cpu(), 1 / 8, True, -1, d, "chain")
    assert bool((a["smax"] > 100).any()), "the case must clip"
    step(a)
    b = fresh()
    step(b)          # warm-up outside of the capture
    c2 = fresh()
    for m in base:
        for key in ("W", "p", "M", "v", "G"):
            b[m][key].copy_(c2[m][key])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step(b)
    gr.replay()
    torch.cuda.synchronize()
    gr.replay()
    torch.cuda.synchronize()
    for m in base:
        for key in ("W", "p", "M", "v", "O"):
            assert torch.equal(su.bits(a[m][key]), su.bits(b[m][key])), (m, key)


def test_stack_muon_is_its_two_calls(S):
    """StackMuon steps, skips and clips as the calls do, bit for bit, with an 8-bit weight."""
    from mixed_precision_optimizer_amd import StackMuon
    b, r, c = 4, 24, 160
    W0 = 0.02 * torch.randn(b, r, c, generator=gen(81))
    W1, W2 = W0.to(DEV), W0.to(DEV)
    p1, s1 = make_param("mx8", (b, r, c))
    p2, s2 = make_param("mx8", (b, r, c))
    opt = StackMuon(W1, p1.view, s1, lr=0.02, weight_decay=0.1)
    cfg, rcfg = S.hpo.make_muon_cfg(), S.make_rms_cfg(0.02, 0.1)
    M, v = torch.zeros_like(W2), torch.zeros(b, r, device=DEV)
    flag, norm = torch.zeros(1, dtype=torch.int32, device=DEV), torch.tensor([4.0], device=DEV)
    for k in range(3):
        G = gradient(82 + k, b, r, c).bfloat16().to(DEV)
        flag.fill_(k == 1)
        opt.step(G, inv_scale=0.25, max_norm=1.0, d_norm=norm, d_found_inf=flag)
        if k != 1:
            O = ortho(S, G, M, cfg=cfg, inv_scale=0.25, max_norm=1.0, d_norm=norm)
            S.hpo_rms_update(O, W2, v, rcfg, workspace(S.hpo_rms_update_workspace(W2)), param=p2.view, scales=s2)
        for x, y in ((W1, W2), (opt.momentum, M), (opt.v, v), (p1.view, p2.view), (s1, s2)):
            assert torch.equal(su.bits(x), su.bits(y)), k
    S.hpo_qk_clip(torch.tensor([90.0, 400.0, 10.0, 100.0], device=DEV), b, 100.0, [opt.clip_weight()])
    f = torch.tensor([1.0, 0.5, 1.0, 1.0], device=DEV)[:, None, None]
    assert torch.equal(W1, W2 * f)
    su.check_weight(W1, p1.view, s1)


def test_calls_on_two_streams_at_once(S):
    """Two stacks worked on by two streams, a workspace each, give what they give alone."""
    def job(seed, n):
        W = (0.02 * torch.randn(3, 40, n, generator=gen(seed))).to(DEV)
        G = gradient(seed + 1, 3, 40, n).to(DEV)
        return dict(W=W, G=G, O=torch.zeros(3, 40, n, dtype=torch.bfloat16, device=DEV),
                    v=torch.zeros(3, 40, device=DEV), ws=workspace(S.hpo_orthogonalize_workspace(G)),
                    ws2=workspace(S.hpo_rms_update_workspace(W)))

    def work(j, times):
        for _ in range(times):
            S.hpo_orthogonalize(j["G"], j["O"], S.hpo.make_muon_cfg(), j["ws"])
            S.hpo_rms_update(j["O"], j["W"], j["v"], S.make_rms_cfg(0.02), j["ws2"])

    alone, both = [job(91, 700), job(93, 300)], [job(91, 700), job(93, 300)]
    for j in alone:
        work(j, 5)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, j in zip(streams, both):
        with torch.cuda.stream(st):
            work(j, 5)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(su.bits(a["W"]), su.bits(b["W"])) and torch.equal(su.bits(a["O"]), su.bits(b["O"]))


def test_offsets_beyond_32_bits(S):
    """Matrices, heads and rows more than 2^31 elements into their buffer."""
    far = (1 << 31) + 64
    buf = torch.zeros(far + 4096, dtype=torch.float32, device=DEV)
    W = buf.as_strided((2, 8, 32), (far, 32, 1))
    W0 = 0.02 * torch.randn(2, 8, 32, generator=gen(95))
    W.copy_(W0)
    O, v = torch.randn(2, 8, 32, generator=gen(96)), torch.zeros(2, 8)
    vd = v.to(DEV)
    S.hpo_rms_update(O.to(DEV), W, vd, S.make_rms_cfg(**CFG), workspace(S.hpo_rms_update_workspace(W)))
    check_rms(W, vd, W0, O, v, CFG, "far")
    g = gradient(97, 2, 8, 32)
    W.copy_(g)
    check_ortho(ortho(S, W), g.double(), tag="far")
    big = gradient(98, 2, 140, 150)   # short side over the thin form's
    far_rows = buf.as_strided((2, 140, 150), (150, (far - 400) // 140, 1))
    far_rows.copy_(big)
    check_ortho(ortho(S, far_rows), big.double(), tag="far rows")
    W.copy_(W0)
    S.hpo_qk_clip(torch.tensor([50.0, 400.0], device=DEV), 2, 100.0, [S.ClipWeight(W, 2, 0.5)])
    assert torch.equal(W.cpu(), W0 * torch.tensor([1.0, 0.5])[:, None, None])
    del buf, W, far_rows
    half = torch.zeros(far + 4096, dtype=torch.bfloat16, device=DEV)
    q, k = (torch.randn(2, 40, 1, 64, generator=gen(n)).bfloat16() for n in (99, 100))
    qd, kd = half.as_strided((2, 40, 1, 64), (far, 64, 64, 1)), torch.zeros(2, 40, 1, 64, dtype=torch.bfloat16, device=DEV)
    qd.copy_(q)
    kd.copy_(k)
    out = torch.empty(1, device=DEV)
    for causal in (False, True):
        S.hpo_qk_max_logits(qd, kd, out, 0.125, causal=causal)
        check_logits(out, q, k, 0.125, causal, -1, 64, "far queries")
        S.hpo_qk_max_logits(kd, qd, out, 0.125, causal=causal)
        check_logits(out, k, q, 0.125, causal, -1, 64, "far keys")


@pytest.mark.parametrize("value", [1.0, -1.0])
def test_qk_max_keeps_a_nan_of_either_sign_when_it_accumulates(S, value):
    """A NaN already in d_max stays one, whatever its sign bit and the sign of the new maxima."""
    q = torch.ones(2, 300, 3, 64, dtype=torch.bfloat16, device=DEV)
    k = value * torch.ones_like(q)
    for pattern in (0x7FC00000, 0xFFC00000 - (1 << 32), 0xFF800001 - (1 << 32)):
        o = torch.full((3,), pattern, dtype=torch.int32, device=DEV).view(torch.float32)
        S.hpo_qk_max_logits(q, k, o, 0.125, causal=False, accumulate=True)
        assert bool(o.isnan().all()), hex(pattern)


def test_stack_muon_of_one_matrix_clips_as_one_head(S):
    from mixed_precision_optimizer_amd import StackMuon
    W = torch.randn(6, 40, generator=gen(91)).to(DEV)
    before = W.clone()
    opt = StackMuon(W, lr=0.02)
    S.hpo_qk_clip(torch.tensor([400.0], device=DEV), 1, 100.0, [opt.clip_weight()])
    assert torch.equal(W, before * 0.5)
