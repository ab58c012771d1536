"""Stack operators on the GPU at sizes that take the forms for much work: runs of pieces, accesses around the caches,
folded sums, stacks in slices, several column tiles a workgroup."""
import math

import pytest

torch = pytest.importorskip("torch")

import stack_util as su  # noqa: E402
from test_gpu_stack import CFG, DEV, Guarded, S, check_rms, gen, ortho, workspace  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def rand(seed, *shape, scale=1.0):
    return scale * torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV)


# --------------------------------------------------------------------------
# hpo_rms_update
# --------------------------------------------------------------------------
@pytest.mark.parametrize("b,r,c,layout", [
    (3, 1100, 2053, "padded"),    # runs of pieces that cross row ends, through the caches
    (1, 4200, 1100, "dense"),     # the same, N from a fold
    (1, 5000, 4099, "padded"),    # around the caches (over 64 MiB), folded, odd row stride
    (2, 450, 24001, "rows"),      # a workgroup per long row, around the caches, no fold
    (1, 1500, 14339, "offset"),   # a workgroup per long row and a fold
    (1, 4200, 33, "padded"),      # little work, folded
])
@pytest.mark.parametrize("kind,odt", [("none", torch.float32), ("bf16", torch.bfloat16), ("mx8", torch.bfloat16)])
def test_rms_update_large(S, b, r, c, layout, kind, odt):
    O0 = (rand(r, b, r, c) * torch.exp(rand(r + 1, b, r, 1)) / math.sqrt(max(r, c))).to(odt)
    W0, v0 = rand(r + 2, b, r, c, scale=0.02), rand(r + 3, b, r).abs() / max(r, c)
    O, W = Guarded((b, r, c), odt, layout, O0), Guarded((b, r, c), torch.float32, layout, W0)
    p = s = None
    if kind != "none":
        p = Guarded((b, r, c), torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn, layout)
        s = torch.full((b, r, -(-c // 32)), 77, dtype=torch.uint8, device=DEV) if kind == "mx8" else None
    v = v0.clone()
    S.hpo_rms_update(O.view, W.view, v, S.make_rms_cfg(**CFG), workspace(S.hpo_rms_update_workspace(W.view)),
                     param=p and p.view, scales=s)
    check_rms(W.view, v, W0.cpu(), O0.cpu(), v0.cpu(), CFG, f"{b}x{r}x{c} {kind}")
    if p:
        su.check_weight(W.view, p.view, s)
        p.untouched_outside()
    O.unchanged()
    W.untouched_outside()


# --------------------------------------------------------------------------
# hpo_qk_clip
# --------------------------------------------------------------------------
@pytest.mark.parametrize("h,hk,d,c", [(48, 24, 96, 4099),   # over 64 MiB: around the caches; runs of four
                                      (40, 8, 48, 4099)])   # through them; runs of two
@pytest.mark.parametrize("kind", ["none", "bf16", "mx8"])
def test_qk_clip_large(S, h, hk, d, c, kind):
    smax = 60.0 + 100.0 * torch.rand(h, generator=gen(h))
    smax[:h // hk] = 50.0          # one group stays
    per = h // hk
    gamma = torch.where(smax > 100, 100.0 / smax.double(), 1.0).view(hk, per).amin(-1)
    jobs = []
    for heads, f in ((h, gamma.repeat_interleave(per)), (hk, gamma)):
        W0 = rand(heads, heads, d, c, scale=0.02)
        W = Guarded((heads, d, c), torch.float32, "padded", W0)
        p = s = None
        if kind != "none":
            p = Guarded((heads, d, c), torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn, "padded")
            s = torch.full((heads, d, -(-c // 32)), 77, dtype=torch.uint8, device=DEV) if kind == "mx8" else None
        before = None if p is None else su.bits(p.view).clone()
        jobs.append((W0.cpu(), W, p, s, f.sqrt(), S.ClipWeight(W.view, heads, 0.5, p and p.view, s), before))
    S.hpo_qk_clip(smax.to(DEV), hk, 100.0, [j[5] for j in jobs])
    for W0, W, p, s, f, _, before in jobs:
        got, want = W.view.double().cpu(), W0.double() * f[:, None, None]
        assert bool(((got - want).abs() <= 4 * su.HALF32 * want.abs()).all())
        same = f == 1.0
        assert bool(same.any()) and not bool(same.all())
        assert torch.equal(su.bits(W.view)[same], su.bits(W0)[same])
        W.untouched_outside()
        if p:
            su.check_weight(W.view.cpu()[~same], p.view.view(torch.uint8 if kind == "mx8" else torch.int16).cpu()[~same].view(
                p.view.dtype), s.cpu()[~same] if s is not None else None)
            assert torch.equal(su.bits(p.view)[same], before[same])
            assert s is None or bool((s.cpu()[same] == 77).all())
            p.untouched_outside()


# --------------------------------------------------------------------------
# hpo_orthogonalize
# --------------------------------------------------------------------------
def check_some(out, gt, places, tag):
    """The matrices at `places` against binary64, on the GPU."""
    for z in places:
        e, tol = su.ns_tolerance(gt(z))
        d = float(torch.linalg.vector_norm(out[z].double() - e) / torch.linalg.vector_norm(e))
        print(f"[ortho] {tag}[{z}] rel {d:.2e} (allowed {tol:.2e})", flush=True)
        assert d <= tol, z


@pytest.mark.parametrize("b,r,c,cut", [(53, 2048, 4096, 27), (40001, 100, 129, 20001), (40001, 129, 100, 20001)])
def test_orthogonalize_stacks_in_slices(S, b, r, c, cut):
    """Stacks whose scratch would pass 4 GiB go through it in slices: matrices on both sides of the cut, the first
    and the last of a shorter last slice."""
    G, M = rand(b, b, r, c, scale=1e-3), rand(b + 1, b, r, c, scale=1e-3)
    n = S.hpo_orthogonalize_workspace(G)
    assert (1 << 31) < n < (1 << 32) + (1 << 20)    # one slice's
    mu = torch.tensor(0.95, device=DEV)
    places = sorted({0, cut // 2, cut - 1, cut, cut + 1, b - 1})
    want = {z: mu * M[z] + G[z] for z in places}
    out = ortho(S, G, M)
    for z in places:
        assert torch.equal(M[z], want[z]), z
    check_some(out, lambda z: (G[z] + mu * M[z]).double(), places, f"{b}x{r}x{c}")


@pytest.mark.parametrize("b,r,c", [(600, 40, 300), (600, 300, 40), (700, 20, 900), (700, 900, 20), (600, 64, 257), (3, 50, 60)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_one_workgroup_a_matrix(S, b, r, c, dtype):
    """A workgroup takes all of a matrix, with momentum, in several column tiles where the stack is large."""
    G0, M0 = rand(b, b, r, c, scale=1e-3).to(dtype), rand(b + 1, b, r, c, scale=1e-2)
    G, M = Guarded((b, r, c), dtype, "padded", G0), Guarded((b, r, c), torch.float32, "padded", M0)
    o = Guarded((b, r, c), torch.bfloat16, "padded")
    ortho(S, G.view, M.view, o.view)
    mu = torch.tensor(0.95, device=DEV)
    M1 = mu * M0 + G0.float()
    assert torch.equal(M.view, M1)
    check_some(o.view, lambda z: (G0[z].float() + mu * M1[z]).double(), sorted({0, 1, b // 2, b - 1}), f"{b}x{r}x{c}")
    G.unchanged()
    M.untouched_outside()
    o.untouched_outside()


@pytest.mark.parametrize("b,r,c", [(2, 140, 300), (1, 1300, 9001), (600, 40, 300), (4, 128, 3000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orthogonalize_skips_in_every_form(S, b, r, c, dtype):
    """Behind a found inf neither form writes: products in parts, whole ones, thin matrices in one launch and in four."""
    G, M = rand(1, b, r, c).to(dtype), rand(2, b, r, c)
    M0, out = M.clone(), torch.full((b, r, c), 9.0, dtype=torch.bfloat16, device=DEV)
    flag = torch.ones(1, dtype=torch.int32, device=DEV)
    ortho(S, G, M, out, d_found_inf=flag)
    assert torch.equal(M, M0) and bool((out == 9.0).all())
    flag.zero_()
    ortho(S, G, M, out, d_found_inf=flag)
    want = ortho(S, G, M0)
    assert torch.equal(M, M0) and torch.equal(out, want) and not bool((out == 9.0).any())


@pytest.mark.parametrize("b,r,c", [(2, 1, 1), (2, 5, 300), (2, 300, 5), (3, 40, 60), (2, 64, 64), (2, 64, 2000), (1, 128, 130)])
def test_orthogonalize_thin_matrices_of_long_schedules(S, b, r, c):
    """Seven steps grow beyond the thin form's range: short sides under one tile in the two-product form."""
    G = rand(r + c, b, r, c, scale=1e-3)
    out = ortho(S, G, cfg=S.hpo.make_muon_cfg(ns_steps=7))
    for z in range(b):
        e, tol = su.ns_tolerance(G[z], 7)
        d = float(torch.linalg.vector_norm(out[z].double() - e) / torch.linalg.vector_norm(e))
        print(f"[ortho] 7 steps {r}x{c}[{z}] rel {d:.2e} (allowed {tol:.2e})", flush=True)
        assert d <= tol


@pytest.mark.parametrize("b,r,c", [(3, 50, 60), (3, 100, 1500), (3, 150, 200), (3, 520, 300), (1, 1300, 9001)])
@pytest.mark.parametrize("form,nesterov", [(0, False), (0, True), (1, False), (1, True)])
@pytest.mark.parametrize("clip", [False, True])
def test_orthogonalize_momentum_and_clip_in_every_form(S, b, r, c, form, nesterov, clip):
    """Unscaling, clip, both momentum rules: one launch, four, whole products, products in parts, tall ones."""
    G, M0 = rand(7, b, r, c, scale=1e-3), rand(8, b, r, c, scale=1e-3)
    cfg = S.hpo.make_muon_cfg(momentum=0.9, nesterov=nesterov, momentum_form=form)
    norm = torch.tensor([3.0 if clip else 1.0], device=DEV)
    M = M0.clone()
    out = ortho(S, G, M, cfg=cfg, inv_scale=0.3, max_norm=1.5, d_norm=norm)
    f = lambda x: torch.tensor(x, dtype=torch.float32, device=DEV)   # noqa: E731
    g = G * f(0.3)
    if clip:
        g = g * f(1.5 / (3.0 + 1e-6))
    mu, omu = f(0.9), f(1.0 - 0.9)
    M1 = mu * M0 + g if form == 0 else mu * M0 + omu * g
    gt = (g + mu * M1 if form == 0 else omu * g + mu * M1) if nesterov else M1
    assert torch.equal(M, M1)
    check_some(out, lambda z: gt[z].double(), sorted({0, b - 1}), f"form {form} {nesterov} {clip} {r}x{c}")
