"""Stack operators on the GPU at sizes that take the forms for much work: runs of pieces, accesses around the caches,
folded sums, stacks in slices, several column tiles a workgroup."""
import math

import pytest

torch = pytest.importorskip("torch")

import stack_util as su  # noqa: E402
from test_gpu_stack import CFG, DEV, Guarded, S, check_rms, gen, workspace  # noqa: E402, F401

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
