"""The 8-bit products on operands whose sums fp32 holds exactly in any order: the result is the sum's one rounding, bit
for bit, however the work is cut.  A stage that is lost, counted twice or multiplied at another's scale shows
(test_product_plan.py).  Every case asserts which kernel it reaches."""
import math

import pytest

torch = pytest.importorskip("torch")

import model_util as mu  # noqa: E402
import product_plan as pp  # noqa: E402
import product_sums as ps  # noqa: E402
import stack_util as su  # noqa: E402
from test_gpu_model import BF16, DEV, F16, F32, Guarded, M, blank, gen, linear_exact, workspace  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def aligned(layout, *row_bytes):
    """Whether rows of so many bytes are whole 16-byte pieces apart in this layout."""
    return layout == "aligned" or (layout in ("dense", "rows") and all(n % 16 == 0 for n in row_bytes))


def check_exact(got, want, tag):
    """want: the sum in binary64, rounded once."""
    want = want.float().to(got.dtype)
    same = got == want
    assert bool(same.all()), f"{tag}: {int((~same).sum())} of {same.numel()} differ, at {(~same).nonzero()[:4].tolist()}"


def dgrad_exact(M, b, t, c, r, dt, out, layout):
    """|sum| <= 6 r, in steps of 2^-3."""
    assert 6 * r * 8 < 2 ** 24
    g = gen(41 + b + 3 * t + 5 * c + 7 * r)
    dy, (wq, ws) = ps.small_int(g, b, t, r).to(dt), ps.small_mx8(g, b, r, c)
    D, W, X = Guarded(dy, layout), Guarded(wq, layout), blank((b, t, c), out, layout)
    M.hpo_mx8_dgrad(D.view, W.view, ws.to(DEV), X.view, workspace(M.hpo_mx8_dgrad_workspace(D.view, W.view)))
    want = dy.to(DEV).double() @ mu.mx_values(wq, ws).to(DEV)
    check_exact(X.view, want, f"dgrad {b}x{t}x{c}x{r} {dt} {out} {layout}")
    X.untouched_outside()


def wgrad_exact(M, b, t, c, r, dt, gt, layout, accumulate):
    """|sum| <= 6 t in steps of 2^-3; half of it joins whole numbers up to 3."""
    assert 6 * t * 8 < 2 ** 24
    g = gen(43 + b + 3 * t + 5 * c + 7 * r)
    dy, (xq, xs) = ps.small_int(g, b, t, r).to(dt), ps.small_mx8(g, b, t, c)
    grad = ps.small_int(g, b, r, c).to(gt)
    D, X = Guarded(dy, layout), Guarded(xq, layout)
    G = Guarded(grad if accumulate else torch.full_like(grad, math.nan), layout)
    M.hpo_mx8_wgrad(D.view, X.view, xs.to(DEV), G.view, workspace(M.hpo_mx8_wgrad_workspace(D.view, X.view)), scale=0.5,
                    accumulate=accumulate)
    want = 0.5 * (dy.to(DEV).double().mT.contiguous() @ mu.mx_values(xq, xs).to(DEV))
    check_exact(G.view, want + grad.to(DEV).double() if accumulate else want, f"wgrad {b}x{t}x{c}x{r} {dt} {gt} {layout}")
    G.untouched_outside()


# --------------------------------------------------------------------------
# sums in parts
# --------------------------------------------------------------------------
# (batch, tokens, columns, rows), side of the tiles and parts where operands are aligned
LINEAR_PARTS = [((1, 1010, 50000, 1000), 256, 16), ((1, 1000, 40000, 912), 128, 4), ((1, 70, 9000, 300), 64, 24)]
DGRAD_PARTS = [((1, 1040, 1008, 30000), 256, 12), ((1, 500, 1100, 9000), 128, 12), ((1, 128, 304, 6000), 64, 24)]
WGRAD_PARTS = [((1, 12000, 1040, 1000), 256, 12), ((1, 30000, 256, 512), 128, 32), ((1, 9000, 64, 72), 64, 48)]


@pytest.mark.parametrize("shape,side,parts", LINEAR_PARTS)
@pytest.mark.parametrize("layout", ["dense", "aligned", "padded"])
def test_linear_in_parts(M, shape, side, parts, layout):
    direct = aligned(layout, shape[2])
    assert pp.plan("linear", *shape, direct)[:2] == (side if direct else min(side, 128), parts)
    linear_exact(M, *shape, F16, layout, dev=DEV)


@pytest.mark.parametrize("shape,side,parts", DGRAD_PARTS)
@pytest.mark.parametrize("layout", ["aligned", "padded"])
def test_dgrad_in_parts(M, shape, side, parts, layout):
    assert pp.plan("dgrad", *shape, layout == "aligned")[:2] == (side if layout == "aligned" else min(side, 128), parts)
    dgrad_exact(M, *shape, BF16, F32, layout)
    dgrad_exact(M, *shape, F16, BF16, layout)


@pytest.mark.parametrize("shape,side,parts", WGRAD_PARTS)
@pytest.mark.parametrize("layout", ["aligned", "padded"])
def test_wgrad_in_parts(M, shape, side, parts, layout):
    assert pp.plan("wgrad", *shape, layout == "aligned")[:2] == (side if layout == "aligned" else min(side, 128), parts)
    wgrad_exact(M, *shape, BF16, F32, layout, True)
    wgrad_exact(M, *shape, F16, BF16, layout, False)


# --------------------------------------------------------------------------
# stacks on large tiles
# --------------------------------------------------------------------------
# A workgroup of the forward tiles of 256 takes tile after tile: more of them than 256 workgroups, over the borders of
# matrices, ragged on both sides, whole sums and parts
LINEAR_STACKS = [((2, 2304, 512, 2304), 162, 1), ((4, 2300, 528, 2600), 396, 1), ((5, 2100, 1040, 2300), 405, 1),
                 ((2, 1010, 50000, 1000), 32, 8)]
GRAD_STACKS = [("dgrad", (3, 1500, 2000, 1000), 144, 1), ("dgrad", (5, 2100, 2000, 1000), 360, 1),
               ("dgrad", (4, 250, 704, 16000), 12, 16), ("wgrad", (3, 250, 512, 16000), 378, 1),
               ("wgrad", (2, 501, 6000, 1000), 192, 1), ("wgrad", (2, 20000, 704, 504), 12, 16)]


@pytest.mark.parametrize("shape,tiles,parts", LINEAR_STACKS)
@pytest.mark.parametrize("layout", ["dense", "aligned", "rows"])
def test_linear_stacks_of_large_tiles(M, shape, tiles, parts, layout):
    assert aligned(layout, shape[2]) and pp.plan("linear", *shape) == (256, parts, tiles)
    linear_exact(M, *shape, BF16 if parts == 1 else F16, layout, dev=DEV)


@pytest.mark.parametrize("kind,shape,tiles,parts", GRAD_STACKS)
@pytest.mark.parametrize("layout", ["dense", "aligned", "rows"])
def test_gradient_stacks_of_large_tiles(M, kind, shape, tiles, parts, layout):
    assert aligned(layout, shape[2], 2 * shape[3]) and pp.plan(kind, *shape) == (256, parts, tiles)
    if kind == "dgrad":
        dgrad_exact(M, *shape, BF16, F32, layout)
    else:
        wgrad_exact(M, *shape, BF16, F32, layout, True)
