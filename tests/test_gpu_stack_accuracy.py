"""What include/hpo_stack.h says of hpo_orthogonalize's error before the result is rounded to bf16."""
import math

import pytest

torch = pytest.importorskip("torch")

import stack_util as su  # noqa: E402
from test_gpu_stack import DEV, S, ortho  # noqa: E402, F401

pytestmark = pytest.mark.gpu

KINDS = ("noise", "mixed", "low", "one", "decay", "equal")


def gradients(kind, b, r, c):
    """Singular values all alike; a few strong ones over 30 % or 1 % of noise; one over 0.1 %; three decades of them;
    elements all but equal."""
    g = torch.Generator(device=DEV).manual_seed(r + c)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    k = {"one": 1, "decay": min(r, c)}.get(kind, max(1, min(r, c) // 16))
    if kind == "noise":
        return 1e-3 * n(b, r, c)
    if kind == "equal":
        return 0.37 + 0.01 * n(b, r, c)
    u = n(b, r, k) * (torch.logspace(0, -3, k, device=DEV) if kind == "decay" else 1.0)
    noise = {"mixed": 0.3, "low": 0.01, "one": 1e-3, "decay": 0.0}[kind]
    return 1e-3 * (u @ n(b, k, c) / math.sqrt(k) + noise * n(b, r, c))


def check_before_rounding(S, kind, b, r, c, claim, steps=5, coeffs=None):
    """The result is x + d rounded: x exact, d the error in question.  A rounding's error does not depend on d's (to
    first order it is spread evenly over a step), so the squares add: |out - x|^2 = |d|^2 + |round(x) - x|^2, up to
    what N elements' chance leaves: the cross term 2 |d| |round(x) - x| / sqrt(N), and the second square from other
    places in the steps, whose own spread is under 1.3 / sqrt(N) (an even spread's fourth moment, over binades).  Four
    deviations of both are allowed."""
    G = gradients(kind, b, r, c)
    out = ortho(S, G, cfg=S.hpo.make_muon_cfg(ns_steps=steps, ns_coeffs=coeffs))
    for z in sorted({0, b // 2, b - 1}):
        x = su.ns_exact(G[z], steps, coeffs)
        n2 = float(x.square().sum())
        got = float((out[z].double() - x).square().sum()) / n2
        q2 = float((x.bfloat16().double() - x).square().sum()) / n2
        chance = 4.0 / math.sqrt(r * c)
        print(f"[ortho] {kind} {b}x{r}x{c}[{z}] before rounding {math.sqrt(max(got - q2, 0.0)):.2e} (said: {claim:.0e})",
              flush=True)
        assert got <= claim ** 2 + 2 * claim * math.sqrt(q2) * chance + q2 * (1 + 1.3 * chance), (kind, z)


@pytest.mark.parametrize("b,r,c", [(2, 64, 2000), (2, 128, 640), (2, 640, 128), (2, 128, 4096), (2, 128, 128), (1, 100, 20000),
                                   (8, 40, 600)])
@pytest.mark.parametrize("kind", KINDS)
def test_thin_form_five_steps(S, kind, b, r, c):
    check_before_rounding(S, kind, b, r, c, 1e-3)


@pytest.mark.parametrize("b,r,c", [(520, 128, 8192), (520, 100, 16000), (600, 64, 8000), (700, 32, 8000), (1, 20, 1000000)])
@pytest.mark.parametrize("kind", KINDS)
def test_thin_form_five_steps_long_sums(S, kind, b, r, c):
    """One workgroup sums all of a matrix, or hundreds of them a part each."""
    check_before_rounding(S, kind, b, r, c, 3e-3)


@pytest.mark.parametrize("b,r,c", [(2, 64, 2000), (2, 128, 640), (2, 640, 128), (1, 100, 20000)])
def test_thin_form_without_directions_that_stand_out(S, b, r, c):
    for kind in ("noise", "mixed"):
        check_before_rounding(S, kind, b, r, c, 2e-4)


@pytest.mark.parametrize("b,r,c", [(2, 140, 1000), (2, 256, 512), (3, 1000, 333), (1, 1024, 1024), (1, 2048, 1024),
                                   (1, 2048, 4096), (1, 520, 5000)])
@pytest.mark.parametrize("kind", KINDS)
def test_two_product_form_five_steps(S, kind, b, r, c):
    check_before_rounding(S, kind, b, r, c, 2e-3)
