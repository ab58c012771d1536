"""Gradients of the 8-bit products over a single token, and at scale bytes from one end of the range to the other."""
import math

import pytest

torch = pytest.importorskip("torch")

import model_util as mu  # noqa: E402
import product_plan as pp  # noqa: E402
from test_gpu_model import BF16, DEV, E4M3, F16, F32, Guarded, M, gen, workspace  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# (batch, columns, rows): every tile; 16-byte pieces, and sizes that leave some over
ONE = [(1, 64, 64), (16, 64, 64), (1, 100, 33), (16, 36, 70), (2, 1000, 1000), (1, 1500, 4000), (1, 2048, 8192)]


def wgrad(M, dy, q, byte, grad, layout, accumulate=True, scale=1.0):
    D, X, G = Guarded(dy, layout), Guarded(q, layout), Guarded(grad, layout)
    M.hpo_mx8_wgrad(D.view, X.view, byte.to(DEV), G.view, workspace(M.hpo_mx8_wgrad_workspace(D.view, X.view)), scale=scale,
                    accumulate=accumulate)
    G.untouched_outside()
    return G.view.cpu()


def values(q, byte, dtype):
    """X^ or W^ in dY's type, as documented."""
    v = mu.mx_values(q, byte)
    return v.half().double() if dtype == F16 else v


def test_one_token_reaches_every_tile():
    assert {pp.plan("wgrad", b, 1, c, r)[0] for b, c, r in ONE} == {64, 128, 256}


@pytest.mark.parametrize("b,c,r", ONE)
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("layout", ["dense", "aligned", "padded"])
def test_weight_gradient_of_one_token(M, b, c, r, dt, layout):
    """One product for each element, so one rounding (none in fp32): G = dY q 2^(byte - 127) bit for bit, at the smallest
    scales too, where a token that is not there, at the scale of a byte that is not there, would count as much."""
    g = gen(b + c + r)
    dy = torch.randint(1, 256, (b, 1, r), generator=g).to(dt)          # eight bits, all of them normal
    dy = dy * (2.0 ** 100 if dt == BF16 else 1.0) * (torch.randint(0, 2, dy.shape, generator=g) * 2 - 1)
    q = (torch.randint(8, 16, (b, 1, c), generator=g) * 0.5).to(E4M3)   # 4 .. 7.5
    nb = -(-c // 32)
    low = torch.tensor([0, 1, 8, 40, 60]) if dt == BF16 else torch.tensor([112, 120, 127])
    byte = low[torch.randint(0, len(low), (b, 1, nb), generator=g)].to(torch.uint8)
    want = dy.double().mT @ values(q, byte, dt)
    got = wgrad(M, dy.to(dt), q, byte, torch.full((b, r, c), math.nan), layout, accumulate=False)
    assert torch.equal(got.double(), want), int((got.double() != want).sum())
    grad = torch.randn(b, r, c, generator=g)
    got = wgrad(M, dy.to(dt), q, byte, grad, layout, scale=0.5)
    mu.check(got, grad.double() + 0.5 * want, mu.product_tolerance(want.abs(), 1, grad.double() + 0.5 * want, F32, 0.5,
                                                                   grad.double()), f"one token {b} {c} {r} {dt} {layout}")


@pytest.mark.parametrize("b,c,r", ONE[:5])
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("layout", ["dense", "aligned", "padded"])
def test_infinite_gradient_of_one_token(M, b, c, r, dt, layout):
    """A loss scale that was too large: infinities stay infinities of their sign, NaN stays in its row."""
    g = gen(c + r)
    dy = torch.randn(b, 1, r, generator=g).to(dt)
    dy[0, 0, 1], dy[b - 1, 0, r - 1], dy[0, 0, 2] = math.inf, -math.inf, math.nan
    q = (torch.randint(8, 16, (b, 1, c), generator=g) * 0.5).to(E4M3)
    byte = torch.full((b, 1, -(-c // 32)), 120, dtype=torch.uint8)
    got = wgrad(M, dy, q, byte, torch.zeros(b, r, c), layout)
    want = dy.float().mT * mu.mx_values(q, byte).float()
    assert torch.equal(got.nan_to_num(nan=-5.0, posinf=1e30, neginf=-1e30), want.nan_to_num(nan=-5.0, posinf=1e30, neginf=-1e30))


@pytest.mark.parametrize("t,c,r", [(1, 96, 80), (3, 96, 80), (40, 64, 64), (65, 100, 33), (600, 512, 600)])
@pytest.mark.parametrize("byte", [0, 1, 8, 246])
@pytest.mark.parametrize("dt", [BF16, F16])
def test_gradients_at_the_ends_of_the_scales(M, t, c, r, byte, dt):
    """All blocks at one scale byte; the values (2 .. 7.5, negative ones too) are normal in bf16 at each, and at 246 under its
    largest.  In fp16 the small ones are 0 and the large ones infinite."""
    g = gen(t + c + r + byte)

    def eight(*s):
        return (torch.randint(4, 16, s, generator=g) * 0.5 * (torch.randint(0, 2, s, generator=g) * 2 - 1)).to(E4M3)
    dy = torch.randint(1, 256, (t, r), generator=g) * (torch.randint(0, 2, (t, r), generator=g) * 2 - 1)
    dy = (dy * (1.0 if dt == F16 else 2.0 ** -30 if byte == 246 else 2.0 ** 60)).to(dt)
    for layout in ("dense", "padded"):
        q, sc = eight(t, c), torch.full((t, -(-c // 32)), byte, dtype=torch.uint8)
        want, size = mu.matmul64(dy.mT, values(q, sc, dt))
        got = wgrad(M, dy, q, sc, torch.full((r, c), math.nan), layout, accumulate=False)
        mu.check(got, want, mu.product_tolerance(size, t, want, F32).nan_to_num(0.0, 0.0), f"wgrad {t} {c} {r} {byte} {dt}")
        q, sc = eight(r, c), torch.full((r, -(-c // 32)), byte, dtype=torch.uint8)
        want, size = mu.matmul64(dy, values(q, sc, dt))
        D, W = Guarded(dy, layout), Guarded(q, layout)
        dx = torch.full((t, c), math.nan, device=DEV)
        M.hpo_mx8_dgrad(D.view, W.view, sc.to(DEV), dx, workspace(M.hpo_mx8_dgrad_workspace(D.view, W.view)))
        mu.check(dx, want, mu.product_tolerance(size, r, want, F32).nan_to_num(0.0, 0.0), f"dgrad {t} {c} {r} {byte} {dt}")
