"""The 8-bit products where values or results are subnormal, and with scale arrays at odd addresses.  One product for
each element, so that nothing rounds but the operands' and the result's types."""
import pytest

torch = pytest.importorskip("torch")

import model_util as mu  # noqa: E402
from test_gpu_model import BF16, DEV, E4M3, F16, M, gen, workspace  # noqa: E402,F401

pytestmark = pytest.mark.gpu
SHAPES = [(64, 64, 64), (40, 100, 33)]   # whole 16-byte pieces, and not


def one_a_row(rows, cols, value, dtype):
    """Column i mod cols of row i, zeros elsewhere."""
    x = torch.zeros(rows, cols, dtype=torch.float64)
    x[torch.arange(rows), torch.arange(rows) % cols] = value
    return x.to(dtype)


def halves(g, rows, cols):
    return (torch.randint(4, 16, (rows, cols), generator=g) * 0.5).to(E4M3)


def scales(rows, cols, byte):
    return torch.full((rows, -(-cols // 32)), byte, dtype=torch.uint8)


def dgrad(M, dy, q, byte):
    dx = torch.empty(dy.shape[0], q.shape[1], device=DEV)
    M.hpo_mx8_dgrad(dy.to(DEV), q.to(DEV), byte.to(DEV), dx, workspace(M.hpo_mx8_dgrad_workspace(dy, q)))
    return dx.double().cpu()


@pytest.mark.parametrize("t,c,r", SHAPES)
@pytest.mark.parametrize("dt,power", [(F16, e) for e in (-14, -15, -18, -24)] + [(BF16, e) for e in (-126, -127, -130, -133)])
def test_subnormal_gradients(M, t, c, r, dt, power):
    g = gen(t - power)
    dy, q, byte = one_a_row(t, r, 2.0 ** power, dt), halves(g, r, c), scales(r, c, 127)
    assert torch.equal(dgrad(M, dy, q, byte), dy.double() @ mu.mx_values(q, byte))
    dy = torch.zeros(t, r, dtype=torch.float64)
    dy[3] = 2.0 ** power
    dy, q, byte = dy.to(dt), halves(g, t, c), scales(t, c, 127)
    G = torch.zeros(r, c, device=DEV)
    M.hpo_mx8_wgrad(dy.to(DEV), q.to(DEV), byte.to(DEV), G, workspace(M.hpo_mx8_wgrad_workspace(dy, q)))
    assert torch.equal(G.double().cpu(), dy.double().T @ mu.mx_values(q, byte))


@pytest.mark.parametrize("t,c,r", SHAPES)
@pytest.mark.parametrize("dt,byte", [(F16, b) for b in (113, 109, 105, 101)] + [(BF16, b) for b in (8, 1, 0)])
def test_weights_that_are_subnormal_in_16_bits(M, t, c, r, dt, byte):
    """Every e4m3 value at scales where dY's type has them as subnormals: rounded to nearest, none flushed."""
    g = gen(t + byte)
    q, s = torch.randint(0, 127, (r, c), generator=g).to(torch.uint8).view(E4M3), scales(r, c, byte)
    dy = one_a_row(t, r, 1.0 if dt == F16 else 2.0 ** 40, dt)
    assert torch.equal(dgrad(M, dy, q, s), dy.double() @ mu.mx_values(q, s).to(dt).double())


@pytest.mark.parametrize("t,c,r", SHAPES)
@pytest.mark.parametrize("xb,wb,out", [(8, 100, BF16), (8, 113, BF16), (0, 127, BF16), (110, 120, F16), (105, 120, F16),
                                       (0, 0, BF16), (254, 1, BF16)])
def test_results_that_are_subnormal(M, t, c, r, xb, wb, out):
    g = gen(t + xb + wb)
    x, xs = one_a_row(t, c, 1.5, E4M3), scales(t, c, xb)
    w, ws = (torch.randint(4, 8, (r, c), generator=g) * 0.5).to(E4M3), scales(r, c, wb)
    y = torch.empty(t, r, dtype=out, device=DEV)
    M.hpo_mx8_linear(x.to(DEV), xs.to(DEV), w.to(DEV), ws.to(DEV), y, workspace(M.hpo_mx8_linear_workspace(x, w)))
    want = mu.mx_values(x, xs) @ mu.mx_values(w, ws).T
    assert torch.equal(y.cpu(), want.float().to(out))
    dy, q, byte = one_a_row(t, r, 2.0 ** -20, BF16), halves(g, r, c), scales(r, c, 8)   # subnormal in fp32
    assert torch.equal(dgrad(M, dy, q, byte), dy.double() @ mu.mx_values(q, byte))


@pytest.mark.parametrize("t,c,r", [(40, 64, 33), (40, 1000, 33), (64, 1024, 64)])
def test_scales_at_odd_addresses(M, t, c, r):
    g = gen(c)

    def odd(s):
        v = torch.empty(s.numel() + 1, dtype=torch.uint8, device=DEV)[1:].view(s.shape)
        v.copy_(s.to(DEV))
        assert v.data_ptr() % 2 == 1
        return v
    x, w, dy = halves(g, t, c).to(DEV), halves(g, r, c).to(DEV), torch.randn(t, r, generator=g).to(BF16).to(DEV)
    xs, ws = (torch.randint(120, 130, (n, -(-c // 32)), generator=g).to(torch.uint8) for n in (t, r))
    outs = []
    for at in (lambda s: s.to(DEV), odd):
        y, dx, G = torch.empty(t, r, dtype=BF16, device=DEV), torch.empty(t, c, device=DEV), torch.zeros(r, c, device=DEV)
        M.hpo_mx8_linear(x, at(xs), w, at(ws), y, workspace(M.hpo_mx8_linear_workspace(x, w)))
        M.hpo_mx8_dgrad(dy, w, at(ws), dx, workspace(M.hpo_mx8_dgrad_workspace(dy, w)))
        M.hpo_mx8_wgrad(dy, x, at(xs), G, workspace(M.hpo_mx8_wgrad_workspace(dy, x)))
        table = torch.empty(t, c, device=DEV)
        M.hpo_embedding(torch.arange(t, device=DEV) % r, w, table, scales=at(ws))
        outs.append([v.cpu() for v in (y, dx, G, table)])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
