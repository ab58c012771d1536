"""Stack operators on the GPU at the ends of their numbers' ranges."""
import math

import pytest

torch = pytest.importorskip("torch")

import stack_util as su  # noqa: E402
from test_gpu_stack import CFG, DEV, S, check_rms, gen, workspace  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# hpo_rms_update: rows whose factor 1 / (sqrt(v) + eps) is beyond fp32
# --------------------------------------------------------------------------
@pytest.mark.parametrize("eps", [5e-324, 1e-310, 1e-150, 1e-40, 2.0 ** -129])
@pytest.mark.parametrize("beta2", [0.0, 0.95])
def test_rms_update_zero_rows_with_a_tiny_eps(S, eps, beta2):
    """A row of zeros without a history has 1 / eps for a factor and is not moved by it.  Beside sqrt(v) such an eps
    is under half a step of binary64: the other rows are those of eps = 0."""
    O, W0, v0 = rms_inputs_with_zeros()
    cfg = dict(CFG, eps=eps, beta2=beta2)
    W, v, p = W0.to(DEV), v0.to(DEV), W0.bfloat16().to(DEV)
    S.hpo_rms_update(O.to(DEV), W, v, S.make_rms_cfg(**cfg), workspace(S.hpo_rms_update_workspace(W)), param=p)
    check_rms(W, v, W0, O, v0, dict(cfg, eps=0.0), f"eps {eps}")
    su.check_weight(W, p)
    keep = W0 * torch.tensor(1 - 0.02 * 0.1, dtype=torch.float32)
    assert torch.equal(W[0].cpu(), keep[0]) and torch.equal(W[1, 3].cpu(), keep[1, 3])


def rms_inputs_with_zeros():
    g = gen(101)
    O = torch.randn(2, 30, 70, generator=g)
    W0, v0 = 0.02 * torch.randn(2, 30, 70, generator=g), torch.rand(2, 30, generator=g) / 70
    O[0], O[1, 3], v0[0], v0[1, 3] = 0.0, 0.0, 0.0, 0.0
    return O, W0, v0


@pytest.mark.parametrize("eps", [1e-310, 1e-40])
def test_rms_update_row_whose_running_mean_rounds_to_zero(S, eps):
    """The squares of the last row are there (2^-148), the share of them in v is under fp32's least value: with a tiny
    eps that row is all of N, and all of the update."""
    rows, cols = 5, 64
    O = torch.randn(1, rows, cols, generator=gen(103))
    O[0, -1] = 2.0 ** -74
    W0 = torch.zeros(1, rows, cols)
    W, v = W0.to(DEV), torch.zeros(1, rows, device=DEV)
    cfg = dict(CFG, eps=eps, weight_decay=0.0)
    S.hpo_rms_update(O.to(DEV), W, v, S.make_rms_cfg(**cfg), workspace(S.hpo_rms_update_workspace(W)))
    assert v[0, -1].item() == 0.0
    # s r_i O_ij = lr target sqrt(rows cols) / (sqrt(cols) |O_ij|) O_ij; the factor and the product round once each
    want = -CFG["lr"] * CFG["target_rms"] * math.sqrt(rows)
    assert bool(((W[0, -1].double() - want).abs() <= 4 * su.HALF32 * abs(want)).all())
    # the others' share is r_i O_ij / (r_last |O|): under 1e-15 of it
    assert bool((W[0, :-1].abs() <= 1e-15 * abs(want)).all())


def test_rms_update_factors_beyond_fp32_leave_rows_of_zeros(S):
    """s r_i is beyond fp32's range where N is small and v_i smaller; so is s where lr asks for it."""
    O, W0 = torch.zeros(1, 3, 64), torch.randn(1, 3, 64, generator=gen(105))
    O[0, 0] = 1e-20
    v0 = torch.tensor([[1e10, 1e-38, 0.0]])
    for cfg in (dict(CFG, eps=0.0), dict(CFG, eps=0.0, lr=1e308, target_rms=1e3, weight_decay=0.0)):
        W, v = W0.to(DEV), v0.to(DEV)
        S.hpo_rms_update(O.to(DEV), W, v, S.make_rms_cfg(**cfg), workspace(S.hpo_rms_update_workspace(W)))
        keep = W0 * torch.tensor(1 - cfg["lr"] * cfg["weight_decay"], dtype=torch.float32)
        assert torch.equal(W[0, 1:].cpu(), keep[0, 1:]), cfg
