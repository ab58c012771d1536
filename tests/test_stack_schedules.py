"""CPU tier: which Newton-Schulz coefficients hpo_orthogonalize takes.  No call here reaches a kernel."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_stack_abi import H, S, ortho, stack  # noqa: E402, F401

# odd quintics fitted to [0, 1] step by step: bounded from a start of 1, and steep there
TIGHT = [(8.2872, -23.5959, 17.3004), (4.1071, -2.9478, 0.5448), (3.9487, -2.9089, 0.5518), (3.3184, -2.4885, 0.5100),
         (2.3007, -1.6689, 0.4188)]


def scaled(f):
    return [(a / f, b / f ** 3, c / f ** 5) for a, b, c in TIGHT]


def call(S, H, coeffs):
    cfg = H.make_muon_cfg(ns_steps=len(coeffs), ns_coeffs=coeffs)
    return ortho(S, H, stack(S), stack(S, dtype=0), cfg=cfg, nbytes=0)


def most(coeffs, start):
    """Largest singular value behind the last step, on a fine grid of [0, start]."""
    s = np.linspace(0.0, start, 200001)
    for a, b, c in coeffs:
        s = s * (a + s * s * (b + s * s * c))
    return float(np.abs(s).max())


def test_a_schedule_that_only_holds_up_to_one_is_refused_and_told_why(S, H):
    st, msg = call(S, H, TIGHT)
    assert st == H.HPO_EINVAL and "1 %" in msg and "step 3" in msg, msg
    # what the 1 % stands for: exact arithmetic holds, a start 1e-3 above 1 does not
    assert most(TIGHT, 1.0) < 2.0
    assert most(TIGHT, 1.001) > 2.0 ** 15


def test_the_same_schedule_with_room_for_roundings_is_taken(S, H):
    st, msg = call(S, H, scaled(1.01))
    assert st == H.HPO_EINVAL and "below" in msg, msg     # as far as the workspace
    assert most(scaled(1.01), 1.001) < 2.0
    st, msg = call(S, H, scaled(1.004))
    assert st == H.HPO_EINVAL and "ns_coeffs" in msg, msg
