"""CPU tier: the rule that product_plan.py writes down is the library's, as far as its workspaces show it."""
import ctypes
import os
import random

import pytest

pytest.importorskip("torch")

import product_plan as pp  # noqa: E402


@pytest.mark.parametrize("kind", ["linear", "dgrad", "wgrad"])
def test_parts_are_the_workspaces(kind):
    from mixed_precision_optimizer_amd import hpo, hpo_model
    if not os.path.exists(hpo.LIB_PATH):
        from mixed_precision_optimizer_amd import build
        build.build()
    fn = getattr(hpo_model.load(), f"hpo_mx8_{kind}_workspace")
    rng, out, in_parts = random.Random(kind), ctypes.c_int64(), 0
    for _ in range(3000):
        b, t, c, r = (int(2 ** rng.uniform(0, top)) for top in (6, 17, 16, 16))
        assert fn(b, t, c, r, ctypes.byref(out)) == hpo.HPO_OK
        m, n, _ = pp.mnk(kind, t, c, r)
        parts = pp.cut(kind, b, t, c, r)[1]
        assert out.value == (4 * b * parts * m * n if parts > 1 else 0), (b, t, c, r)
        in_parts += parts > 1
    assert 300 < in_parts < 2700


@pytest.mark.parametrize("drop", [0, 3, 195, 390])
def test_a_lost_stage_shows_in_an_exact_case(drop):
    """Of the deepest exact case (k = 50000, results in fp16) one stage of 128 left out, or at half its scale, changes
    most results; of a gradient's (k = 30000, fp32) one of 64 changes nearly all."""
    import torch

    import model_util as mu
    import product_sums as ps
    g = torch.Generator().manual_seed(drop)
    a, b = (mu.mx_values(*ps.small_mx8(g, 50, 50000)) for _ in range(2))
    at = slice(128 * drop, min(128 * drop + 128, 50000))
    whole, lost = a @ b.T, a[:, at] @ b[:, at].T
    for other in (whole - lost, whole - lost / 2):
        assert float((whole.half() != other.half()).double().mean()) > 0.75
    a = ps.small_int(g, 50, 30000).double()
    lost = a[:, 64 * drop: 64 * drop + 64] @ b[:, 64 * drop: 64 * drop + 64].T
    whole = a @ b[:, :30000].T
    assert float((whole.float() != (whole - lost).float()).double().mean()) > 0.95
