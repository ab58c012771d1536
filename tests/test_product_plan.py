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
