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


@pytest.mark.parametrize("kind,shape", [("dgrad", (1024, 1, 1 << 20, 8)), ("wgrad", (32768, 8, 32768, 64)),
                                        ("linear", (1, 1 << 20, 16, 1 << 19))])
def test_more_threads_than_a_launch_holds_are_refused(kind, shape):
    """2^24 tiles of 256 threads and more: a launch has 2^32 - 1 at most.  The refusal is the call's own, found before
    anything is enqueued: a launch that the runtime refuses would leave its error to the caller's next check."""
    from mixed_precision_optimizer_amd import hpo, hpo_model as M
    b, t, c, r = shape
    lib, at, size = M.load(), 0x10000, 1 << 60
    side, parts, tiles = pp.plan(kind, *shape)
    assert side < 256 and tiles * parts * 256 >= 2 ** 32

    def stack(rows, cols, dtype):
        return ctypes.byref(M.c_stack(at, b, rows, cols, rows * cols, cols, dtype, 0))
    x, w, dy = stack(t, c, 16), stack(r, c, 16), stack(t, r, 0)
    st = {"linear": lambda: lib.hpo_mx8_linear(x, at, w, at, dy, at, size, None),
          "dgrad": lambda: lib.hpo_mx8_dgrad(dy, w, at, stack(t, c, 0), at, size, None),
          "wgrad": lambda: lib.hpo_mx8_wgrad(dy, x, at, 1.0, 1, stack(r, c, 1), at, size, None)}[kind]()
    assert st == hpo.HPO_EINVAL and "more tiles" in hpo.hpo_last_error(), (st, hpo.hpo_last_error())
