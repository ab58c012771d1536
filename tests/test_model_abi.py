"""CPU tier: the model operators' symbols and argument checks.  No call here
reaches a kernel."""
import ctypes
import os
import re

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

P = 0x10000   # a 256-byte aligned address that no accepted call may use
MX8, BF16, FP32, FP16 = 16, 0, 1, 2
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def M():
    from mixed_precision_optimizer_amd import hpo, hpo_model
    if not os.path.exists(hpo.LIB_PATH):
        from mixed_precision_optimizer_amd import build
        build.build()
    hpo_model.load()
    return hpo_model


@pytest.fixture(scope="module")
def H(M):
    return M.hpo


def test_exports_every_declared_symbol(M):
    src = open(os.path.join(ROOT, "include", "hpo_model.h")).read()
    names = re.findall(r"^(?:hpo_status|const char\*|int32_t)\s+(hpo_\w+)\(", src, re.M)
    assert set(names) == set(M.SIGNATURES)
    for n in names:
        assert hasattr(M.load(), n), n


def stack(M, rows, cols, dtype, batch=1, rs=None, data=P, reserved=0, bs=None):
    rs = cols if rs is None else rs
    return M.c_stack(data, batch, rows, cols, rows * rs if bs is None else bs, rs, dtype, reserved)


def ref(s):
    return None if s is None else ctypes.byref(s)


def refused(H, calls, status):
    for k, (call, word) in enumerate(calls):
        st, msg = call(), H.hpo_last_error()
        assert st == status and word in msg, (k, st, msg, word)


def test_embedding_refusals(M, H):
    L = M.load()

    def call(ids=P, nb=8, n=4, first=0, w=stack(M, 10, 32, BF16), sc=None, scale=1.0, out=stack(M, 4, 32, BF16)):
        return lambda: L.hpo_embedding(ids, nb, n, first, ref(w), sc, scale, ref(out), None)

    refused(H, [
        (call(ids=None), "d_ids"), (call(ids=P + 4), "d_ids"), (call(ids=P + 2, nb=4), "d_ids"), (call(n=-1), "n must"),
        (call(n=H.HPO_MUON_MAX_DIM + 1), "n must"), (call(first=-1), "first"), (call(first=2 ** 62 + 1), "first"),
        (call(w=None), "weight is NULL"), (call(w=stack(M, 10, 32, BF16, batch=2)), "one matrix"),
        (call(w=stack(M, 10, 32, MX8)), "d_scales"), (call(sc=P), "d_scales"), (call(out=None), "out is NULL"),
        (call(out=stack(M, 5, 32, BF16)), "expected"), (call(out=stack(M, 4, 31, BF16)), "expected"),
        (call(out=stack(M, 4, 32, BF16, batch=2)), "expected"), (call(scale=NAN), "scale"), (call(scale=INF), "scale"),
        (call(w=stack(M, 10, 32, BF16, rs=31)), "stride"), (call(out=stack(M, 4, 32, FP32, data=P + 2)), "aligned"),
        (call(out=stack(M, 4, 32, FP32, data=0)), "non-NULL"), (call(w=stack(M, 10, 32, BF16, reserved=1)), "reserved"),
    ], H.HPO_EINVAL)
    refused(H, [(call(nb=2), "id_bytes"), (call(w=stack(M, 10, 32, 5)), "weight dtype"),
                (call(out=stack(M, 4, 32, MX8)), "out dtype")], H.HPO_EDTYPE)
    assert call(ids=None, n=0, out=stack(M, 0, 32, BF16, data=0))() == H.HPO_OK
    assert call(w=stack(M, 10, 0, BF16, data=0), out=stack(M, 4, 0, BF16, data=0))() == H.HPO_OK


def test_embedding_grad_refusals(M, H):
    L = M.load()

    def call(ids=P, nb=4, n=200, first=0, dy=stack(M, 200, 32, BF16), scale=1.0, g=stack(M, 10, 32, FP32), ws=P, size=BIG):
        return lambda: L.hpo_embedding_grad(ids, nb, n, first, ref(dy), scale, ref(g), ws, size, None)

    refused(H, [
        (call(ids=None), "d_ids"), (call(ids=P + 2), "d_ids"), (call(n=-1), "n must"), (call(first=-1), "first"),
        (call(g=None), "grad is NULL"), (call(g=stack(M, 10, 32, FP32, batch=3)), "one matrix"),
        (call(dy=None), "dy is NULL"), (call(dy=stack(M, 199, 32, BF16)), "expected"),
        (call(dy=stack(M, 200, 33, BF16)), "expected"), (call(scale=NAN), "scale"), (call(ws=None), "workspace"),
        (call(ws=P + 16), "256-byte"), (call(size=64), "below"),
    ], H.HPO_EINVAL)
    refused(H, [(call(g=stack(M, 10, 32, FP16)), "grad dtype"), (call(g=stack(M, 10, 32, MX8)), "grad dtype"),
                (call(dy=stack(M, 200, 32, MX8)), "dy dtype"), (call(nb=1), "id_bytes")], H.HPO_EDTYPE)
    assert call(ids=None, n=0, dy=stack(M, 0, 32, BF16, data=0), ws=None, size=0)() == H.HPO_OK
    assert call(g=stack(M, 0, 32, FP32, data=0), ws=None, size=0)() == H.HPO_OK
    out = ctypes.c_int64(7)
    for n, cols, ok in ((0, 5, True), (5, 0, True), (-1, 5, False), (5, -1, False), (H.HPO_MUON_MAX_DIM + 1, 5, False)):
        st = L.hpo_embedding_grad_workspace(n, cols, ctypes.byref(out))
        assert st == (H.HPO_OK if ok else H.HPO_EINVAL) and (not ok or out.value == 0)
    assert L.hpo_embedding_grad_workspace(5, 5, None) == H.HPO_EINVAL
    for n in (200, 8192, 8193, 65536, H.HPO_MUON_MAX_DIM):
        assert L.hpo_embedding_grad_workspace(n, 4096, ctypes.byref(out)) == H.HPO_OK
        # two lists of (row, token), two fp32 rows for each slab of 8 tokens at least, counts of blocks of 4096
        assert 8 * n <= out.value <= 16 * n + 2 * 4096 * 4 * (n // 8 + 1) + (n // 4096 + 1) * 8192 + 4096


def test_save_refusals(M, H):
    L = M.load()

    def call(x=stack(M, 4, 70, BF16, batch=2), q=stack(M, 4, 70, MX8, batch=2), sc=P):
        return lambda: L.hpo_mx8_save(ref(x), ref(q), sc, None)

    refused(H, [(call(x=None), "x is NULL"), (call(q=None), "q is NULL"), (call(sc=None), "scales"),
                (call(q=stack(M, 4, 69, MX8, batch=2)), "q is"), (call(q=stack(M, 4, 70, MX8, batch=2, bs=64)), "stride")],
            H.HPO_EINVAL)
    refused(H, [(call(x=stack(M, 4, 70, MX8, batch=2)), "x dtype"), (call(q=stack(M, 4, 70, BF16, batch=2)), "q must")],
            H.HPO_EDTYPE)
    assert call(stack(M, 0, 70, BF16, data=0), stack(M, 0, 70, MX8, data=0), None)() == H.HPO_OK


def test_product_refusals(M, H):
    L = M.load()
    t, c, r, b = 6, 64, 40, 2
    x, w = stack(M, t, c, MX8, b), stack(M, r, c, MX8, b)
    dy, y, dx, g = stack(M, t, r, BF16, b), stack(M, t, r, FP16, b), stack(M, t, c, BF16, b), stack(M, r, c, FP32, b)

    def linear(x=x, xs=P, w=w, ws=P, y=y, work=P, size=BIG):
        return lambda: L.hpo_mx8_linear(ref(x), xs, ref(w), ws, ref(y), work, size, None)

    def dgrad(dy=dy, w=w, ws=P, dx=dx, work=P, size=BIG):
        return lambda: L.hpo_mx8_dgrad(ref(dy), ref(w), ws, ref(dx), work, size, None)

    def wgrad(dy=dy, x=x, xs=P, scale=1.0, acc=1, g=g, work=P, size=BIG):
        return lambda: L.hpo_mx8_wgrad(ref(dy), ref(x), xs, scale, acc, ref(g), work, size, None)

    refused(H, [
        (linear(x=None), "x is NULL"), (linear(w=None), "w is NULL"), (linear(y=None), "y is NULL"), (linear(xs=None), "scales"),
        (linear(ws=None), "scales"), (linear(w=stack(M, r, c + 1, MX8, b)), "agree"), (linear(w=stack(M, r, c, MX8, 1)), "agree"),
        (linear(y=stack(M, t, r + 1, BF16, b)), "expected"), (linear(y=stack(M, t, r, BF16, 1)), "expected"),
        (dgrad(dy=None), "dy is NULL"), (dgrad(w=None), "w is NULL"), (dgrad(ws=None), "scales"), (dgrad(dx=None), "dx is NULL"),
        (dgrad(dy=stack(M, t, r + 1, BF16, b)), "agree"), (dgrad(dx=stack(M, t, c - 1, BF16, b)), "expected"),
        (wgrad(dy=None), "dy is NULL"), (wgrad(x=None), "x is NULL"), (wgrad(xs=None), "scales"), (wgrad(g=None), "grad is NULL"),
        (wgrad(dy=stack(M, t + 1, r, BF16, b)), "agree"), (wgrad(g=stack(M, r + 1, c, FP32, b)), "expected"),
        (wgrad(scale=INF), "scale"), (wgrad(acc=2), "accumulate"), (wgrad(acc=-1), "accumulate"),
    ], H.HPO_EINVAL)
    refused(H, [
        (linear(x=stack(M, t, c, BF16, b)), "x must"), (linear(w=stack(M, r, c, FP16, b)), "w must"),
        (linear(y=stack(M, t, r, MX8, b)), "y dtype"), (linear(y=stack(M, t, r, FP32, b)), "y dtype"), (dgrad(dy=stack(M, t, r, FP32, b)), "dy dtype"),
        (dgrad(dx=stack(M, t, c, MX8, b)), "dx dtype"), (wgrad(dy=stack(M, t, r, FP32, b)), "dy dtype"),
        (wgrad(g=stack(M, r, c, FP16, b)), "grad dtype"),
    ], H.HPO_EDTYPE)


def test_products_of_nothing_do_nothing(M, H):
    L = M.load()
    none = lambda rows, cols, dt: stack(M, rows, cols, dt, data=0)   # noqa: E731
    assert L.hpo_mx8_linear(ref(none(0, 8, MX8)), None, ref(stack(M, 4, 8, MX8)), P, ref(none(0, 4, BF16)), None, 0,
                            None) == H.HPO_OK
    assert L.hpo_mx8_dgrad(ref(stack(M, 4, 8, BF16)), ref(none(8, 0, MX8)), None, ref(none(4, 0, BF16)), None, 0,
                           None) == H.HPO_OK
    # no tokens: the main grad is kept
    assert L.hpo_mx8_wgrad(ref(none(0, 8, BF16)), ref(none(0, 4, MX8)), None, 1.0, 1, ref(stack(M, 8, 4, FP32)), None, 0,
                           None) == H.HPO_OK


@pytest.mark.parametrize("name", ["linear", "dgrad", "wgrad"])
def test_product_workspaces(M, H, name):
    fn = getattr(M.load(), f"hpo_mx8_{name}_workspace")
    out = ctypes.c_int64(7)
    for bad in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, -1), (65536, 1, 1, 1), (1, H.HPO_MUON_MAX_DIM + 1, 1, 1)):
        assert fn(*bad, ctypes.byref(out)) == H.HPO_EINVAL
    assert fn(1, 1, 1, 1, None) == H.HPO_EINVAL
    # much work: one pass; little and deep: the depth is cut
    assert fn(1, 8192, 4096, 14336, ctypes.byref(out)) == H.HPO_OK and out.value == 0
    deep = {"linear": (1, 64, 65536, 64), "dgrad": (1, 64, 64, 65536), "wgrad": (1, 65536, 64, 64)}[name]
    assert fn(*deep, ctypes.byref(out)) == H.HPO_OK and out.value > 0 and out.value % (4 * 64 * 64) == 0


def test_binding_refuses_what_is_not_on_the_device(M):
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError, match="device"):
        M.hpo_mx8_save(x, x.to(torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(TypeError, match="int32 or int64"):
        M.hpo_embedding(torch.zeros(4), x, x)
    with pytest.raises(ValueError, match="device"):
        M.hpo_embedding(torch.zeros(4, dtype=torch.int64), x, x)
