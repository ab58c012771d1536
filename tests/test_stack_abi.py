"""CPU tier: the stack operators' symbols, struct layouts and argument checks.
No call here reaches a kernel."""
import ctypes
import os
import re

import pytest

from conftest import ROOT

torch = pytest.importorskip("torch")

P = 0x10000   # a 16-byte aligned address that no accepted call may use


@pytest.fixture(scope="module")
def S():
    from mixed_precision_optimizer_amd import hpo, hpo_stack
    if not os.path.exists(hpo.LIB_PATH):
        from mixed_precision_optimizer_amd import build
        build.build()
    hpo_stack.load()
    return hpo_stack


@pytest.fixture(scope="module")
def H(S):
    return S.hpo


def test_exports_every_declared_symbol(S):
    src = open(os.path.join(ROOT, "include", "hpo_stack.h")).read()
    names = re.findall(r"^(?:hpo_status|const char\*|int32_t)\s+(hpo_\w+)\(", src, re.M)
    assert set(names) == set(S.SIGNATURES)
    for n in names:
        assert hasattr(S.load(), n), n


def test_struct_layouts(S):
    assert ctypes.sizeof(S.c_stack) == 56
    assert ctypes.sizeof(S.hpo_rms_cfg) == 40
    assert ctypes.sizeof(S.c_qk) == 2 * 8 + 6 * 4 + 11 * 8 + 4 * 8 + 8
    assert ctypes.sizeof(S.c_clip_weight) == 40


def stack(S, dtype=1, batch=2, rows=4, cols=8, bs=None, rs=None, data=P, reserved=0):
    rs = cols if rs is None else rs
    return S.c_stack(data, batch, rows, cols, rows * rs if bs is None else bs, rs, dtype, reserved)


def ortho(S, H, G, out, M=None, cfg=None, inv=1.0, max_norm=0.0, d_norm=None, ws=P, nbytes=1 << 40):
    cfg = H.make_muon_cfg() if cfg is None else cfg
    st = S.load().hpo_orthogonalize(ctypes.byref(G) if G else None, ctypes.byref(M) if M else None,
                                    ctypes.byref(out) if out else None, ctypes.byref(cfg), inv, max_norm, d_norm, None,
                                    ws, nbytes, None)
    return st, H.hpo_last_error()


def test_orthogonalize_refusals(S, H):
    good, out = stack(S), stack(S, dtype=0)
    bad = [
        (dict(G=None, out=out), "NULL"),
        (dict(G=good, out=None), "NULL"),
        (dict(G=stack(S, batch=-1), out=out), "negative"),
        (dict(G=stack(S, rows=H.HPO_MUON_MAX_DIM + 1), out=out), "too large"),
        (dict(G=stack(S, batch=65536), out=stack(S, dtype=0, batch=65536)), "too large"),
        (dict(G=stack(S, data=0), out=out), "non-NULL"),
        (dict(G=stack(S, data=P + 2), out=out), "aligned"),
        (dict(G=stack(S, rs=7), out=out), "stride"),
        (dict(G=stack(S, bs=0), out=out), "stride"),
        (dict(G=stack(S, bs=16), out=out), "overlap"),
        (dict(G=stack(S, bs=-8), out=out), "strides"),
        (dict(G=stack(S, reserved=1), out=out), "reserved"),
        (dict(G=good, out=stack(S, dtype=0, cols=9)), "out is"),
        (dict(G=good, out=out, M=stack(S, rows=5)), "momentum is"),
        (dict(G=good, out=out, inv=float("inf")), "inv_scale"),
        (dict(G=good, out=out, max_norm=float("nan")), "NaN"),
        (dict(G=good, out=out, max_norm=1.0), "d_norm"),
        (dict(G=good, out=out, ws=0), "workspace"),
        (dict(G=good, out=out, ws=P + 128), "256-byte"),
        (dict(G=good, out=out, nbytes=16), "below"),
        (dict(G=good, out=out, cfg=H.make_muon_cfg(ns_steps=0)), "ns_steps"),
        (dict(G=good, out=out, cfg=H.make_muon_cfg(ns_eps=-1.0)), "ns_eps"),
        (dict(G=good, out=out, cfg=H.make_muon_cfg(ns_steps=2, ns_coeffs=[(9.0, 0.0, 9e9)] * 2)), "ns_coeffs"),
        (dict(G=good, out=out, cfg=H.make_muon_cfg(ns_steps=16, ns_coeffs=[(4.0, 0.0, 0.0)] * 16)), "ns_coeffs"),
        (dict(G=good, out=out, M=good, cfg=H.make_muon_cfg(momentum=1.0)), "momentum"),
    ]
    for kw, word in bad:
        st, msg = ortho(S, H, **kw)
        assert st == H.HPO_EINVAL and word in msg, (kw, st, msg)
    for kw in (dict(G=stack(S, dtype=2), out=out), dict(G=good, out=stack(S, dtype=1)),
               dict(G=good, out=out, M=stack(S, dtype=0)), dict(G=stack(S, dtype=16), out=out)):
        st, msg = ortho(S, H, **kw)
        assert st == H.HPO_EDTYPE, (kw, msg)


def test_interleaved_rows_are_accepted_and_empty_stacks_do_nothing(S, H):
    """The heads of an output projection lie side by side in every row; the
    call gets as far as the (too small) workspace."""
    inter = stack(S, batch=4, rows=6, cols=8, bs=8, rs=32)
    st, msg = ortho(S, H, inter, stack(S, dtype=0, batch=4, rows=6, cols=8), nbytes=0)
    assert st == H.HPO_EINVAL and "below" in msg
    for kw in (dict(batch=0), dict(rows=0), dict(cols=0)):
        st, _ = ortho(S, H, stack(S, data=0, **kw), stack(S, dtype=0, data=0, **kw), ws=0, nbytes=0)
        assert st == H.HPO_OK
    out = ctypes.c_int64(7)
    assert S.load().hpo_orthogonalize_workspace(0, 5, 5, ctypes.byref(out)) == H.HPO_OK and out.value == 0
    assert S.load().hpo_orthogonalize_workspace(-1, 5, 5, ctypes.byref(out)) == H.HPO_EINVAL
    assert S.load().hpo_orthogonalize_workspace(1, 5, 5, None) == H.HPO_EINVAL


def rms(S, H, O, W, param=None, scales=None, v=P, cfg=None, ws=P, nbytes=1 << 40):
    cfg = S.make_rms_cfg(0.02) if cfg is None else cfg
    st = S.load().hpo_rms_update(ctypes.byref(O), ctypes.byref(W), v, ctypes.byref(param) if param else None, scales,
                                 ctypes.byref(cfg), None, ws, nbytes, None)
    return st, H.hpo_last_error()


def test_rms_update_refusals(S, H):
    O, W = stack(S, dtype=0), stack(S)
    nan = float("nan")
    bad = [
        (dict(O=stack(S, dtype=0, rows=5), W=W), "O is"),
        (dict(O=O, W=W, param=stack(S, dtype=0, cols=7)), "param is"),
        (dict(O=O, W=W, param=stack(S, dtype=16)), "d_scales"),
        (dict(O=O, W=W, param=stack(S, dtype=0), scales=P), "8-bit"),
        (dict(O=O, W=W, scales=P), "d_scales"),
        (dict(O=O, W=W, v=None), "d_v"),
        (dict(O=O, W=W, v=P + 2), "d_v"),
        (dict(O=O, W=W, ws=None), "workspace"),
        (dict(O=O, W=W, ws=P + 4), "8-byte"),
        (dict(O=O, W=W, nbytes=8), "below"),
        (dict(O=O, W=W, cfg=S.make_rms_cfg(nan)), "finite"),
        (dict(O=O, W=W, cfg=S.make_rms_cfg(0.1, target_rms=float("inf"))), "finite"),
        (dict(O=O, W=W, cfg=S.make_rms_cfg(0.1, beta2=1.0)), "beta2"),
        (dict(O=O, W=W, cfg=S.make_rms_cfg(0.1, eps=-1e-8)), "eps"),
        (dict(O=stack(S, dtype=0, batch=16, rows=H.HPO_MUON_MAX_DIM), W=stack(S, batch=16, rows=H.HPO_MUON_MAX_DIM)),
         "rows in all"),
    ]
    for kw, word in bad:
        st, msg = rms(S, H, **kw)
        assert st == H.HPO_EINVAL and word in msg, (kw, st, msg)
    for kw in (dict(O=stack(S, dtype=2), W=W), dict(O=O, W=stack(S, dtype=0)), dict(O=O, W=W, param=stack(S, dtype=1))):
        assert rms(S, H, **kw)[0] == H.HPO_EDTYPE
    e = lambda d: stack(S, dtype=d, rows=0, data=0)
    assert rms(S, H, e(0), e(1), v=None, ws=None, nbytes=0)[0] == H.HPO_OK


def qk(S, **kw):
    d = dict(q=P, k=P, dtype=0, batch=2, heads=4, kv_heads=2, head_dim=64, causal=1, window=-1, seq_q=16, seq_k=16,
             max_seqlen_q=0, max_seqlen_k=0, q_stride_batch=4096, q_stride_token=256, q_stride_head=64,
             k_stride_batch=2048, k_stride_token=128, k_stride_head=64, scale=0.125)
    d.update(kw)
    return S.c_qk(**d)


def test_qk_max_refusals(S, H):
    L = S.load()
    bad = [
        (dict(batch=-1), "negative"), (dict(seq_k=-1), "negative"), (dict(heads=5), "multiple"),
        (dict(kv_heads=0), "multiple"), (dict(head_dim=0), "head_dim"), (dict(head_dim=257), "head_dim"),
        (dict(causal=2), "causal"), (dict(window=-2), "window"), (dict(window=3, causal=0), "window"),
        (dict(scale=0.0), "scale"), (dict(scale=float("inf")), "scale"), (dict(scale=-1.0), "scale"),
        (dict(scale=float("nan")), "scale"), (dict(cu_seqlens_q=P), "together"),
        (dict(cu_seqlens_q=P, cu_seqlens_k=P, seqlens_q=P), "padded"),
        (dict(cu_seqlens_q=P, cu_seqlens_k=P, max_seqlen_q=-1), "max_seqlen"),
        (dict(cu_seqlens_q=P + 2, cu_seqlens_k=P), "4-byte"),
        (dict(q_stride_token=-1), "strides"), (dict(k_stride_token=(1 << 23) + 1), "k_stride_token"),
        (dict(seq_q=(1 << 30) + 1), "2^30"), (dict(reserved=1), "reserved"), (dict(q=0), "q and k"),
        (dict(k=P + 1), "q and k"), (dict(batch=65535, heads=65534, seq_q=1 << 20), "tiles"),
    ]
    for kw, word in bad:
        st = L.hpo_qk_max_logits(ctypes.byref(qk(S, **kw)), 0, P, None)
        msg = H.hpo_last_error()
        assert st == H.HPO_EINVAL and word in msg, (kw, st, msg)
    assert L.hpo_qk_max_logits(ctypes.byref(qk(S, dtype=1)), 0, P, None) == H.HPO_EDTYPE
    assert L.hpo_qk_max_logits(ctypes.byref(qk(S)), 2, P, None) == H.HPO_EINVAL
    assert L.hpo_qk_max_logits(ctypes.byref(qk(S)), 0, None, None) == H.HPO_EINVAL
    assert L.hpo_qk_max_logits(None, 0, P, None) == H.HPO_EINVAL
    assert L.hpo_qk_max_logits(ctypes.byref(qk(S, heads=0)), 0, None, None) == H.HPO_OK
    # nothing to see and nothing to initialise: no launch
    assert L.hpo_qk_max_logits(ctypes.byref(qk(S, batch=0)), 1, P, None) == H.HPO_OK


def clip(S, H, *weights, heads=4, kv_heads=2, tau=100.0, n=None, d_max=P):
    arr = (S.c_clip_weight * max(1, len(weights)))()
    for k, (m, p, s, power, group) in enumerate(weights):
        arr[k].master = ctypes.pointer(m) if m else None
        if p:
            arr[k].param = ctypes.pointer(p)
        arr[k].d_scales, arr[k].power, arr[k].per_group = s, power, group
    st = S.load().hpo_qk_clip(d_max, heads, kv_heads, tau, arr, len(weights) if n is None else n, None, None)
    return st, H.hpo_last_error()


def test_qk_clip_refusals(S, H):
    W = stack(S, batch=4)
    bad = [
        (((W, None, None, 0.5, 0),), dict(heads=0), "heads"),
        (((W, None, None, 0.5, 0),), dict(kv_heads=3), "multiple"),
        (((W, None, None, 0.5, 0),), dict(tau=0.0), "tau"),
        (((W, None, None, 0.5, 0),), dict(tau=float("nan")), "tau"),
        (((W, None, None, 0.5, 0),), dict(d_max=None), "d_max"),
        ((), dict(n=0), "n_weights"),
        (((W, None, None, 0.5, 0),) * 9, {}, "n_weights"),
        (((stack(S, batch=3), None, None, 0.5, 0),), {}, "per head"),
        (((W, None, None, -0.5, 0),), {}, "power"),
        (((W, None, None, float("nan"), 0),), {}, "power"),
        (((W, None, None, 0.5, 2),), {}, "per_group"),
        (((None, None, None, 0.5, 0),), {}, "NULL"),
        (((W, None, None, 0.5, 0), (W, None, None, 1.0, 1)), {}, "twice"),
        (((W, stack(S, dtype=16, batch=4), None, 0.5, 0),), {}, "d_scales"),
        (((W, stack(S, dtype=0, batch=4, cols=9), None, 0.5, 0),), {}, "param is"),
    ]
    for ws, kw, word in bad:
        st, msg = clip(S, H, *ws, **kw)
        assert st == H.HPO_EINVAL and word in msg, (kw, st, msg)
    assert clip(S, H, (stack(S, dtype=0, batch=4), None, None, 0.5, 0))[0] == H.HPO_EDTYPE
    assert clip(S, H, (stack(S, batch=4, cols=0, data=0), None, None, 0.5, 0))[0] == H.HPO_OK


def test_host_tensors_are_refused(S, H):
    """Without a GPU, and with one, a host tensor never reaches the library."""
    W = torch.zeros(2, 4, 8)
    for call in (lambda: S.hpo_orthogonalize(W, W.bfloat16(), H.make_muon_cfg(), None),
                 lambda: S.hpo_rms_update(W, W, None, S.make_rms_cfg(0.1), None),
                 lambda: S.hpo_qk_max_logits(torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(2), 1.0),
                 lambda: S.hpo_qk_clip(torch.zeros(2), 2, 100.0, [S.ClipWeight(W, 2, 0.5)])):
        with pytest.raises(ValueError):
            call()
