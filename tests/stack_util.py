"""References in binary64 for the stack operators, and the arithmetic their
tolerances come from."""
from __future__ import annotations

import math

import numpy as np
import torch

ABC = (3.4445, -4.7750, 2.0315)
HALF32 = 2.0 ** -24      # half a step of fp32, relative
HALF_BF16 = 2.0 ** -8


def ns_exact(g, steps=5, coeffs=None, eps=1e-7):
    """Newton-Schulz of one matrix in binary64 (CPU)."""
    x = g.double()
    x = x / (torch.linalg.vector_norm(x) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for k in range(steps):
        a, b, c = coeffs[k] if coeffs is not None else ABC
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.T if tall else x


def ns_emulated(g, steps=5, coeffs=None, eps=1e-7):
    """The documented arithmetic: fp16 operands (near the top of fp16's range:
    relative roundings of 2^-11), the term a X from X with what its rounding
    lost, everything else exact."""
    def r16(t):
        m = float(t.abs().max())
        s = 2.0 ** (14 - math.ceil(math.log2(m))) if m > 0 else 1.0
        return (t * s).half().double() / s

    x = g.double()
    x = x / (torch.linalg.vector_norm(x) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for k in range(steps):
        a, b, c = coeffs[k] if coeffs is not None else ABC
        h = r16(x)
        A = r16(h @ h.T)
        x = a * (x if k + 1 < steps else h) + r16(b * A + c * (A @ A)) @ h
    return x.T if tall else x


def ns_tolerance(g, steps=5, coeffs=None, eps=1e-7):
    """(exact result, allowed relative distance in the Frobenius norm).  The
    kernel rounds where the emulation rounds; its sums are fp32, so some of
    its roundings fall the other way, each no further off than the rounding
    itself: twice the emulation's distance, plus fp32's own share, plus the
    half step of the bf16 result."""
    e = ns_exact(g, steps, coeffs, eps)
    n = float(torch.linalg.vector_norm(e))
    if n == 0.0:
        return e, 0.0
    d = float(torch.linalg.vector_norm(ns_emulated(g, steps, coeffs, eps) - e)) / n
    amplify = 4.0 ** steps   # |a s + b s^3 + c s^5| grows a small s by a < 4 a step
    return e, 2.0 * d + amplify * HALF32 * math.sqrt(max(g.shape)) + HALF_BF16


def mx_reference(w):
    """(e4m3 values, scale bytes) of the rows of w (fp32, CPU, [..., cols])."""
    cols = w.shape[-1]
    nb = -(-cols // 32)
    x = torch.zeros(*w.shape[:-1], nb * 32, dtype=torch.float64)
    x[..., :cols] = w.double()
    x = x.view(*w.shape[:-1], nb, 32)
    bad = ~torch.isfinite(x).all(-1)
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    e = torch.where(amax > 0, torch.frexp(torch.where(amax > 0, amax, 1.0))[1].double() - 9, -127.0).clamp(min=-127.0)
    y = (x * torch.exp2(-e)[..., None]).clamp(-448.0, 448.0)
    q = y.float().to(torch.float8_e4m3fn).view(torch.uint8)
    q = torch.where(bad[..., None], torch.tensor(0x7F, dtype=torch.uint8), q)
    byte = torch.where(bad, 255.0, e + 127.0).to(torch.uint8)
    return q.reshape(*w.shape[:-1], nb * 32)[..., :cols], byte


def bits(t):
    n = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
    return t.detach().cpu().contiguous().view(n)


def check_weight(master, param, scales=None):
    """The model weight is its own master's rounding, bit for bit."""
    w = master.detach().cpu().contiguous()
    if param.dtype == torch.bfloat16:
        assert torch.equal(bits(param), bits(w.bfloat16()))
        return
    q, byte = mx_reference(w)
    assert torch.equal(scales.detach().cpu().view(torch.uint8).reshape(byte.shape), byte)
    # -0 and 0 stand for the same weight
    got = bits(param)
    same = (got == q) | (((got | q) & 0x7F) == 0)
    assert bool(same.all()), f"{int((~same).sum())} of {same.numel()} values differ"


def rms_reference(O, W, v, lr, wd, beta2, eps, target):
    """(W, v, u) in binary64 for [batch, rows, cols] tensors on the CPU."""
    o, w = O.double(), W.double()
    ms = o.square().mean(-1)
    v = beta2 * v.double() + (1 - beta2) * ms
    den = v.sqrt() + eps
    r = torch.where(den > 0, 1.0 / den, 0.0)
    rows, cols = o.shape[-2:]
    n = (cols * ms * r * r).sum(-1).sqrt()
    s = torch.where(n > 0, lr * target * math.sqrt(rows * cols) / n, 0.0)
    u = (s[:, None] * r)[..., None] * o
    return w * (1 - lr * wd) - u, v, u


def rms_terms(cols):
    """fp32 additions behind one lane's sum of squares, at most: relative error of
    a mean square is that many half steps (all terms are positive)."""
    return 4 * math.ceil(cols / 256) + 2


def logits_reference(q, k, scale, causal, window, lens=None):
    """(max per head, largest sum of |products| per head) over a list of
    (queries [n, h, d], keys [m, hk, d]) in binary64."""
    h, hk = q[0].shape[1], k[0].shape[1]
    best = torch.full((h,), -math.inf, dtype=torch.float64)
    size = torch.zeros(h, dtype=torch.float64)
    for x, y in zip(q, k):
        n, m = x.shape[0], y.shape[0]
        if n == 0 or m == 0:
            continue
        at = torch.arange(n)[:, None] + m - n
        j = torch.arange(m)
        ok = torch.ones(n, m, dtype=torch.bool)
        if causal:
            ok = j <= at
            if window >= 0:
                ok &= j >= at - window
        if not bool(ok.any()):
            continue
        for i in range(h):
            a, b = x[:, i].double(), y[:, i // (h // hk)].double()
            s = torch.where(ok, (a @ b.T) * scale, -math.inf)
            # a seen NaN wins; matmul spreads a NaN of one row or key only over its own logits
            t = s[ok]
            best[i] = torch.nan if bool(t.isnan().any() | best[i].isnan()) else torch.maximum(best[i], t.max())
            fin = torch.where(ok, a.abs().nan_to_num(0, 0, 0) @ b.abs().nan_to_num(0, 0, 0).T, 0.0)
            size[i] = torch.maximum(size[i], fin.max())
    return best, size * scale


def logits_tolerance(dim, size):
    """Products of 16-bit values are exact in fp32; each of dim additions rounds by
    at most a step of the partial sum (the matrix cores may cut instead of
    rounding), then the product with scale."""
    return (dim + 2) * 2 * HALF32 * size


def np_of(t):
    return t.detach().float().cpu().numpy().astype(np.float64)
