"""References in binary64 for the model operators, and the arithmetic their
tolerances come from."""
from __future__ import annotations

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step, relative
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}   # smallest subnormal


def mx_values(q, byte):
    """What 8-bit values and scale bytes stand for, in binary64: [..., cols]."""
    cols = q.shape[-1]
    f = torch.exp2(byte.cpu().view(torch.uint8).double() - 127.0)
    f = torch.where(byte.cpu().view(torch.uint8) == 255, torch.nan, f)
    return q.cpu().float().double() * f.repeat_interleave(32, -1)[..., :cols]


def embedding(ids, w, scale, first):
    """Rows of w (fp32) by id, times fp32(scale), rounded to fp32."""
    at = ids.long().reshape(-1) - first
    ok = (at >= 0) & (at < w.shape[0])
    rows = torch.zeros(at.numel(), w.shape[1])
    rows[ok] = w[at[ok]] * torch.tensor(scale, dtype=torch.float32)
    return rows


def embedding_grad(ids, dy, grad, scale, first):
    """(result, tolerance) in binary64.  A row of n tokens is n - 1 additions of fp32 in some order, each
    off by half a step of a partial sum that the magnitudes' sum bounds (parts of it start from 0, which
    adds nothing); then the product, the sum with G and the rounding to G's type."""
    at = ids.long().reshape(-1) - first
    ok = (at >= 0) & (at < grad.shape[0])
    d = dy.double().reshape(at.numel(), -1)
    total = torch.zeros(grad.shape, dtype=torch.float64)
    size = torch.zeros_like(total)
    count = torch.zeros(grad.shape[0], dtype=torch.float64)
    total.index_add_(0, at[ok], d[ok])
    size.index_add_(0, at[ok], d[ok].abs())
    count.index_add_(0, at[ok], torch.ones(int(ok.sum()), dtype=torch.float64))
    s = float(torch.tensor(scale, dtype=torch.float32))
    res = grad.double() + s * total
    h = HALF[torch.float32]
    tol = abs(s) * (count[:, None] + 2) * h * size * 1.01 + h * res.abs() + TINY[torch.float32] * count[:, None]
    if grad.dtype != torch.float32:
        tol = tol * 1.01 + HALF[grad.dtype] * res.abs() + TINY[grad.dtype]
    return res, torch.where(count[:, None] > 0, tol, 0.0), count > 0


def product_tolerance(size, k, result, dtype, scale=1.0, before=None):
    """Products of 8-bit and 16-bit values are exact in fp32; each of k additions is off by at most a step of
    a partial sum (the matrix cores may cut instead of rounding), which `size`, the sum of the magnitudes, bounds; then
    the product with scale, the sum with what was there, and the rounding to the result's type."""
    h = HALF[torch.float32]
    tol = abs(scale) * (k + 2) * 2 * h * size + 2 * h * result.abs() + TINY[torch.float32]
    if before is not None:
        tol = tol + h * before.abs()
    if dtype != torch.float32:
        tol = tol * 1.01 + HALF[dtype] * result.abs() + TINY[dtype]
    return tol


def aligned_cut(a, b):
    """What hpo_mx8_linear's matrix instructions may cut off a result: of the 64 products that one of them adds, each
    loses less than 2^-13 of the largest, which the largest magnitudes of the two rows' 64 elements bound."""
    def top(x):
        c = x.shape[-1]
        n = -(-c // 64)
        y = torch.zeros(*x.shape[:-1], n * 64, dtype=torch.float64, device=x.device)
        y[..., :c] = x.abs()
        return y.unflatten(-1, (n, 64)).amax(-1)
    return 64 * 2.0 ** -13 * (top(a) @ top(b).mT.contiguous())


def matmul64(a, b):
    """a @ b and |a| @ |b| in binary64, batched, on whatever device they are."""
    a, b = a.double().contiguous(), b.double().contiguous()
    return a @ b, a.abs() @ b.abs()


def check(got, want, tol, tag=""):
    got = got.detach().double().cpu()
    want, tol = want.cpu(), tol.cpu()
    assert got.shape == want.shape, (tag, got.shape, want.shape)
    same = (got == want) | (got.isnan() & want.isnan())
    d = torch.where(same, 0.0, (got - want).abs())
    bad = ~(same | (d <= tol))
    part = (torch.where(tol > 0, d / tol, 0.0)).nan_to_num(0).max() if d.numel() else torch.zeros(())
    print(f"[model] {tag}: largest share of the tolerance {float(part):.3f}", flush=True)
    assert not bool(bad.any()), f"{tag}: {int(bad.sum())} of {bad.numel()} off, at {bad.nonzero()[:4].tolist()}: " \
                                f"{got[bad][:4].tolist()} for {want[bad][:4].tolist()}"
