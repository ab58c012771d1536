"""Cases of the stack operators: orthogonalised updates, the row-normalised
master update, the largest attention logit of each head and the clip of the
query / key weights by it.

A case is a dict of plain values with an "op":
  ortho   Newton-Schulz of a stack of gradient matrices (momentum folded in)
  update  row-normalised update of the fp32 master and the model weight
  logits  largest attention logit of each head
  clip    rescaling of the query / key rows of the heads over the threshold

`run` computes the plain form with elementary torch operations in fp32, or,
where `own` is true, calls the library.  `exact` evaluates the definitions in
binary64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
F32, BF16, F16, F64 = torch.float32, torch.bfloat16, torch.float16, torch.float64
DTYPES = {"fp32": F32, "bf16": BF16, "fp16": F16}
NS_ABC = (3.4445, -4.7750, 2.0315)
NS_EPS = 1e-7
MU = 0.95
LR, WD, BETA2, ROW_EPS, TARGET = 0.02, 0.1, 0.95, 1e-8, 0.2
TAU = 100.0
MX_BLOCK = 32          # elements that share one power-of-two scale
E4M3_MAX = 448.0


def listed():
    return [
        # A query projection's gradient seen as 32 heads of 128 rows, each orthogonalised on its own, with momentum.
        {"name": "ortho_heads", "op": "ortho", "batch": 32, "rows": 128, "cols": 4096, "dtype": "fp32", "pad": 0,
         "momentum": True},
        # A stack of expert matrices, taller than wide, bf16 gradients.
        {"name": "ortho_experts", "op": "ortho", "batch": 16, "rows": 2048, "cols": 1024, "dtype": "bf16", "pad": 0,
         "momentum": False},
        # Odd sizes in a padded buffer: nothing is a multiple of a tile or of a vector.
        {"name": "ortho_odd", "op": "ortho", "batch": 3, "rows": 1000, "cols": 333, "dtype": "fp32", "pad": 7,
         "momentum": True},
        # An MLP matrix of an 8B model.
        {"name": "ortho_mlp", "op": "ortho", "batch": 1, "rows": 4096, "cols": 14336, "dtype": "fp32", "pad": 0,
         "momentum": False},
        # The same matrix's master update with a bf16 model weight.
        {"name": "update_mlp", "op": "update", "batch": 1, "rows": 4096, "cols": 14336, "o": "bf16", "param": "bf16",
         "pad": 0},
        # Expert stack whose model weights are held in 8 bits.
        {"name": "update_experts_mx8", "op": "update", "batch": 16, "rows": 1024, "cols": 2048, "o": "bf16",
         "param": "mx8", "pad": 0},
        # A small odd matrix in 8 bits: launches are what counts.
        {"name": "update_small", "op": "update", "batch": 1, "rows": 129, "cols": 257, "o": "fp32", "param": "mx8",
         "pad": 3},
        # One training sequence of 8192 tokens, causal, 32 query heads over 8 key heads.
        {"name": "logits_8k", "op": "logits", "batch": 1, "seq_q": 8192, "seq_k": 8192, "heads": 32, "kv_heads": 8,
         "dim": 128, "dtype": "bf16", "causal": True, "window": -1, "packed": False},
        # Packed sequences of uneven lengths, one of them empty, with a sliding window.
        {"name": "logits_packed", "op": "logits", "batch": 7, "seq_q": 2048, "seq_k": 2048, "heads": 16,
         "kv_heads": 16, "dim": 64, "dtype": "fp16", "causal": True, "window": 512, "packed": True},
        # A short micro-batch without a mask, odd length, wide heads.
        {"name": "logits_short", "op": "logits", "batch": 2, "seq_q": 333, "seq_k": 333, "heads": 8, "kv_heads": 8,
         "dim": 192, "dtype": "bf16", "causal": False, "window": -1, "packed": False},
        # One layer's query and key weights, half of the heads over the threshold.
        {"name": "clip_layer", "op": "clip", "heads": 32, "kv_heads": 8, "dim": 128, "cols": 4096, "over": 16,
         "param": "bf16"},
        # Wide layer early in training: about one head in eight over the threshold, weights held in 8 bits.
        {"name": "clip_wide_mx8", "op": "clip", "heads": 64, "kv_heads": 64, "dim": 128, "cols": 7168, "over": 8,
         "param": "mx8"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ortho", "update", "logits", "clip"])
    if op == "ortho":
        while True:
            b, r, c = _log_int(rng, 1, 48), _log_int(rng, 1, 6000), _log_int(rng, 8, 9000)
            if 1 <= b * r * c <= 40_000_000 and b * r * c * min(r, c) <= 60_000_000_000:
                break
        return {"op": op, "batch": b, "rows": r, "cols": c, "dtype": rng.choice(["fp32", "bf16"]),
                "pad": rng.choice([0, 0, 1, 5, 8]), "momentum": rng.random() < 0.5}
    if op == "update":
        while True:
            b, r, c = _log_int(rng, 1, 48), _log_int(rng, 1, 8000), _log_int(rng, 1, 16000)
            if 64 <= b * r * c <= 40_000_000:
                break
        return {"op": op, "batch": b, "rows": r, "cols": c, "o": rng.choice(["bf16", "fp32"]),
                "param": rng.choice(["bf16", "mx8", "none"]), "pad": rng.choice([0, 0, 1, 8])}
    if op == "logits":
        while True:
            b, hk = _log_int(rng, 1, 8), rng.choice([1, 2, 4, 8])
            h, d = hk * rng.choice([1, 2, 4]), rng.choice([40, 64, 80, 96, 128, 192, 256, 57])
            sq = _log_int(rng, 1, 6000)
            sk = sq if rng.random() < 0.6 else _log_int(rng, 1, 6000)
            if 64 <= b * h * sq * sk <= 600_000_000:
                break
        causal = rng.random() < 0.6
        return {"op": op, "batch": b, "seq_q": sq, "seq_k": sk, "heads": h, "kv_heads": hk, "dim": d,
                "dtype": rng.choice(["bf16", "fp16"]), "causal": causal,
                "window": _log_int(rng, 1, 4000) if causal and rng.random() < 0.4 else -1,
                "packed": rng.random() < 0.5}
    hk = rng.choice([1, 2, 4, 8, 16])
    h = hk * rng.choice([1, 2, 4])
    return {"op": op, "heads": h, "kv_heads": hk, "dim": rng.choice([64, 96, 128, 77]),
            "cols": _log_int(rng, 64, 7000), "over": rng.randint(0, h), "param": rng.choice(["bf16", "mx8", "none"])}


# ---------------------------------------------------------------------------
# inputs: from the seed alone
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _padded(x, pad):
    """x as a view of a buffer whose rows are `pad` elements longer."""
    if pad == 0:
        return x.contiguous()
    buf = torch.zeros(*x.shape[:-1], x.shape[-1] + pad, dtype=x.dtype, device=x.device)
    buf[..., : x.shape[-1]] = x
    return buf[..., : x.shape[-1]]


def _gradient(g, b, r, c):
    """Weight gradients: a few strong directions over a noise floor, at a gradient's usual size."""
    k = max(1, min(r, c) // 16)
    u = torch.randn(b, r, k, generator=g, device=DEV) * torch.logspace(0.5, -0.5, k, device=DEV)
    return (u @ torch.randn(b, k, c, generator=g, device=DEV) / math.sqrt(k)
            + 0.3 * torch.randn(b, r, c, generator=g, device=DEV)) * 1e-3


def _lengths(case):
    """Lengths of a packed batch, from the case alone: uneven, the second one empty."""
    r = random.Random("%(batch)d %(seq_q)d %(seq_k)d %(heads)d" % case)
    lq = [r.randint(1, case["seq_q"]) for _ in range(case["batch"])]
    lk = [max(1, min(case["seq_k"], n)) if case["seq_q"] == case["seq_k"] else r.randint(1, case["seq_k"]) for n in lq]
    if case["batch"] > 1:
        lq[1] = lk[1] = 0
    return lq, lk


def _inputs(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "ortho":
        b, r, c = case["batch"], case["rows"], case["cols"]
        s = {"G": _padded(_gradient(g, b, r, c).to(DTYPES[case["dtype"]]), case["pad"])}
        if case["momentum"]:
            s["M"] = _padded(10.0 * _gradient(g, b, r, c), case["pad"])
        return s
    if op == "update":
        b, r, c = case["batch"], case["rows"], case["cols"]
        o = torch.randn(b, r, c, generator=g, device=DEV) * torch.exp(0.3 * torch.randn(b, r, 1, generator=g, device=DEV))
        return {"O": _padded((o / math.sqrt(max(r, c))).to(DTYPES[case["o"]]), case["pad"]),
                "W": _padded(0.02 * torch.randn(b, r, c, generator=g, device=DEV), case["pad"]),
                "v": torch.rand(b, r, generator=g, device=DEV) / max(r, c)}
    if op == "logits":
        h, hk, d, dt = case["heads"], case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
        if case["packed"]:
            lq, lk = _lengths(case)
            q = torch.randn(sum(lq), h, d, generator=g, device=DEV).to(dt)
            k = torch.randn(sum(lk), hk, d, generator=g, device=DEV).to(dt)
            cum = lambda n: torch.tensor([0] + n, dtype=torch.int32, device=DEV).cumsum(0, dtype=torch.int32)
            return {"q": q, "k": k, "cu_q": cum(lq), "cu_k": cum(lk)}
        b = case["batch"]
        return {"q": torch.randn(b, case["seq_q"], h, d, generator=g, device=DEV).to(dt),
                "k": torch.randn(b, case["seq_k"], hk, d, generator=g, device=DEV).to(dt)}
    h, hk, d, c = case["heads"], case["kv_heads"], case["dim"], case["cols"]
    smax = 20.0 + 70.0 * torch.rand(h, generator=g, device=DEV)
    over = torch.randperm(h, generator=g, device=DEV)[: case["over"]]
    smax[over] = 102.0 + 50.0 * torch.rand(case["over"], generator=g, device=DEV)
    return {"smax": smax, "Wq": 0.02 * torch.randn(h * d, c, generator=g, device=DEV),
            "Wk": 0.02 * torch.randn(hk * d, c, generator=g, device=DEV)}


def _mx_quantize(w):
    """(e4m3 values, e8m0 scales) of w's rows in blocks of 32: scale 2^(floor(log2 amax) - 8), values rounded to
    nearest even and saturated at 448."""
    c = w.shape[-1]
    nb = -(-c // MX_BLOCK)
    x = torch.nn.functional.pad(w, (0, nb * MX_BLOCK - c)).unflatten(-1, (nb, MX_BLOCK))
    amax = x.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 1 - 8, -127).clamp(-127, 127)
    q = torch.ldexp(x, -e.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX)
    return q.flatten(-2)[..., :c], e


def _mx_encode(w):
    q, e = _mx_quantize(w)
    return q.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _weight_out(w, kind):
    """Buffers of a model weight that holds round(w) already: {} / {"p"} / {"p", "s"}."""
    if kind == "bf16":
        return {"p": w.to(BF16).contiguous()}
    if kind == "mx8":
        p, s = _mx_encode(w)
        return {"p": p.contiguous(), "s": s.contiguous()}
    return {}


def prepare(case, seed):
    s = {"case": case, **_inputs(case, seed)}
    op = case["op"]
    if op == "ortho":
        b, r, c = case["batch"], case["rows"], case["cols"]
        s["out"] = torch.empty(b, r, c, dtype=BF16, device=DEV)
        s["ws"] = None
        if own:
            from mixed_precision_optimizer_amd import hpo, hpo_stack
            s["cfg"] = hpo.make_muon_cfg(momentum=MU)
            s["ws"] = torch.empty(hpo_stack.hpo_orthogonalize_workspace(s["G"], s["cfg"], s.get("M")),
                                  dtype=torch.uint8, device=DEV)
    elif op == "update":
        s.update(_weight_out(s["W"], case["param"]))
        if own:
            from mixed_precision_optimizer_amd import hpo_stack
            s["cfg"] = hpo_stack.make_rms_cfg(lr=LR, weight_decay=WD, beta2=BETA2, eps=ROW_EPS, target_rms=TARGET)
            s["ws"] = torch.empty(hpo_stack.hpo_rms_update_workspace(s["W"]), dtype=torch.uint8, device=DEV)
    elif op == "logits":
        s["smax"] = torch.empty(case["heads"], dtype=F32, device=DEV)
        s["scale"] = 1.0 / math.sqrt(case["dim"])
        if case["packed"]:
            lq, lk = _lengths(case)
            s["max_q"], s["max_k"] = max(lq), max(lk)
    else:
        for w in ("q", "k"):
            for n, t in _weight_out(s["W" + w], case["param"]).items():
                s[n + w] = t
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return {"ortho": _run_ortho, "update": _run_update, "logits": _run_logits, "clip": _run_clip}[s["case"]["op"]](s)


def _run_ortho(s):
    if own:
        from mixed_precision_optimizer_amd import hpo_stack
        hpo_stack.hpo_orthogonalize(s["G"], s["out"], s["cfg"], s["ws"], momentum=s.get("M"))
        return {"out": s["out"], "M": s["M"]} if "M" in s else {"out": s["out"]}
    g = s["G"].float()
    if "M" in s:
        s["M"].mul_(MU).add_(g)
        g = g + MU * s["M"]
    x = g / (g.square().sum((-2, -1), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT.contiguous()
    a, b, c = NS_ABC
    x = _ns_step(_ns_step(_ns_step(_ns_step(_ns_step(x, a, b, c), a, b, c), a, b, c), a, b, c), a, b, c)
    s["out"].copy_(x.mT if tall else x)
    return {"out": s["out"], "M": s["M"]} if "M" in s else {"out": s["out"]}


def _ns_step(x, a, b, c):
    gram = x @ x.mT
    return a * x + (b * gram + c * (gram @ gram)) @ x


def _store(w, s, suffix=""):
    """The model weight of master w, rounded into its buffers; what the pass returns of it."""
    out = {}
    if "s" + suffix in s:
        p, e = _mx_encode(w)
        s["p" + suffix].copy_(p)
        s["s" + suffix].copy_(e)
        out["s" + suffix] = s["s" + suffix]
    elif "p" + suffix in s:
        s["p" + suffix].copy_(w)
    if "p" + suffix in s:
        out["p" + suffix] = s["p" + suffix]
    return out


def _held(s, suffix=""):
    return {n + suffix: s[n + suffix] for n in ("p", "s") if n + suffix in s}


def _run_update(s):
    if own:
        from mixed_precision_optimizer_amd import hpo_stack
        hpo_stack.hpo_rms_update(s["O"], s["W"], s["v"], s["cfg"], s["ws"], param=s.get("p"), scales=s.get("s"))
        return {"W": s["W"], "v": s["v"], **_held(s)}
    o, w, v = s["O"].float(), s["W"], s["v"]
    rows, cols = o.shape[-2:]
    ms = o.square().mean(-1)
    v.mul_(BETA2).add_((1 - BETA2) * ms)
    r = 1.0 / (v.sqrt() + ROW_EPS)
    norm = (cols * ms * r * r).sum(-1, keepdim=True).sqrt()
    k = torch.where(norm > 0, LR * TARGET * math.sqrt(rows * cols) / norm, 0.0) * r
    w.mul_(1.0 - LR * WD).sub_(k.unsqueeze(-1) * o)
    return {"W": w, "v": v, **_store(w, s)}


def _run_logits(s):
    case = s["case"]
    if own:
        from mixed_precision_optimizer_amd import hpo_stack
        hpo_stack.hpo_qk_max_logits(s["q"], s["k"], s["smax"], scale=s["scale"], causal=case["causal"],
                                    window=case["window"], cu_seqlens_q=s.get("cu_q"), cu_seqlens_k=s.get("cu_k"),
                                    max_seqlen_q=s.get("max_q"), max_seqlen_k=s.get("max_k"))
        return s["smax"]
    q, k = s["q"], s["k"]
    if case["packed"]:   # each sequence in a row of its own, zero rows behind its end
        q, lq = _unpack(q, s["cu_q"], s["max_q"])
        k, lk = _unpack(k, s["cu_k"], s["max_k"])
    else:
        lq = torch.full((q.shape[0],), q.shape[1], device=DEV)
        lk = torch.full((k.shape[0],), k.shape[1], device=DEV)
    b, n, h, d = q.shape
    m, hk = k.shape[1], k.shape[2]
    x = (q.float().permute(0, 2, 1, 3).reshape(b, hk, (h // hk) * n, d)
         @ k.float().permute(0, 2, 3, 1).contiguous()).view(b, h, n, m) * s["scale"]
    x.masked_fill_(~_allowed(case, lq, lk, n, m).unsqueeze(1), -math.inf)
    s["smax"].copy_(x.amax((0, 2, 3)))
    return s["smax"]


def _unpack(x, cu, longest):
    at = cu[:-1, None].long() + torch.arange(longest, device=DEV)
    lens = (cu[1:] - cu[:-1]).long()
    inside = torch.arange(longest, device=DEV) < lens[:, None]
    y = x[torch.where(inside, at, 0).clamp(max=x.shape[0] - 1)]
    return torch.where(inside[..., None, None], y, 0), lens


def _allowed(case, lq, lk, n, m):
    """[batch, n, m]: the pairs whose logits count; the last query sees the last key."""
    i, j = torch.arange(n, device=DEV)[:, None], torch.arange(m, device=DEV)
    ok = (i < lq[:, None, None]) & (j < lk[:, None, None])
    if case["causal"]:
        at = i + (lk - lq)[:, None, None]
        ok = ok & (j <= at)
        if case["window"] >= 0:
            ok = ok & (j >= at - case["window"])
    return ok


def _run_clip(s):
    case = s["case"]
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if own:
        from mixed_precision_optimizer_amd import hpo_stack
        hpo_stack.hpo_qk_clip(s["smax"], hk, TAU, [
            hpo_stack.ClipWeight(s["Wq"], h, 0.5, param=s.get("pq"), scales=s.get("sq")),
            hpo_stack.ClipWeight(s["Wk"], hk, 0.5, param=s.get("pk"), scales=s.get("sk"))])
    else:
        top = s["smax"].view(hk, h // hk).amax(-1)
        f = torch.where(torch.isfinite(top) & (top > TAU), TAU / top, 1.0).sqrt()
        s["Wq"].view(hk, -1).mul_(f[:, None])
        s["Wk"].view(hk, -1).mul_(f[:, None])
        _store(s["Wq"], s, "q")
        _store(s["Wk"], s, "k")
    return {"Wq": s["Wq"], "Wk": s["Wk"], **_held(s, "q"), **_held(s, "k")}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _pairs(n, m, case):
    if not case["causal"]:
        return n * m
    w, off = case["window"], m - n
    total = 0
    for i in range(n):
        hi = i + off
        lo = max(0, hi - w) if w >= 0 else 0
        total += max(0, min(hi, m - 1) - lo + 1)
    return total


def work(case):
    op = case["op"]
    if op == "ortho":
        b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": b * m * n * (size + 2 + (8 if case["momentum"] else 0)),
                # one triangle of each symmetric product; where the Gram matrix is much the smaller, the iteration on
                # it (about four products a step) and one product with the input
                "flops": b * min(5 * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n),
                                 m * (m + 1) * n + 2 * m * m * n + 5 * 4 * m * m * (m + 1))}
    if op == "update":
        n = case["batch"] * case["rows"] * case["cols"]
        p = {"none": 0, "bf16": 2, "mx8": 1 + 1 / 32}[case["param"]]
        return {"bytes": n * ((2 if case["o"] == "bf16" else 4) + 8 + p) + 8 * case["batch"] * case["rows"],
                "flops": 6 * n}
    if op == "logits":
        d, h, hk = case["dim"], case["heads"], case["kv_heads"]
        if case["packed"]:
            lq, lk = _lengths(case)
        else:
            lq, lk = [case["seq_q"]] * case["batch"], [case["seq_k"]] * case["batch"]
        return {"bytes": 2 * d * (sum(lq) * h + sum(lk) * hk) + 4 * h,
                "flops": 2 * d * h * sum(_pairs(n, m, case) for n, m in zip(lq, lk))}
    h, hk, d, c = case["heads"], case["kv_heads"], case["dim"], case["cols"]
    p = {"none": 0, "bf16": 2, "mx8": 1 + 1 / 32}[case["param"]]
    # the groups with a head over the threshold, at the least: the heads over it may share groups
    groups = -(-case["over"] // (h // hk))
    return {"bytes": groups * (h // hk + 1) * d * c * (8 + p) + 4 * h, "flops": 2 * groups * (h // hk + 1) * d * c}


# ---------------------------------------------------------------------------
# the definitions in binary64
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    return {"ortho": _exact_ortho, "update": _exact_update, "logits": _exact_logits, "clip": _exact_clip}[case["op"]](
        case, s)


def _exact_ortho(case, s):
    g, out = s["G"].to(F64), {}
    if "M" in s:
        m = MU * s["M"].to(F64) + g
        g, out["M"] = g + MU * m, m
    a, b, c = NS_ABC
    res = torch.empty_like(g)
    for z in range(g.shape[0]):
        x = g[z] / (torch.linalg.vector_norm(g[z]) + NS_EPS)
        left = x.shape[0] <= x.shape[1]
        for _ in range(5):
            gram = x @ x.T if left else x.T @ x
            poly = torch.addmm(b * gram, gram, gram, alpha=c)
            x = a * x + (poly @ x if left else x @ poly)
        res[z] = x
    return {"out": res, **out}


def _exact_mx(w):
    """Values and scales of w in blocks of 32, from the definition: the value nearest to w / 2^e on e4m3's grid."""
    c = w.shape[-1]
    nb = -(-c // MX_BLOCK)
    x = torch.zeros(*w.shape[:-1], nb * MX_BLOCK, dtype=F64, device=DEV)
    x[..., :c] = w
    x = x.view(*w.shape[:-1], nb, MX_BLOCK)
    amax = x.abs().max(-1).values
    e = torch.where(amax > 0, torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0))) - 8, -127.0).clamp(-127, 127)
    y = x * torch.exp2(-e)[..., None]
    # spacing of the grid at |y|: 2^(exponent - 3), from 2^-6 down 2^-9
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return y.reshape(*w.shape[:-1], nb * MX_BLOCK)[..., :c], torch.exp2(e)


def _exact_weight(case, w, suffix=""):
    if case["param"] == "mx8":
        p, e = _exact_mx(w)
        return {"p" + suffix: p, "s" + suffix: e}
    return {"p" + suffix: w} if case["param"] == "bf16" else {}


def _exact_update(case, s):
    o, w = s["O"].to(F64), s["W"].to(F64)
    rows, cols = o.shape[-2:]
    ms = torch.einsum("brc,brc->br", o, o) / cols
    v = BETA2 * s["v"].to(F64) + (1 - BETA2) * ms
    u = o / (torch.sqrt(v) + ROW_EPS)[..., None]
    norm = torch.linalg.vector_norm(u, dim=(-2, -1), keepdim=True)
    w = w * (1 - LR * WD) - torch.where(norm > 0, LR * TARGET * math.sqrt(rows * cols) / norm, 0.0) * u
    return {"W": w, "v": v, **_exact_weight(case, w)}


def _exact_logits(case, s):
    h, hk = case["heads"], case["kv_heads"]
    best = torch.full((h,), -math.inf, dtype=F64, device=DEV)
    for z in range(case["batch"]):
        if case["packed"]:
            (q0, q1), (k0, k1) = s["cu_q"][z:z + 2].tolist(), s["cu_k"][z:z + 2].tolist()
            q, k = s["q"][q0:q1], s["k"][k0:k1]
        else:
            q, k = s["q"][z], s["k"][z]
        n, m = q.shape[0], k.shape[0]
        if n == 0 or m == 0:
            continue
        lag = torch.arange(n, device=DEV)[:, None] + (m - n) - torch.arange(m, device=DEV)   # keys behind the query's own
        hidden = torch.zeros_like(lag, dtype=torch.bool)
        if case["causal"]:
            hidden = lag < 0
            if case["window"] >= 0:
                hidden |= lag > case["window"]
        for j in range(h):
            x = q[:, j].to(F64) @ k[:, j // (h // hk)].to(F64).T / math.sqrt(case["dim"])
            best[j] = torch.maximum(best[j], x.masked_fill(hidden, -math.inf).max())
    return best


def _exact_clip(case, s):
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    top = s["smax"].to(F64).reshape(hk, h // hk).max(1).values
    f = torch.sqrt(torch.clamp(TAU / top, max=1.0))
    wq = s["Wq"].to(F64) * f.repeat_interleave(h // hk * d)[:, None]
    wk = s["Wk"].to(F64) * f.repeat_interleave(d)[:, None]
    return {"Wq": wq, "Wk": wk, **_exact_weight(case, wq, "q"), **_exact_weight(case, wk, "k")}
