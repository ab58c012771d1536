"""Stack operators on the GPU at the ends of their numbers' ranges."""
import math

import pytest

torch = pytest.importorskip("torch")

import stack_util as su  # noqa: E402
from test_gpu_stack import (CFG, DEV, S, check_logits, check_ortho, check_rms, gen, gradient, ortho,  # noqa: E402, F401
                            workspace)

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


# --------------------------------------------------------------------------
# hpo_orthogonalize: norms far under ns_eps, or under fp32's normal numbers
# --------------------------------------------------------------------------
@pytest.mark.parametrize("r,c", [(40, 60), (60, 40), (90, 3000), (20000, 128), (140, 150), (300, 520),
                                 (520, 300), (1000, 1030), (2048, 2600)])
@pytest.mark.parametrize("below", [1e-2, 1e-4, 1e-8, 1e-12, 1e-20, 1e-28])
def test_orthogonalize_gradients_far_below_eps(S, r, c, below):
    """The iteration is all but linear there; its direction and size are as exact as anywhere else."""
    G = gradient(111, 2, r, c).double()
    G = (G / torch.linalg.vector_norm(G, dim=(1, 2), keepdim=True) * 1e-7 * below).float()
    G[1] *= 1e6 / below * 1e-3      # one matrix at an ordinary norm beside it
    check_ortho(ortho(S, G.to(DEV)), G.double(), tag=f"norm {below} eps")


@pytest.mark.parametrize("steps,coeffs", [(1, None), (7, None), (4, [(1.5, -0.5, 0.0)] * 4),
                                          (3, [(8.2, -23.6, 17.3), (4.1, -2.9, 0.5), (1.875, -1.25, 0.375)])])
@pytest.mark.parametrize("r,c", [(40, 60), (140, 300)])
@pytest.mark.parametrize("below", [1e-3, 1e-5, 1e-9, 1e-15])
def test_orthogonalize_schedules_far_below_eps(S, steps, coeffs, r, c, below):
    """Schedules that grow X by more or less than the default; 1e-3 and 1e-5 lie where not all of them are scaled."""
    G = gradient(119, 1, r, c)
    G = G / torch.linalg.vector_norm(G) * 1e-7 * below
    out = ortho(S, G.to(DEV), cfg=S.hpo.make_muon_cfg(ns_steps=steps, ns_coeffs=coeffs))
    check_ortho(out, G.double(), steps, coeffs, tag=f"{steps} steps, norm {below} eps")


@pytest.mark.parametrize("r,c", [(40, 60), (300, 20), (90, 3000), (140, 150), (300, 520)])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-7])
@pytest.mark.parametrize("momentum", [False, True])
def test_orthogonalize_subnormal_gradients(S, r, c, eps, momentum):
    """Gradients of a few of fp32's least steps: dense, and two elements of one row."""
    step = 2.0 ** -149
    G = torch.zeros(2, r, c)
    G[0] = torch.randint(-3, 4, (r, c), generator=gen(113)).float() * step
    G[1, r // 2, 3], G[1, r // 2, c - 1] = step, step
    cfg = S.hpo.make_muon_cfg(ns_eps=eps, momentum=0.5, nesterov=False)
    M = 4.0 * G if momentum else None      # 0.5 * 4 G + G: exact
    m = M.to(DEV) if momentum else None
    out = ortho(S, G.to(DEV), m, cfg=cfg)
    g = 3.0 * G if momentum else G
    if momentum:
        assert torch.equal(m.cpu(), g)
    # the library holds eps as fp32
    check_ortho(out, g.double(), eps=float(torch.tensor(eps, dtype=torch.float32)), tag=f"subnormal, eps {eps}")


def test_orthogonalize_beyond_fp32_still_gives_zeros(S):
    """A norm over fp32's largest value gives zeros."""
    for r, c in ((40, 60), (100, 3000), (140, 150)):
        assert bool((ortho(S, torch.full((1, r, c), 3e38, device=DEV)) == 0).all())


@pytest.mark.parametrize("r,c", [(40, 60), (90, 3000), (140, 150)])
@pytest.mark.parametrize("eps", [1.0, 1e20, 3e38, 1e39, 1e300])
def test_orthogonalize_large_eps(S, r, c, eps):
    """An eps beyond fp32 is infinite to the library, as a norm would be: zeros.  Under it the result is what the
    formula gives, down to bf16's subnormals (2^-133 apart)."""
    G = gradient(121, 2, r, c)
    out = ortho(S, G.to(DEV), cfg=S.hpo.make_muon_cfg(ns_eps=eps)).double().cpu()
    if eps > 3.4e38:
        assert bool((out == 0).all())
        return
    for z in range(2):
        x, tol = su.ns_tolerance(G[z].double(), eps=float(torch.tensor(eps, dtype=torch.float32)))
        d = float(torch.linalg.vector_norm(out[z] - x))
        assert d <= tol * float(torch.linalg.vector_norm(x)) + 2.0 ** -134 * math.sqrt(r * c), (z, d)


@pytest.mark.parametrize("r,c", [(40, 300), (100, 3000), (140, 300), (1300, 5000)])
def test_orthogonalize_far_below_eps_in_a_graph(S, r, c):
    """The exponent that such a matrix is held at belongs to each run of the graph."""
    G = gradient(115, 2, r, c).to(DEV)
    out, ws = torch.zeros(G.shape, dtype=torch.bfloat16, device=DEV), workspace(S.hpo_orthogonalize_workspace(G))
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        ortho(S, G, out=out, ws=ws)
    for size in (1.0, 1e-20, 1e-9, 1.0, 1e-25):
        G.copy_(gradient(117, 2, r, c) * size)
        gr.replay()
        got = su.bits(out)
        torch.cuda.synchronize()
        assert torch.equal(got, su.bits(ortho(S, G))), size
        check_ortho(out, G.double().cpu(), tag=f"graph, size {size}")


# --------------------------------------------------------------------------
# hpo_qk_max_logits: what lies beside the heads
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dim", [1, 3, 8, 16, 24, 32, 48, 57, 80, 100, 112, 136, 144, 160, 176, 191, 208, 224, 240, 248, 255])
@pytest.mark.parametrize("pad", [0, 16, 9])
def test_qk_max_does_not_see_what_lies_beside_a_head(S, dim, pad):
    """NaN between the heads of a padded buffer, infinities behind a sequence's end, dims of every way into LDS."""
    g = gen(dim * 3 + pad)
    b, n, m, h = 2, 70, 331, 4
    wide = lambda t, heads: torch.full((b, t, heads, dim + pad), math.nan, dtype=torch.bfloat16)   # noqa: E731
    Q, K = wide(n, h), wide(m, 2)
    q, k = torch.randn(b, n, h, dim, generator=g).bfloat16(), torch.randn(b, m, 2, dim, generator=g).bfloat16()
    Q[..., :dim], K[..., :dim] = q, k
    lens = torch.tensor([331, 200], dtype=torch.int32)
    K[1, 200:, :, :dim] = math.inf
    Q, K = Q.to(DEV), K.to(DEV)
    for causal in (True, False):
        out = torch.empty(h, device=DEV)
        S.hpo_qk_max_logits(Q[..., :dim], K[..., :dim], out, 0.25, causal=causal, seqlens_k=lens.to(DEV))
        check_logits(out, list(q), [k[0], k[1, :200]], 0.25, causal, -1, dim, f"dim {dim} pad {pad}")
