/*
 * hpo_stack_api.cpp -- host side of the stack operators (hpo_stack.h):
 * argument checks, the scales of the Newton-Schulz iteration and the launches.
 * Host code only (compiled as plain C++ against the HIP runtime API).
 */
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "hpo_set.h"
#include "hpo_stack_impl.h"

using namespace hpo_host;

namespace {

constexpr int64_t kMaxBatch = 65535;              /* a launch's z dimension */
constexpr int64_t kMaxRows = int64_t{1} << 24;    /* rows of a whole stack: one workgroup each, at most */
constexpr int64_t kMaxSpan = int64_t{1} << 44;    /* elements between a stack's first and last */

}  // namespace

/* Stacks as every call that takes them checks them (hpo_set.h). */
namespace hpo_host {

int64_t elem_size(int32_t dtype) { return dtype == HPO_PARAM_FP32 ? 4 : (dtype == HPO_WEIGHT_MX8 ? 1 : 2); }

bool is_empty(const hpo_stack* s) { return s->batch == 0 || s->rows == 0 || s->cols == 0; }

hpo_status check_stack(const hpo_stack* s, const char* what)
{
    if (!s)
        return fail(HPO_EINVAL, "%s is NULL", what);
    if (s->batch < 0 || s->rows < 0 || s->cols < 0)
        return fail(HPO_EINVAL, "%s: negative shape %lld x %lld x %lld", what, (long long)s->batch, (long long)s->rows,
                    (long long)s->cols);
    if (s->batch > kMaxBatch || s->rows > HPO_MUON_MAX_DIM || s->cols > HPO_MUON_MAX_DIM)
        return fail(HPO_EINVAL, "%s: %lld x %lld x %lld is too large (at most %lld matrices, each side at most %lld)", what,
                    (long long)s->batch, (long long)s->rows, (long long)s->cols, (long long)kMaxBatch,
                    (long long)HPO_MUON_MAX_DIM);
    if (s->reserved != 0)
        return fail(HPO_EINVAL, "%s: reserved must be 0", what);
    if (is_empty(s))
        return HPO_OK;
    if (!s->data || !aligned(s->data, static_cast<uintptr_t>(elem_size(s->dtype))))
        return fail(HPO_EINVAL, "%s: data must be a non-NULL device pointer aligned to its element", what);
    if (s->batch_stride < 0 || s->row_stride < 0 || s->batch_stride > kMaxSpan || s->row_stride > kMaxSpan)
        return fail(HPO_EINVAL, "%s: strides must lie in [0, 2^44]", what);
    if (s->batch * s->rows > kMaxRows)
        return fail(HPO_EINVAL, "%s: %lld rows in all, at most %lld", what, (long long)(s->batch * s->rows),
                    (long long)kMaxRows);
    const int64_t bs = s->batch_stride, rs = s->row_stride;
    if ((s->rows > 1 && rs < s->cols) || (s->batch > 1 && bs < s->cols))
        return fail(HPO_EINVAL, "%s: a stride is below the %lld columns", what, (long long)s->cols);
    const __int128 matrix = static_cast<__int128>(s->rows - 1) * rs + s->cols;
    const __int128 across = static_cast<__int128>(s->batch - 1) * bs + s->cols;
    if (s->batch > 1 && s->rows > 1 && bs < matrix && rs < across)
        return fail(HPO_EINVAL, "%s: the strides make matrices overlap", what);
    if (static_cast<__int128>(s->batch - 1) * bs + matrix > kMaxSpan)
        return fail(HPO_EINVAL, "%s: the stack spans more than 2^44 elements", what);
    return HPO_OK;
}

hpo_status check_like(const hpo_stack* s, const char* what, const hpo_stack* o, const char* other)
{
    hpo_status st = check_stack(s, what);
    if (st != HPO_OK)
        return st;
    if (s->batch != o->batch || s->rows != o->rows || s->cols != o->cols)
        return fail(HPO_EINVAL, "%s is %lld x %lld x %lld, %s is %lld x %lld x %lld", what, (long long)s->batch,
                    (long long)s->rows, (long long)s->cols, other, (long long)o->batch, (long long)o->rows,
                    (long long)o->cols);
    return HPO_OK;
}

hpo::StackView view(const hpo_stack* s)
{
    hpo::StackView v{};
    if (s) {
        v.data = s->data;
        v.bs = s->batch > 1 ? s->batch_stride : 0;
        v.rs = s->rows > 1 ? s->row_stride : 0;
    }
    return v;
}

}  // namespace hpo_host

namespace {

/* Master and model weight of a row-wise update. */
hpo_status weight_view(const hpo_stack* master, const hpo_stack* param, uint8_t* scales, hpo::WeightView& w)
{
    w = hpo::WeightView{};
    w.master = view(master);
    w.rows = master->rows;
    w.cols = master->cols;
    w.param_dtype = HPO_PARAM_FP32;
    if (!param) {
        if (scales)
            return fail(HPO_EINVAL, "d_scales without a param");
        return HPO_OK;
    }
    w.param_dtype = param->dtype;
    w.param = view(param);
    w.scales = scales;
    return HPO_OK;
}

hpo_status check_weight(const hpo_stack* master, const hpo_stack* param, const uint8_t* scales)
{
    hpo_status st = check_stack(master, "master");
    if (st != HPO_OK)
        return st;
    if (master->dtype != HPO_PARAM_FP32)
        return fail(HPO_EDTYPE, "master must be fp32");
    if (!param)
        return HPO_OK;
    if (param->dtype != HPO_PARAM_BF16 && param->dtype != HPO_WEIGHT_MX8)
        return fail(HPO_EDTYPE, "param dtype %d is not supported (bf16 = 0, 8 bits with scales = 16)", param->dtype);
    st = check_like(param, "param", master, "master");
    if (st != HPO_OK)
        return st;
    if (param->dtype == HPO_WEIGHT_MX8 && !scales && !is_empty(param))
        return fail(HPO_EINVAL, "an 8-bit param needs d_scales");
    if (param->dtype != HPO_WEIGHT_MX8 && scales)
        return fail(HPO_EINVAL, "d_scales is for an 8-bit param");
    return HPO_OK;
}

/* ---------------------------------------------------------------------- */
/* scales of the Newton-Schulz iteration                                   */
/* ---------------------------------------------------------------------- */
/* Largest |a s + b s^3 + c s^5| over 0 <= s <= S. */
double odd_quintic_max(double a, double b, double c, double S)
{
    auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
    double best = f(S);
    /* a + 3 b u + 5 c u^2 = 0, u = s^2 */
    double u[2] = {-1.0, -1.0};
    if (c != 0.0) {
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (d >= 0.0) {
            u[0] = (-3.0 * b + std::sqrt(d)) / (10.0 * c);
            u[1] = (-3.0 * b - std::sqrt(d)) / (10.0 * c);
        }
    } else if (b != 0.0) {
        u[0] = -a / (3.0 * b);
    }
    for (double x : u)
        if (x > 0.0 && x < S * S)
            best = std::max(best, f(std::sqrt(x)));
    return best;
}

/* Largest |b l + c l^2| over 0 <= l <= L. */
double quadratic_max(double b, double c, double L)
{
    double best = std::fabs(L * (b + c * L));
    if (c != 0.0) {
        const double x = -b / (2.0 * c);
        if (x > 0.0 && x < L)
            best = std::max(best, std::fabs(x * (b + c * x)));
    }
    return best;
}

/* Largest |a + b l + c l^2| over 0 <= l <= L. */
double shifted_max(double a, double b, double c, double L)
{
    double best = std::max(std::fabs(a), std::fabs(a + L * (b + c * L)));
    if (c != 0.0) {
        const double x = -b / (2.0 * c);
        if (x > 0.0 && x < L)
            best = std::max(best, std::fabs(a + x * (b + c * x)));
    }
    return best;
}

/* The exponent e with bound * 2^e in (2^13, 2^14]: a factor of four below
 * fp16's largest value is left for roundings; zero bounds take 0. */
int fit(double bound)
{
    if (!(bound > 0.0))
        return 0;
    return std::max(-60, std::min(60, 14 - static_cast<int>(std::ceil(std::log2(bound)))));
}

/* The singular values of X start in [0, 1] (X0 = g / (||g||_F + eps)) and
 * every step maps them by a s + b s^3 + c s^5, so its entries, those of A =
 * X X^T (squares) and of B (b l + c l^2 at those squares) are bounded on the host. */
hpo_status ns_scales(const hpo_muon_cfg* cfg, hpo::OrthoArgs& out)
{
    constexpr double kDefault[3] = {3.4445, -4.7750, 2.0315};
    constexpr double kMost = 32768.0;
    double S = 1.0;
    out.steps = cfg->ns_steps;
    int ex = fit(S);
    double Pb = 1.0;   /* bound of the product of the steps' Q */
    out.x0_scale = static_cast<float>(std::ldexp(1.0, ex));
    for (int32_t k = 0; k < cfg->ns_steps; ++k) {
        const double* c = cfg->ns_coeffs ? cfg->ns_coeffs + 3 * k : kDefault;
        const bool last = k + 1 == cfg->ns_steps;
        /* 1 % for the roundings of the steps so far: half a step of fp16 that falls one way everywhere
         * is 2^-11 of s, times p'(s) (24 at s = 1 for steep first steps), times the next
         * step's.  (More would leave the basin of the default coefficients, which grow without bound
         * from s = 1.28 on.) */
        const double T = 1.01 * S, L = T * T, P = quadratic_max(c[1], c[2], L),
                     next = odd_quintic_max(c[0], c[1], c[2], T);
        if (!(next <= kMost) || !(P <= kMost) || !(L <= kMost))
            return fail(HPO_EINVAL,
                        "ns_coeffs: step %d may leave the range of the iteration (|X| up to %g from a start of 1 widened by 1 %% a "
                        "step)",
                        k, next);
        const int ea = fit(L), eb = fit(P), en = last ? 0 : fit(next);
        hpo::NsStepScale& s = out.step[k];
        s.gram = static_cast<float>(std::ldexp(1.0, ea - 2 * ex));
        s.poly_b = static_cast<float>(std::ldexp(static_cast<double>(static_cast<float>(c[1])), eb - ea));
        s.poly_c = static_cast<float>(std::ldexp(static_cast<double>(static_cast<float>(c[2])), eb - 2 * ea));
        s.step_a = static_cast<float>(std::ldexp(static_cast<double>(static_cast<float>(c[0])), en - ex));
        s.step_c = static_cast<float>(std::ldexp(1.0, en - eb - ex));
        const double Qb = shifted_max(c[0], c[1], c[2], L);
        hpo::GramStep& q = out.gram[k];
        q.a = static_cast<float>(c[0]);
        q.b = static_cast<float>(c[1]);
        q.c = static_cast<float>(c[2]);
        q.a_exp = fit(L);
        q.q_exp = fit(Qb);
        q.t_exp = fit(Qb * L);
        q.p_exp = fit(Pb);
        Pb *= std::max(Qb, 1e-6);
        S = std::max(next, 1e-6);
        ex = en;
        if (!last)
            out.lift_room = std::max(out.lift_room, static_cast<int32_t>(std::ceil(std::log2(Pb / S))));
    }
    out.p_exp = fit(Pb);
    /* What fp32 sums lose of S and A grows, in the directions of the small singular values, by the square of
     * the steps' growth.  Up to 2^11 (the default coefficients' six steps) it stays under 3e-2 where
     * one direction is a thousand times the others, and under 5e-4 where none is ten times them: the
     * two-product form has 6e-4 and 3.6e-3 there, at eight times the time (32 x 128 x 4096). */
    out.use_gram = Pb <= 2048.0 ? 1 : 0;
    return HPO_OK;
}

hpo_status check_qk_shape(const hpo_qk* a)
{
    if (a->dtype != HPO_PARAM_BF16 && a->dtype != HPO_PARAM_FP16)
        return fail(HPO_EDTYPE, "q / k dtype %d is not supported (bf16 = 0, fp16 = 2)", a->dtype);
    if (a->batch < 0 || a->heads < 0 || a->kv_heads < 0 || a->seq_q < 0 || a->seq_k < 0)
        return fail(HPO_EINVAL, "negative batch, heads or sequence");
    if (a->batch > 65535 || a->heads > 65535)
        return fail(HPO_EINVAL, "batch and heads must be at most 65535");
    if (a->heads > 0 && (a->kv_heads < 1 || a->heads % a->kv_heads != 0))
        return fail(HPO_EINVAL, "heads (%d) must be a multiple of kv_heads (%d)", a->heads, a->kv_heads);
    if (a->head_dim < 1 || a->head_dim > HPO_QK_MAX_DIM)
        return fail(HPO_EINVAL, "head_dim must be in [1, %d] (got %d)", HPO_QK_MAX_DIM, a->head_dim);
    constexpr int64_t kMaxSeq = int64_t{1} << 30;
    if (a->seq_q > kMaxSeq || a->seq_k > kMaxSeq)
        return fail(HPO_EINVAL, "sequences must be at most 2^30 tokens");
    if (a->causal != 0 && a->causal != 1)
        return fail(HPO_EINVAL, "causal must be 0 or 1 (got %d)", a->causal);
    if (a->window < -1 || (a->window >= 0 && !a->causal))
        return fail(HPO_EINVAL, "window must be -1, or >= 0 with causal = 1 (got %lld)", (long long)a->window);
    if (!(a->scale > 0.0f) || !std::isfinite(a->scale))
        return fail(HPO_EINVAL, "scale must be positive and finite (got %g)", static_cast<double>(a->scale));
    if (a->reserved != 0)
        return fail(HPO_EINVAL, "reserved must be 0");
    if ((a->cu_seqlens_q == nullptr) != (a->cu_seqlens_k == nullptr))
        return fail(HPO_EINVAL, "cu_seqlens_q and cu_seqlens_k go together");
    if (a->cu_seqlens_q && (a->seqlens_q || a->seqlens_k))
        return fail(HPO_EINVAL, "seqlens_* are for padded batches");
    if (a->cu_seqlens_q && (a->max_seqlen_q < 0 || a->max_seqlen_k < 0))
        return fail(HPO_EINVAL, "max_seqlen_q and max_seqlen_k must be >= 0");
    for (const int32_t* p : {a->cu_seqlens_q, a->cu_seqlens_k, a->seqlens_q, a->seqlens_k})
        if (!aligned(p, 4))
            return fail(HPO_EINVAL, "lengths must be 4-byte aligned");
    const int64_t strides[] = {a->q_stride_batch, a->q_stride_token, a->q_stride_head,
                               a->k_stride_batch, a->k_stride_token, a->k_stride_head};
    for (int64_t s : strides)
        if (s < 0 || s > kMaxSpan)
            return fail(HPO_EINVAL, "q / k strides must lie in [0, 2^44]");
    if (a->k_stride_token > HPO_QK_MAX_STRIDE)
        return fail(HPO_EINVAL, "k_stride_token must be at most %lld", (long long)HPO_QK_MAX_STRIDE);
    return HPO_OK;
}

}  // namespace

extern "C" {

hpo_status hpo_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, int64_t* out_bytes)
{
    if (!out_bytes)
        return fail(HPO_EINVAL, "out_bytes is NULL");
    if (batch < 0 || rows < 0 || cols < 0 || batch > kMaxBatch || rows > HPO_MUON_MAX_DIM || cols > HPO_MUON_MAX_DIM)
        return fail(HPO_EINVAL, "bad shape %lld x %lld x %lld", (long long)batch, (long long)rows, (long long)cols);
    if (rows > 0 && cols > (int64_t{1} << 40) / rows)
        return fail(HPO_EINVAL, "matrices of %lld x %lld are too large (2^40 elements)", (long long)rows, (long long)cols);
    *out_bytes = batch == 0 || rows == 0 || cols == 0 ? 0 : hpo::ortho_workspace(batch, rows, cols);
    if (*out_bytes != 0 && std::min(rows, cols) <= hpo::kGramMax)   /* either form, as the coefficients allow */
        *out_bytes = std::max(*out_bytes, hpo::gram_workspace(batch, rows, cols));
    return ok();
}

hpo_status hpo_orthogonalize(const hpo_stack* G, const hpo_stack* momentum, const hpo_stack* out,
                             const hpo_muon_cfg* cfg, float inv_scale, double max_norm, const float* d_norm,
                             const int32_t* d_found_inf, void* d_workspace, int64_t workspace_bytes, void* stream)
{
    hpo_status st = check_muon_cfg(cfg, momentum == nullptr);
    if (st != HPO_OK)
        return st;
    st = check_stack(G, "G");
    if (st != HPO_OK)
        return st;
    if (G->dtype != HPO_PARAM_FP32 && G->dtype != HPO_PARAM_BF16)
        return fail(HPO_EDTYPE, "G dtype %d is not supported (bf16 = 0, fp32 = 1)", G->dtype);
    st = check_like(out, "out", G, "G");
    if (st != HPO_OK)
        return st;
    if (out->dtype != HPO_PARAM_BF16)
        return fail(HPO_EDTYPE, "out must be bf16");
    if (momentum) {
        st = check_like(momentum, "momentum", G, "G");
        if (st != HPO_OK)
            return st;
        if (momentum->dtype != HPO_PARAM_FP32)
            return fail(HPO_EDTYPE, "momentum must be fp32");
    }
    if (!std::isfinite(inv_scale))
        return fail(HPO_EINVAL, "inv_scale must be finite");
    if (std::isnan(max_norm))
        return fail(HPO_EINVAL, "max_norm is NaN");
    if (max_norm > 0.0 && !d_norm)
        return fail(HPO_EINVAL, "clipping (max_norm > 0) needs d_norm");
    hpo::OrthoArgs a{};
    st = ns_scales(cfg, a);
    if (st != HPO_OK)
        return st;
    int64_t need = 0;
    st = hpo_orthogonalize_workspace(G->batch, G->rows, G->cols, &need);
    if (st != HPO_OK)
        return st;
    if (need == 0)
        return ok();
    if (!d_workspace || !aligned(d_workspace, 256))
        return fail(HPO_EINVAL, "d_workspace must be a non-NULL, 256-byte aligned device pointer");
    if (workspace_bytes < need)
        return fail(HPO_EINVAL, "workspace of %lld bytes is below the %lld this stack needs", (long long)workspace_bytes,
                    (long long)need);
    a.G = view(G);
    a.M = view(momentum);
    a.out = view(out);
    a.g_bf16 = G->dtype == HPO_PARAM_BF16 ? 1 : 0;
    /* the thin form addresses a matrix with 32-bit offsets */
    auto near = [](const hpo_stack* s) { return !s || (s->rows - 1) * s->row_stride + s->cols <= int64_t{1} << 30; };
    a.use_gram = a.use_gram && std::min(G->rows, G->cols) <= hpo::kGramMax && near(G) && near(momentum) && near(out);
    a.batch = G->batch;
    a.rows = G->rows;
    a.cols = G->cols;
    a.sc.inv_scale = inv_scale;
    a.sc.mu = static_cast<float>(cfg->momentum);
    a.sc.omu = static_cast<float>(1.0 - cfg->momentum);
    a.sc.eps = static_cast<float>(cfg->ns_eps);
    a.sc.max_norm = max_norm;
    a.sc.d_norm = d_norm;
    a.sc.gate.d_found = d_found_inf;
    a.sc.form = cfg->momentum_form;
    a.sc.nesterov = cfg->nesterov;
    a.ws = d_workspace;
    const hipError_t e = a.use_gram ? hpo::launch_gram(a, as_stream(stream)) : hpo::launch_orthogonalize(a, as_stream(stream));
    if (e != hipSuccess)
        return hip_fail(e, "launch Newton-Schulz of a stack");
    return ok();
}

hpo_status hpo_rms_update_workspace(int64_t batch, int64_t rows, int64_t* out_bytes)
{
    if (!out_bytes)
        return fail(HPO_EINVAL, "out_bytes is NULL");
    if (batch < 0 || rows < 0 || batch > kMaxBatch || rows > HPO_MUON_MAX_DIM || batch * rows > kMaxRows)
        return fail(HPO_EINVAL, "bad shape: %lld matrices of %lld rows", (long long)batch, (long long)rows);
    /* q and N^2 in binary64, r in fp32 */
    *out_bytes = batch * rows == 0 ? 0 : 8 * batch * rows + 8 * batch + 4 * batch * rows;
    return ok();
}

hpo_status hpo_rms_update(const hpo_stack* O, const hpo_stack* master, float* d_v, const hpo_stack* param,
                          uint8_t* d_scales, const hpo_rms_cfg* cfg, const int32_t* d_found_inf, void* d_workspace,
                          int64_t workspace_bytes, void* stream)
{
    hpo_status st = check_weight(master, param, d_scales);
    if (st != HPO_OK)
        return st;
    st = check_like(O, "O", master, "master");
    if (st != HPO_OK)
        return st;
    if (O->dtype != HPO_PARAM_FP32 && O->dtype != HPO_PARAM_BF16)
        return fail(HPO_EDTYPE, "O dtype %d is not supported (bf16 = 0, fp32 = 1)", O->dtype);
    if (!cfg)
        return fail(HPO_EINVAL, "cfg is NULL");
    if (!is_finite(cfg->lr) || !is_finite(cfg->weight_decay) || !is_finite(cfg->target_rms))
        return fail(HPO_EINVAL, "lr, weight_decay and target_rms must be finite");
    if (!(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0))
        return fail(HPO_EINVAL, "beta2 must lie in [0, 1) (got %g)", cfg->beta2);
    if (!(cfg->eps >= 0.0) || !is_finite(cfg->eps))
        return fail(HPO_EINVAL, "eps must be finite and >= 0 (got %g)", cfg->eps);
    if (is_empty(master))
        return ok();
    if ((!d_v && cfg->beta2 > 0.0) || !aligned(d_v, 4))
        return fail(HPO_EINVAL, "d_v must be a 4-byte aligned device pointer (NULL only with beta2 = 0)");
    int64_t need = 0;
    st = hpo_rms_update_workspace(master->batch, master->rows, &need);
    if (st != HPO_OK)
        return st;
    if (!d_workspace || !aligned(d_workspace, 8))
        return fail(HPO_EINVAL, "d_workspace must be a non-NULL, 8-byte aligned device pointer");
    if (workspace_bytes < need)
        return fail(HPO_EINVAL, "workspace of %lld bytes is below the %lld this stack needs", (long long)workspace_bytes,
                    (long long)need);
    hpo::RmsArgs a{};
    st = weight_view(master, param, d_scales, a.w);
    if (st != HPO_OK)
        return st;
    a.O = view(O);
    a.o_fp32 = O->dtype == HPO_PARAM_FP32 ? 1 : 0;
    a.v = d_v;
    a.batch = master->batch;
    const int64_t n = master->batch * master->rows;
    a.q = static_cast<double*>(d_workspace);
    a.norm2 = a.q + n;
    a.r = reinterpret_cast<float*>(a.norm2 + master->batch);
    a.beta2 = cfg->beta2;
    a.eps = cfg->eps;
    a.gain = cfg->lr * cfg->target_rms * std::sqrt(static_cast<double>(master->rows) * static_cast<double>(master->cols));
    a.keep = static_cast<float>(1.0 - cfg->lr * cfg->weight_decay);
    a.d_found = d_found_inf;
    const hipError_t e = hpo::launch_rms_update(a, as_stream(stream));
    if (e != hipSuccess)
        return hip_fail(e, "launch row-normalised update");
    return ok();
}

hpo_status hpo_qk_max_logits(const hpo_qk* a, int32_t accumulate, float* d_max, void* stream)
{
    if (!a)
        return fail(HPO_EINVAL, "a is NULL");
    hpo_status st = check_qk_shape(a);
    if (st != HPO_OK)
        return st;
    if (accumulate != 0 && accumulate != 1)
        return fail(HPO_EINVAL, "accumulate must be 0 or 1 (got %d)", accumulate);
    if (a->heads == 0)
        return ok();
    if (!d_max || !aligned(d_max, 4))
        return fail(HPO_EINVAL, "d_max must be a non-NULL, 4-byte aligned device pointer");
    const bool some = a->batch > 0 && a->seq_q > 0 && a->seq_k > 0;
    if (some && (!a->q || !a->k || !aligned(a->q, 2) || !aligned(a->k, 2)))
        return fail(HPO_EINVAL, "q and k must be non-NULL, 2-byte aligned device pointers");
    const bool packed = a->cu_seqlens_q != nullptr;
    hpo::QkArgs g{};
    g.q = static_cast<const uint16_t*>(a->q);
    g.k = static_cast<const uint16_t*>(a->k);
    g.qsb = packed ? 0 : a->q_stride_batch;
    g.qst = a->q_stride_token;
    g.qsh = a->q_stride_head;
    g.ksb = packed ? 0 : a->k_stride_batch;
    g.kst = a->k_stride_token;
    g.ksh = a->k_stride_head;
    g.cu_q = a->cu_seqlens_q;
    g.cu_k = a->cu_seqlens_k;
    g.len_q = a->seqlens_q;
    g.len_k = a->seqlens_k;
    g.batch = a->batch;
    g.heads = a->heads;
    g.kv_heads = a->kv_heads;
    g.dim = a->head_dim;
    g.seq_q = static_cast<int32_t>(a->seq_q);
    g.seq_k = static_cast<int32_t>(a->seq_k);
    /* a sequence of a packed batch is no longer than all of it, and one tile at least is launched */
    g.max_q = static_cast<int32_t>(packed ? std::max<int64_t>(1, std::min(a->max_seqlen_q, a->seq_q)) : a->seq_q);
    g.max_k = static_cast<int32_t>(packed ? std::max<int64_t>(1, std::min(a->max_seqlen_k, a->seq_k)) : a->seq_k);
    g.causal = a->causal;
    g.window = a->window < 0 ? -1 : static_cast<int32_t>(std::min<int64_t>(a->window, int64_t{1} << 30));
    g.accumulate = accumulate;
    g.scale = a->scale;
    g.out = d_max;
    /* what only one batch row or head would step over does not decide the access width */
    const int64_t strides[] = {g.batch > 1 ? g.qsb : 0, g.qst, g.heads > 1 ? g.qsh : 0,
                               g.batch > 1 ? g.ksb : 0, g.kst, g.kv_heads > 1 ? g.ksh : 0};
    bool wide = aligned(a->q, 16) && aligned(a->k, 16);
    for (int64_t s : strides)
        wide = wide && s % 8 == 0;
    if (some) {
        const int64_t tiles = static_cast<int64_t>(g.batch) * g.heads * ((g.max_q + 255) / 256);
        if (tiles > (int64_t{1} << 23))
            return fail(HPO_EINVAL, "%lld query tiles are more than one launch can hold", (long long)tiles);
    }
    const hipError_t e = hpo::launch_qk_max(g, a->dtype == HPO_PARAM_FP16, wide, as_stream(stream));
    if (e != hipSuccess)
        return hip_fail(e, "launch attention logit maxima");
    return ok();
}

hpo_status hpo_qk_clip(const float* d_max, int32_t heads, int32_t kv_heads, double tau, const hpo_clip_weight* weights,
                       int32_t n_weights, const int32_t* d_found_inf, void* stream)
{
    if (heads < 1 || kv_heads < 1 || heads > 65535 || heads % kv_heads != 0)
        return fail(HPO_EINVAL, "heads (%d) must be in [1, 65535] and a multiple of kv_heads (%d)", heads, kv_heads);
    if (!d_max || !aligned(d_max, 4))
        return fail(HPO_EINVAL, "d_max must be a non-NULL, 4-byte aligned device pointer");
    if (!(tau > 0.0) || !is_finite(tau))
        return fail(HPO_EINVAL, "tau must be positive and finite (got %g)", tau);
    if (n_weights < 1 || n_weights > HPO_CLIP_MAX_WEIGHTS || !weights)
        return fail(HPO_EINVAL, "n_weights must be in [1, %d] (got %d), weights non-NULL", HPO_CLIP_MAX_WEIGHTS, n_weights);
    hpo::ClipArgs a{};
    a.d_max = d_max;
    a.d_found = d_found_inf;
    a.tau = tau;
    a.heads = heads;
    a.kv_heads = kv_heads;
    for (int32_t k = 0; k < n_weights; ++k) {
        const hpo_clip_weight& w = weights[k];
        hpo_status st = check_weight(w.master, w.param, w.d_scales);
        if (st != HPO_OK)
            return st;
        if (w.master->batch != heads && w.master->batch != kv_heads)
            return fail(HPO_EINVAL, "weight %d: %lld matrices, expected one per head (%d) or per key head (%d)", k,
                        (long long)w.master->batch, heads, kv_heads);
        if (!(w.power >= 0.0) || !is_finite(w.power))
            return fail(HPO_EINVAL, "weight %d: power must be finite and >= 0 (got %g)", k, w.power);
        if ((w.per_group != 0 && w.per_group != 1) || w.reserved != 0)
            return fail(HPO_EINVAL, "weight %d: per_group must be 0 or 1, reserved 0", k);
        if (is_empty(w.master))
            continue;
        for (int32_t j = 0; j < a.n; ++j)
            if (a.item[j].w.master.data == w.master->data)
                return fail(HPO_EINVAL, "weight %d: the same master is given twice", k);
        hpo::ClipItem& it = a.item[a.n];
        st = weight_view(w.master, w.param, w.d_scales, it.w);
        if (st != HPO_OK)
            return st;
        it.heads = static_cast<int32_t>(w.master->batch);
        it.per_group = w.per_group;
        it.power = w.power;
        ++a.n;
    }
    if (a.n == 0)
        return ok();
    const hipError_t e = hpo::launch_qk_clip(a, as_stream(stream));
    if (e != hipSuccess)
        return hip_fail(e, "launch QK-clip");
    return ok();
}

}  // extern "C"
