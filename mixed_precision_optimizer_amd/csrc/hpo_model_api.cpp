/*
 * hpo_model_api.cpp -- host side of the model operators (hpo_model.h):
 * argument checks and launches.  Host code only (compiled as plain C++ against
 * the HIP runtime API).
 */
#include <cmath>
#include <cstdint>

#include "hpo_model_impl.h"
#include "hpo_set.h"

using namespace hpo_host;

namespace {

bool is_float(int32_t dtype)
{
    return dtype == HPO_PARAM_BF16 || dtype == HPO_PARAM_FP16 || dtype == HPO_PARAM_FP32;
}

bool is_16bit(int32_t dtype) { return dtype == HPO_PARAM_BF16 || dtype == HPO_PARAM_FP16; }

bool is_grad(int32_t dtype) { return dtype == HPO_PARAM_FP32 || dtype == HPO_PARAM_BF16; }

hpo_status check_dims(const hpo_stack* s, const char* what, int64_t batch, int64_t rows, int64_t cols)
{
    const hpo_status st = check_stack(s, what);
    if (st != HPO_OK)
        return st;
    if (s->batch != batch || s->rows != rows || s->cols != cols)
        return fail(HPO_EINVAL, "%s is %lld x %lld x %lld, expected %lld x %lld x %lld", what, (long long)s->batch,
                    (long long)s->rows, (long long)s->cols, (long long)batch, (long long)rows, (long long)cols);
    return HPO_OK;
}

hpo_status check_ids(const void* d_ids, int32_t id_bytes, int64_t n, int64_t first)
{
    if (id_bytes != 4 && id_bytes != 8)
        return fail(HPO_EDTYPE, "id_bytes must be 4 or 8 (got %d)", id_bytes);
    if (n < 0 || n > HPO_MUON_MAX_DIM)
        return fail(HPO_EINVAL, "n must lie in [0, %lld] (got %lld)", (long long)HPO_MUON_MAX_DIM, (long long)n);
    if (first < 0 || first > (int64_t{1} << 62))
        return fail(HPO_EINVAL, "first must lie in [0, 2^62] (got %lld)", (long long)first);
    if (n > 0 && (!d_ids || !aligned(d_ids, static_cast<uintptr_t>(id_bytes))))
        return fail(HPO_EINVAL, "d_ids must be a non-NULL device pointer aligned to %d bytes", id_bytes);
    return HPO_OK;
}

hpo_status check_one(const hpo_stack* s, const char* what)
{
    const hpo_status st = check_stack(s, what);
    if (st != HPO_OK)
        return st;
    if (s->batch != 1)
        return fail(HPO_EINVAL, "%s must be one matrix (batch 1, got %lld)", what, (long long)s->batch);
    return HPO_OK;
}

hpo_status check_scale(float scale)
{
    return std::isfinite(scale) ? HPO_OK : fail(HPO_EINVAL, "scale must be finite");
}

hpo_status check_workspace(const void* ws, int64_t bytes, int64_t need)
{
    if (need == 0)
        return HPO_OK;
    if (!ws || !aligned(ws, 256))
        return fail(HPO_EINVAL, "d_workspace must be a non-NULL, 256-byte aligned device pointer");
    if (bytes < need)
        return fail(HPO_EINVAL, "workspace of %lld bytes is below the %lld this call needs", (long long)bytes,
                    (long long)need);
    return HPO_OK;
}

/* An 8-bit operand of a product. */
hpo_status check_mx8(const hpo_stack* s, const uint8_t* scales, const char* what)
{
    const hpo_status st = check_stack(s, what);
    if (st != HPO_OK)
        return st;
    if (s->dtype != HPO_WEIGHT_MX8)
        return fail(HPO_EDTYPE, "%s must be HPO_WEIGHT_MX8", what);
    if (!scales && !is_empty(s))
        return fail(HPO_EINVAL, "%s needs its scales", what);
    return HPO_OK;
}

hpo_status workspace(hpo::ProductKind kind, int64_t batch, int64_t m, int64_t n, int64_t k, int64_t* out)
{
    if (!out)
        return fail(HPO_EINVAL, "out_bytes is NULL");
    const int64_t most = HPO_MUON_MAX_DIM;
    if (batch < 0 || m < 0 || n < 0 || k < 0 || batch > 65535 || m > most || n > most || k > most)
        return fail(HPO_EINVAL, "bad shape: %lld products of %lld x %lld x %lld", (long long)batch, (long long)m,
                    (long long)n, (long long)k);
    *out = batch == 0 || m == 0 || n == 0 ? 0 : hpo::product_workspace(kind, batch, m, n, k);
    return ok();
}

/* What the products share; a, b and the dtypes are the caller's. */
hpo_status run_product(hpo::ProductKind kind, hpo::ProductArgs& p, const hpo_stack* a, const hpo_stack* b,
                       const hpo_stack* c, int64_t k, void* ws, int64_t ws_bytes, void* stream)
{
    p.batch = c->batch;
    p.m = c->rows;
    p.n = c->cols;
    p.k = k;
    int64_t need = 0;
    hpo_status st = workspace(kind, p.batch, p.m, p.n, p.k, &need);
    if (st != HPO_OK)
        return st;
    if (is_empty(c))
        return ok();
    st = check_workspace(ws, ws_bytes, need);
    if (st != HPO_OK)
        return st;
    const hpo::StackView va = view(a), vb = view(b), vc = view(c);
    p.a = va.data;
    p.a_bs = va.bs;
    p.a_rs = va.rs;
    p.b = static_cast<const uint8_t*>(vb.data);
    p.b_bs = vb.bs;
    p.b_rs = vb.rs;
    p.c = vc.data;
    p.c_bs = vc.bs;
    p.c_rs = vc.rs;
    p.c_dtype = c->dtype;
    p.part = static_cast<float*>(ws);
    const hipError_t e = hpo::launch_product(kind, p, as_stream(stream));
    if (e == hipErrorInvalidConfiguration)
        return fail(HPO_EINVAL, "the product has more tiles than one launch can hold");
    if (e != hipSuccess)
        return hip_fail(e, "launch 8-bit product");
    return ok();
}

}  // namespace

extern "C" {

hpo_status hpo_embedding(const void* d_ids, int32_t id_bytes, int64_t n, int64_t first, const hpo_stack* weight,
                         const uint8_t* d_scales, float scale, const hpo_stack* out, void* stream)
{
    hpo_status st = check_ids(d_ids, id_bytes, n, first);
    if (st != HPO_OK)
        return st;
    st = check_one(weight, "weight");
    if (st != HPO_OK)
        return st;
    if (!is_float(weight->dtype) && weight->dtype != HPO_WEIGHT_MX8)
        return fail(HPO_EDTYPE, "weight dtype %d is not supported (bf16 = 0, fp32 = 1, fp16 = 2, 8 bits = 16)",
                    weight->dtype);
    if (weight->dtype == HPO_WEIGHT_MX8 && !d_scales && !is_empty(weight))
        return fail(HPO_EINVAL, "an 8-bit weight needs d_scales");
    if (weight->dtype != HPO_WEIGHT_MX8 && d_scales)
        return fail(HPO_EINVAL, "d_scales is for an 8-bit weight");
    st = check_dims(out, "out", 1, n, weight->cols);
    if (st != HPO_OK)
        return st;
    if (!is_float(out->dtype))
        return fail(HPO_EDTYPE, "out dtype %d is not supported (bf16 = 0, fp32 = 1, fp16 = 2)", out->dtype);
    st = check_scale(scale);
    if (st != HPO_OK)
        return st;
    if (is_empty(out))
        return ok();
    hpo::EmbedArgs a{};
    a.ids = d_ids;
    a.id64 = id_bytes == 8 ? 1 : 0;
    a.w_dtype = weight->dtype;
    a.out_dtype = out->dtype;
    a.n = n;
    a.first = first;
    a.rows = weight->rows;
    a.cols = weight->cols;
    a.w = weight->data;
    a.w_rs = view(weight).rs;
    a.scales = d_scales;
    a.out = out->data;
    a.out_rs = view(out).rs;
    a.scale = scale;
    const hipError_t e = hpo::launch_embedding(a, as_stream(stream));
    if (e != hipSuccess)
        return hip_fail(e, "launch embedding");
    return ok();
}

hpo_status hpo_embedding_grad_workspace(int64_t n, int64_t cols, int64_t* out_bytes)
{
    if (!out_bytes)
        return fail(HPO_EINVAL, "out_bytes is NULL");
    if (n < 0 || cols < 0 || n > HPO_MUON_MAX_DIM || cols > HPO_MUON_MAX_DIM)
        return fail(HPO_EINVAL, "bad shape: %lld rows of %lld elements", (long long)n, (long long)cols);
    *out_bytes = n == 0 || cols == 0 ? 0 : hpo::embed_grad_workspace(n, cols);
    return ok();
}

hpo_status hpo_embedding_grad(const void* d_ids, int32_t id_bytes, int64_t n, int64_t first, const hpo_stack* dy,
                              float scale, const hpo_stack* grad, void* d_workspace, int64_t workspace_bytes,
                              void* stream)
{
    hpo_status st = check_ids(d_ids, id_bytes, n, first);
    if (st != HPO_OK)
        return st;
    st = check_one(grad, "grad");
    if (st != HPO_OK)
        return st;
    if (!is_grad(grad->dtype))
        return fail(HPO_EDTYPE, "grad dtype %d is not supported (bf16 = 0, fp32 = 1)", grad->dtype);
    st = check_dims(dy, "dy", 1, n, grad->cols);
    if (st != HPO_OK)
        return st;
    if (!is_float(dy->dtype))
        return fail(HPO_EDTYPE, "dy dtype %d is not supported (bf16 = 0, fp32 = 1, fp16 = 2)", dy->dtype);
    st = check_scale(scale);
    if (st != HPO_OK)
        return st;
    if (is_empty(dy) || is_empty(grad))
        return ok();
    int64_t need = 0;
    st = hpo_embedding_grad_workspace(n, grad->cols, &need);
    if (st != HPO_OK)
        return st;
    st = check_workspace(d_workspace, workspace_bytes, need);
    if (st != HPO_OK)
        return st;
    hpo::EmbedGradArgs a{};
    a.ids = d_ids;
    a.id64 = id_bytes == 8 ? 1 : 0;
    a.dy_dtype = dy->dtype;
    a.g_dtype = grad->dtype;
    a.n = n;
    a.first = first;
    a.rows = grad->rows;
    a.cols = grad->cols;
    a.dy = dy->data;
    a.dy_rs = view(dy).rs;
    a.g = grad->data;
    a.g_rs = view(grad).rs;
    a.scale = scale;
    a.ws = d_workspace;
    const hipError_t e = hpo::launch_embedding_grad(a, as_stream(stream));
    if (e != hipSuccess)
        return hip_fail(e, "launch embedding gradient");
    return ok();
}

hpo_status hpo_mx8_save(const hpo_stack* x, const hpo_stack* q, uint8_t* d_scales, void* stream)
{
    hpo_status st = check_stack(x, "x");
    if (st != HPO_OK)
        return st;
    if (!is_float(x->dtype))
        return fail(HPO_EDTYPE, "x dtype %d is not supported (bf16 = 0, fp32 = 1, fp16 = 2)", x->dtype);
    st = check_like(q, "q", x, "x");
    if (st != HPO_OK)
        return st;
    st = check_mx8(q, d_scales, "q");
    if (st != HPO_OK)
        return st;
    if (is_empty(x))
        return ok();
    hpo::SaveArgs a{};
    a.x = view(x);
    a.q = view(q);
    a.scales = d_scales;
    a.x_dtype = x->dtype;
    a.batch = x->batch;
    a.rows = x->rows;
    a.cols = x->cols;
    const hipError_t e = hpo::launch_mx8_save(a, as_stream(stream));
    if (e != hipSuccess)
        return hip_fail(e, "launch 8-bit activation");
    return ok();
}

hpo_status hpo_mx8_linear_workspace(int64_t batch, int64_t tokens, int64_t cols, int64_t rows, int64_t* out_bytes)
{
    return workspace(hpo::kLinear, batch, tokens, rows, cols, out_bytes);
}

hpo_status hpo_mx8_dgrad_workspace(int64_t batch, int64_t tokens, int64_t cols, int64_t rows, int64_t* out_bytes)
{
    return workspace(hpo::kDgrad, batch, tokens, cols, rows, out_bytes);
}

hpo_status hpo_mx8_wgrad_workspace(int64_t batch, int64_t tokens, int64_t cols, int64_t rows, int64_t* out_bytes)
{
    return workspace(hpo::kWgrad, batch, rows, cols, tokens, out_bytes);
}

hpo_status hpo_mx8_linear(const hpo_stack* x, const uint8_t* d_x_scales, const hpo_stack* w, const uint8_t* d_w_scales,
                          const hpo_stack* y, void* d_workspace, int64_t workspace_bytes, void* stream)
{
    hpo_status st = check_mx8(x, d_x_scales, "x");
    if (st != HPO_OK)
        return st;
    st = check_mx8(w, d_w_scales, "w");
    if (st != HPO_OK)
        return st;
    if (w->batch != x->batch || w->cols != x->cols)
        return fail(HPO_EINVAL, "x is %lld x %lld x %lld, w %lld x %lld x %lld: batch and cols must agree",
                    (long long)x->batch, (long long)x->rows, (long long)x->cols, (long long)w->batch, (long long)w->rows,
                    (long long)w->cols);
    st = check_dims(y, "y", x->batch, x->rows, w->rows);
    if (st != HPO_OK)
        return st;
    if (!is_16bit(y->dtype))
        return fail(HPO_EDTYPE, "y dtype %d is not supported (bf16 = 0, fp16 = 2)", y->dtype);
    hpo::ProductArgs p{};
    p.a_scales = d_x_scales;
    p.b_scales = d_w_scales;
    p.scale = 1.0f;
    return run_product(hpo::kLinear, p, x, w, y, x->cols, d_workspace, workspace_bytes, stream);
}

hpo_status hpo_mx8_dgrad(const hpo_stack* dy, const hpo_stack* w, const uint8_t* d_w_scales, const hpo_stack* dx,
                         void* d_workspace, int64_t workspace_bytes, void* stream)
{
    hpo_status st = check_mx8(w, d_w_scales, "w");
    if (st != HPO_OK)
        return st;
    st = check_stack(dy, "dy");
    if (st != HPO_OK)
        return st;
    if (!is_16bit(dy->dtype))
        return fail(HPO_EDTYPE, "dy dtype %d is not supported (bf16 = 0, fp16 = 2)", dy->dtype);
    if (dy->batch != w->batch || dy->cols != w->rows)
        return fail(HPO_EINVAL, "dy is %lld x %lld x %lld, w %lld x %lld x %lld: batch must agree, dy's cols with w's rows",
                    (long long)dy->batch, (long long)dy->rows, (long long)dy->cols, (long long)w->batch,
                    (long long)w->rows, (long long)w->cols);
    st = check_dims(dx, "dx", dy->batch, dy->rows, w->cols);
    if (st != HPO_OK)
        return st;
    if (!is_float(dx->dtype))
        return fail(HPO_EDTYPE, "dx dtype %d is not supported (bf16 = 0, fp32 = 1, fp16 = 2)", dx->dtype);
    hpo::ProductArgs p{};
    p.b_scales = d_w_scales;
    p.scale = 1.0f;
    p.fp16 = dy->dtype == HPO_PARAM_FP16 ? 1 : 0;
    return run_product(hpo::kDgrad, p, dy, w, dx, dy->cols, d_workspace, workspace_bytes, stream);
}

hpo_status hpo_mx8_wgrad(const hpo_stack* dy, const hpo_stack* x, const uint8_t* d_x_scales, float scale,
                         int32_t accumulate, const hpo_stack* grad, void* d_workspace, int64_t workspace_bytes,
                         void* stream)
{
    hpo_status st = check_mx8(x, d_x_scales, "x");
    if (st != HPO_OK)
        return st;
    st = check_stack(dy, "dy");
    if (st != HPO_OK)
        return st;
    if (!is_16bit(dy->dtype))
        return fail(HPO_EDTYPE, "dy dtype %d is not supported (bf16 = 0, fp16 = 2)", dy->dtype);
    if (dy->batch != x->batch || dy->rows != x->rows)
        return fail(HPO_EINVAL, "dy is %lld x %lld x %lld, x %lld x %lld x %lld: batch and rows must agree",
                    (long long)dy->batch, (long long)dy->rows, (long long)dy->cols, (long long)x->batch,
                    (long long)x->rows, (long long)x->cols);
    st = check_dims(grad, "grad", dy->batch, dy->cols, x->cols);
    if (st != HPO_OK)
        return st;
    if (!is_grad(grad->dtype))
        return fail(HPO_EDTYPE, "grad dtype %d is not supported (bf16 = 0, fp32 = 1)", grad->dtype);
    if (accumulate != 0 && accumulate != 1)
        return fail(HPO_EINVAL, "accumulate must be 0 or 1 (got %d)", accumulate);
    st = check_scale(scale);
    if (st != HPO_OK)
        return st;
    if (accumulate && dy->rows == 0)
        return ok();   /* a sum of nothing */
    hpo::ProductArgs p{};
    p.b_scales = d_x_scales;
    p.scale = scale;
    p.accumulate = accumulate;
    p.fp16 = dy->dtype == HPO_PARAM_FP16 ? 1 : 0;
    return run_product(hpo::kWgrad, p, dy, x, grad, dy->rows, d_workspace, workspace_bytes, stream);
}

}  // extern "C"
