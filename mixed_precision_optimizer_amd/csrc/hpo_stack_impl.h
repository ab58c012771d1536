/*
 * hpo_stack_impl.h -- layouts shared by the stack operators' host code
 * (hpo_stack_api.cpp) and their kernels (hpo_rows.hip, hpo_qk.hip,
 * hpo_gram.hip, hpo_muon.hip).  Not part of the public ABI.
 */
#ifndef HPO_STACK_IMPL_H
#define HPO_STACK_IMPL_H

#include "hpo_muon_impl.h"
#include "hpo_stack.h"

namespace hpo {

/* ---------------------------------------------------------------------- */
/* row-wise updates of masters and model weights                           */
/* ---------------------------------------------------------------------- */
/* A stack as the kernels see it. */
struct StackView {
    void* data;
    int64_t bs, rs;   /* batch and row stride, elements */
};

/* Master and model weight of one stack. */
struct WeightView {
    StackView master;   /* fp32 */
    StackView param;    /* data NULL: none */
    uint8_t* scales;    /* HPO_WEIGHT_MX8 */
    int64_t rows, cols;
    int32_t param_dtype;   /* HPO_PARAM_FP32 (none), HPO_PARAM_BF16 or HPO_WEIGHT_MX8 */
};

struct RmsArgs {
    StackView O;
    WeightView w;
    float* v;        /* [batch][rows], nullable */
    double* q;       /* [batch][parts] sums of cols * ms * r^2 over a part's rows */
    float* r;        /* [batch][rows] 1 / (sqrt(v) + eps) */
    double* norm2;   /* [batch], written by the fold (large stacks only) */
    int64_t batch;
    int64_t parts;
    int32_t rounds;  /* groups of pieces per wavefront of the update */
    double beta2, eps;
    double gain;     /* lr * target_rms * sqrt(rows * cols) */
    float keep;      /* fp32(1 - lr * weight_decay) */
    int32_t o_fp32;
    const int32_t* d_found;
};

struct ClipItem {
    WeightView w;
    int64_t first_block;   /* workgroups before this weight's */
    int32_t heads;         /* matrices of the stack */
    int32_t blocks;        /* workgroups of one head */
    int32_t per_group;
    int32_t rounds;        /* groups of pieces per wavefront */
    double power;
};

struct ClipArgs {
    const float* d_max;
    const int32_t* d_found;
    double tau;
    int32_t heads, kv_heads;
    int32_t n;
    ClipItem item[HPO_CLIP_MAX_WEIGHTS];
};

hipError_t launch_rms_update(const RmsArgs& a, hipStream_t stream);
/* Fills in first_block / blocks of the items and launches. */
hipError_t launch_qk_clip(ClipArgs& a, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* attention logits                                                        */
/* ---------------------------------------------------------------------- */
struct QkArgs {
    const uint16_t* q;
    const uint16_t* k;
    int64_t qsb, qst, qsh, ksb, kst, ksh;
    const int32_t *cu_q, *cu_k, *len_q, *len_k;
    int32_t batch, heads, kv_heads, dim;
    int32_t seq_q, seq_k;      /* tokens per batch row, or in all when packed */
    int32_t max_q, max_k;      /* lengths the launch is sized for */
    int32_t causal, window;    /* window < 0: none */
    int32_t q_tiles, splits;
    int32_t accumulate;        /* out holds values of the caller's */
    float scale;
    float* out;
};

hipError_t launch_qk_max(QkArgs a, bool fp16, bool aligned, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Newton-Schulz of a stack                                                */
/* ---------------------------------------------------------------------- */
/* Scales of one Newton-Schulz step: X, A and B are held in fp16 as x * 2^ex
 * and so on; coefficients with the powers of two folded in (exact). */
struct NsStepScale {
    float gram;           /* A' = gram * (X' X'^T) */
    float poly_b, poly_c; /* B' = poly_b * A' + poly_c * (A' A'^T) */
    float step_a, step_c; /* Y = step_a * X' + step_c * (B' X'), Y = X of the next step at its scale (last: 1) */
};

/* One step in the space of the Gram matrix: coefficients, and the exponents
 * at which A, Q = a I + b A + c A^2, T = Q A and P (the product of the earlier Q)
 * are split into two fp16 values. */
struct GramStep {
    float a, b, c;
    int32_t a_exp, q_exp, t_exp, p_exp;
};

/* Short sides up to this take the Gram form. */
constexpr int64_t kGramMax = 128;

struct OrthoArgs {
    StackView G, M, out;   /* M.data NULL: no momentum */
    int32_t g_bf16;
    int32_t use_gram;      /* the short side fits and P stays in range */
    int32_t p_exp;         /* exponent of the final P */
    GramStep gram[HPO_NS_MAX_STEPS];
    int32_t steps;
    int64_t batch, rows, cols;
    MuonScalars sc;        /* gate, inv_scale, clip, momentum, eps */
    float x0_scale;        /* 2^ex of the first X */
    int32_t lift_room;     /* log2 of the most that a X alone grows beyond the bounds of X's scales */
    NsStepScale step[HPO_NS_MAX_STEPS];
    void* ws;
};

int64_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols);
int64_t gram_workspace(int64_t batch, int64_t rows, int64_t cols);
hipError_t launch_gram(const OrthoArgs& a, hipStream_t stream);
hipError_t launch_orthogonalize(const OrthoArgs& a, hipStream_t stream);

}  // namespace hpo

#endif /* HPO_STACK_IMPL_H */
