/*
 * hpo_stack.h -- C ABI of libhpo's stack operators: what a run with Muon needs
 * around the sets of hpo.h, for weights that are stacks of matrices (the heads
 * of a fused projection, the experts of a layer).
 *
 *   hpo_orthogonalize   momentum and Newton-Schulz of a stack
 *   hpo_rms_update      row-normalised update of the fp32 master and the
 *                       model weight (bf16, or 8 bits with block scales)
 *   hpo_qk_max_logits   largest attention logit of each head
 *   hpo_qk_clip         QK-clip: rescales the query / key rows of the heads
 *                       whose largest logit is over the threshold
 *
 * Sources (web pages):
 *   [OPT-INFRA]  "02 · Optimizer：算法与 infra" (llm-infra-atlas, train/02_optimizer):
 *                §5 (Muon), §6 (MuonClip's QK-clip, run after the step)
 *   [HANDBOOK]   "优化器：AdamW、Muon 与分布式优化器" (ai-infra-handbooks,
 *                train/algo/optimizer), section on Muon
 *
 * The conventions are those of hpo.h: device pointers are addresses on the
 * current device, which the call runs on; `stream` is a hipStream_t passed as
 * void*; calls only enqueue kernels (no allocation, copy or synchronisation,
 * so they can be captured in a HIP graph), argument errors are found before
 * anything is enqueued, and the return value is HPO_OK or a negative
 * hpo_status with hpo_last_error().  Nothing is kept from one call to the
 * next.  A workspace belongs to one call at a time: calls that may run at the
 * same time (two streams, two captured graphs) need a workspace each.
 */
#ifndef HPO_STACK_H
#define HPO_STACK_H

#include "hpo.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A stack of `batch` matrices of rows x cols elements in device memory:
 * element (z, i, j) is at data[z * batch_stride + i * row_stride + j] (strides
 * in elements, >= 0).  No two elements may share an address: either the
 * matrices follow one another (batch_stride >= (rows - 1) * row_stride + cols)
 * or their rows interleave (row_stride >= (batch - 1) * batch_stride + cols: the
 * heads of an output projection, side by side in every row); row_stride >=
 * cols and batch_stride >= cols where there is more than one row or matrix.
 * batch <= 65535, rows and cols <= HPO_MUON_MAX_DIM; any of them may be 0 (the
 * call then does nothing).  data needs the alignment of its element; 16-byte
 * aligned data and strides that are whole 16-byte pieces take wide accesses. */
typedef struct {
    void* data;
    int64_t batch, rows, cols;
    int64_t batch_stride, row_stride;
    int32_t dtype;     /* HPO_PARAM_BF16, HPO_PARAM_FP32 or HPO_WEIGHT_MX8, as each call says */
    int32_t reserved;  /* 0 */
} hpo_stack;

/* A model weight in 8 bits: OCP e4m3 values with one power-of-two scale for
 * each 32 consecutive elements of a row (the last block of a row may be
 * shorter).  With e = floor(log2(largest magnitude of the block)) - 8, at least
 * -127, the scale is 2^e, stored as the byte e + 127, and each value is
 * x / 2^e rounded to nearest even, at most 448 in magnitude; the weight stands
 * for value * 2^e.  A block of zeros has scale byte 0.  A block that holds an
 * inf or NaN becomes scale byte 255 and values 0x7F (NaN).
 * The scales of a stack are one contiguous uint8 array
 * [batch][rows][ceil(cols / 32)]. */
#define HPO_WEIGHT_MX8 16

/* ---------------------------------------------------------------------- */
/* Momentum and Newton-Schulz of a stack                                   */
/* ---------------------------------------------------------------------- */
/* For every matrix of the stack ([HANDBOOK] Muon listing; [OPT-INFRA] §5.2):
 *   g  = G * inv_scale, times C when max_norm > 0 clips (as hpo_muon_step);
 *   with momentum != NULL:  M = mu M + g or mu M + (1 - mu) g, and g~ as
 *     hpo_muon_step forms it (cfg's momentum, momentum_form, nesterov; fp32,
 *     one rounding per operation); without:  g~ = g;
 *   X = g~ / (||g~||_F + eps), then ns_steps times A = X X^T, B = b A + c A A,
 *   X = a X + B X (on the transpose when rows > cols);  out = bf16(X).
 * G is fp32 or bf16, momentum fp32 (updated in place), out bf16; the three
 * have one shape, each its own strides, and do not overlap.  The scale fields
 * of cfg are not read.
 *
 * Arithmetic: products on the matrix cores with fp16 operands at power-of-two
 * scales that the host derives from the coefficients (bounds on X, A and B at
 * every step), accumulated in fp32.
 *   Short side over 128: the norm in binary64; what the rounding of X to fp16
 *     loses is kept beside it for the term a X of every step but the last, so that the small
 *     singular values, which grow by a each step, keep their accuracy.  With the default five
 *     steps within 2e-3 (relative, Frobenius) of the exact iteration before the rounding to
 *     bf16; within 4e-3 with other schedules that grow by up to 2^10 in all and six default
 *     steps, 1e-2 with sixteen (3e-2 for short sides under 64).
 *   Short side up to 128 (unless the coefficients' steps multiply to more than
 *     2^11 in growth): the iteration runs on the Gram matrix of X0 in 22-bit
 *     products and the long side is touched only at its ends; the norm is the
 *     root of the Gram matrix's trace.  With the default five steps within 1e-3 before the
 *     rounding (3e-3 for long sides of 5000 and more in stacks of hundreds, or of 10^6);
 *     gradients without directions that stand out by ten and more: 2e-4.  What fp32 sums
 *     lose of the Gram matrix grows by the square of the steps' growth: beside one
 *     dominant direction 1e-2 at a growth of 2^10, 3e-2 with six default steps.
 * Coefficients whose iteration may leave |X| <= 2^15 (or |X X^T|, |b A + c A A| <= 2^15)
 * are refused (HPO_EINVAL).  The bound on the singular values starts at 1 and is
 * widened by 1 % before every step, for the roundings: those of fp16 can all fall one
 * way (equal elements), and coefficients that just hold on [0, 1] may multiply that by
 * ten and more a step.  Such a schedule passes with its argument divided by 1.01:
 * a / 1.01, b / 1.01^3, c / 1.01^5 for every step.  A matrix that is all zero
 * gives zeros, as does one whose norm (or an ns_eps that) is beyond fp32's largest value; one that
 * holds an inf or NaN gives NaN everywhere.
 * The same inputs give the same bits.
 * With a non-zero *d_found_inf (nullable) nothing is written. */
hpo_status hpo_orthogonalize(const hpo_stack* G, const hpo_stack* momentum, const hpo_stack* out,
                             const hpo_muon_cfg* cfg, float inv_scale, double max_norm, const float* d_norm,
                             const int32_t* d_found_inf, void* d_workspace, int64_t workspace_bytes, void* stream);
/* Bytes of the workspace (256-byte aligned) for such a stack. */
hpo_status hpo_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols, int64_t* out_bytes);

/* ---------------------------------------------------------------------- */
/* Row-normalised update                                                   */
/* ---------------------------------------------------------------------- */
/* For every matrix O of a stack of updates (bf16 or fp32, for example
 * hpo_orthogonalize's output) and its fp32 master W:
 *   ms_i = mean over j of O_ij^2
 *   v_i  = beta2 v_i + (1 - beta2) ms_i       (d_v, fp32 [batch][rows], in place)
 *   r_i  = 1 / (sqrt(v_i) + eps)
 *   N    = sqrt(sum over i of cols * ms_i * r_i^2)   (the norm of the rows r_i O_i)
 *   s    = lr * target_rms * sqrt(rows * cols) / N,  0 where N is 0 or not a number
 *   W    = fp32(W * fp32(1 - lr * weight_decay)); W_ij = fp32(W_ij - fp32(s r_i) O_ij)
 * and the model weight, if param is given, takes W rounded to nearest even to
 * bf16, or to HPO_WEIGHT_MX8 with d_scales.  beta2 = 0 is the plain
 * root-mean-square norm of each row (d_v may then be NULL; it is written, not
 * read, if it is given).  Squares and the mean are summed in fp32 per lane and in
 * binary64 across lanes; N and s in binary64, r_i rounded to fp32 where it meets s (r_i
 * and s r_i at most fp32's largest value in magnitude: rows of zeros stay).  The sums'
 * order is fixed: the same inputs give the same bits.
 * 0 <= beta2 < 1; eps >= 0, and a row with sqrt(v_i) + eps = 0 is left out of the
 * update; lr, weight_decay and target_rms are finite.  A stack has at most 2^24 rows
 * in all.  O, the master, the model weight, d_scales and d_v do not overlap.
 * With a non-zero *d_found_inf (nullable) nothing is written. */
typedef struct {
    double lr;
    double weight_decay;
    double beta2;
    double eps;
    double target_rms;   /* root mean square of the update before lr */
} hpo_rms_cfg;

hpo_status hpo_rms_update(const hpo_stack* O, const hpo_stack* master, float* d_v, const hpo_stack* param,
                          uint8_t* d_scales, const hpo_rms_cfg* cfg, const int32_t* d_found_inf, void* d_workspace,
                          int64_t workspace_bytes, void* stream);
/* Bytes of the workspace (8-byte aligned). */
hpo_status hpo_rms_update_workspace(int64_t batch, int64_t rows, int64_t* out_bytes);

/* ---------------------------------------------------------------------- */
/* Largest attention logit of each head                                    */
/* ---------------------------------------------------------------------- */
/* Queries and keys as the attention of a training step sees them, bf16 or
 * fp16.  Element (b, t, h, d) of q is at q[b * q_stride_batch + t *
 * q_stride_token + h * q_stride_head + d], k alike (strides in elements); query head h
 * reads key head h / (heads / kv_heads).
 *   Padded batch (cu_seqlens_* NULL): batch rows of seq_q / seq_k tokens, of
 *     which the first seqlens_q[b] / seqlens_k[b] count (device int32,
 *     nullable: all).
 *   Packed (both cu_seqlens_* given, device int32 [batch + 1]): sequence b is
 *     tokens cu[b] .. cu[b + 1] - 1 of seq_q / seq_k tokens in all; the batch
 *     strides and seqlens_* are not read (seqlens_* must be NULL).  max_seqlen_* say
 *     how long a sequence may be (they size the launch; a longer one is still
 *     seen whole).
 * Lengths and offsets read from the device are cut to [0, seq_*].
 * Query i sees key j of its sequence when, with at = i + len_k - len_q,
 *   causal = 0: always;   causal = 1: j <= at, and j >= at - window when window >= 0. */
typedef struct {
    const void* q;
    const void* k;
    int32_t dtype;              /* HPO_PARAM_BF16 or HPO_PARAM_FP16 */
    int32_t batch;
    int32_t heads, kv_heads;    /* heads a multiple of kv_heads */
    int32_t head_dim;           /* 1 .. HPO_QK_MAX_DIM */
    int32_t causal;
    int64_t window;             /* -1: none; >= 0 only with causal = 1 */
    int64_t seq_q, seq_k;
    int64_t max_seqlen_q, max_seqlen_k;   /* packed only */
    int64_t q_stride_batch, q_stride_token, q_stride_head;
    int64_t k_stride_batch, k_stride_token, k_stride_head;
    const int32_t* cu_seqlens_q;
    const int32_t* cu_seqlens_k;
    const int32_t* seqlens_q;
    const int32_t* seqlens_k;
    float scale;                /* > 0, finite */
    int32_t reserved;           /* 0 */
} hpo_qk;

#define HPO_QK_MAX_DIM 256
/* Largest token stride (elements): 64 key rows are addressed with 32-bit
 * byte offsets. */
#define HPO_QK_MAX_STRIDE (((int64_t)1) << 23)

/* d_max[h] (device fp32, `heads` of them) = the largest scale * (q . k) over all
 * pairs that head h sees, in every sequence ([OPT-INFRA] §6: S_max^h); products
 * exact, sums in fp32 on the matrix cores.  -inf where no pair is seen; NaN if
 * a seen logit is NaN (values behind the mask or behind a sequence's end never
 * count).  accumulate = 1 takes the larger of that and d_max[h] as it is (NaN if
 * either is): the maximum over micro-batches.  The result does not depend on the order of the
 * work. */
hpo_status hpo_qk_max_logits(const hpo_qk* a, int32_t accumulate, float* d_max, void* stream);

/* ---------------------------------------------------------------------- */
/* QK-clip                                                                 */
/* ---------------------------------------------------------------------- */
/* One weight to clip: a stack with one matrix per head (rows = the head's
 * rows of the projection), its model weight and the power of gamma it takes:
 * 0.5 for query and key weights that share the clip, 1 for one that takes it all
 * ([OPT-INFRA] §6). */
typedef struct {
    const hpo_stack* master;   /* fp32 */
    const hpo_stack* param;    /* bf16 or HPO_WEIGHT_MX8, nullable */
    uint8_t* d_scales;         /* HPO_WEIGHT_MX8 only */
    double power;              /* finite, >= 0 */
    int32_t per_group;         /* 1: every head of a key group takes the group's smallest gamma */
    int32_t reserved;          /* 0 */
} hpo_clip_weight;

#define HPO_CLIP_MAX_WEIGHTS 8

/* gamma_h = tau / S_h where S_h = d_max[h] is finite and over tau, else 1.  A
 * weight of `heads` matrices takes gamma_h (per_group: the smallest of its
 * key group); one of kv_heads matrices always takes its group's.  Every row of a
 * head whose gamma is under 1: W = fp32(W * f) with f = fp32(gamma^power), and
 * the model weight takes W rounded as in hpo_rms_update.  The rows of the other heads
 * are neither read nor written. With heads == kv_heads both
 * readings are one.  1 <= n_weights <= HPO_CLIP_MAX_WEIGHTS; tau > 0.  The weights do
 * not overlap (views of one buffer are fine); one given twice is refused.
 * With a non-zero *d_found_inf (nullable) nothing is written. */
hpo_status hpo_qk_clip(const float* d_max, int32_t heads, int32_t kv_heads, double tau, const hpo_clip_weight* weights,
                       int32_t n_weights, const int32_t* d_found_inf, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* HPO_STACK_H */
