/*
 * hpo_model_impl.h -- layouts shared by the model operators' host code
 * (hpo_model_api.cpp) and their kernels (hpo_embed.hip, hpo_mx8.hip).  Not
 * part of the public ABI.
 */
#ifndef HPO_MODEL_IMPL_H
#define HPO_MODEL_IMPL_H

#include "hpo_model.h"
#include "hpo_stack_impl.h"

namespace hpo {

/* ---------------------------------------------------------------------- */
/* embedding                                                               */
/* ---------------------------------------------------------------------- */
struct EmbedArgs {
    const void* ids;
    int32_t id64;
    int32_t w_dtype, out_dtype;
    int64_t n, first, rows, cols;
    const void* w;
    int64_t w_rs;
    const uint8_t* scales;   /* HPO_WEIGHT_MX8 */
    void* out;
    int64_t out_rs;
    float scale;
};

struct EmbedGradArgs {
    const void* ids;
    int32_t id64;
    int32_t dy_dtype, g_dtype;
    int64_t n, first, rows, cols;
    const void* dy;
    int64_t dy_rs;
    void* g;
    int64_t g_rs;
    float scale;
    void* ws;
};

int64_t embed_grad_workspace(int64_t n, int64_t cols);
hipError_t launch_embedding(const EmbedArgs& a, hipStream_t stream);
hipError_t launch_embedding_grad(const EmbedGradArgs& a, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* 8-bit activations and products                                          */
/* ---------------------------------------------------------------------- */
struct SaveArgs {
    StackView x, q;
    uint8_t* scales;
    int32_t x_dtype;
    int64_t batch, rows, cols;
};

hipError_t launch_mx8_save(const SaveArgs& a, hipStream_t stream);

enum ProductKind : int32_t { kLinear = 0, kDgrad = 1, kWgrad = 2 };

/* C[m][n] = sum over k of A[m][k] B[n][k], per matrix of the stacks:
 *            m       n      k       A             B
 *   linear   tokens  rows   cols    x  [m][k]     w [n][k]    both 8 bits
 *   dgrad    tokens  cols   rows    dY [m][k]     w [k][n]    16 bits, 8 bits
 *   wgrad    rows    cols   tokens  dY [k][m]     x [k][n]    16 bits, 8 bits
 * Strides in elements. */
struct ProductArgs {
    const void* a;
    const uint8_t* a_scales;    /* linear */
    const uint8_t* b;
    const uint8_t* b_scales;
    int64_t a_bs, a_rs, b_bs, b_rs, c_bs, c_rs;
    int64_t batch, m, n, k;
    void* c;
    float* part;                /* [batch][splits][m][n] sums of the splits, splits > 1 */
    float scale;
    int32_t accumulate;
    int32_t c_dtype;
    int32_t fp16;               /* A is fp16, not bf16 (dgrad, wgrad) */
    int32_t tiles_m, tiles_n, splits;
};

int64_t product_workspace(ProductKind kind, int64_t batch, int64_t m, int64_t n, int64_t k);
/* hpo_mx8_grad.hip: the tiles of dgrad and wgrad. */
hipError_t launch_mx8_grad(bool wgrad, const ProductArgs& p, int32_t tile, bool direct, uint32_t grid, hipStream_t stream);
hipError_t launch_product(ProductKind kind, ProductArgs a, hipStream_t stream);

}  // namespace hpo

#endif /* HPO_MODEL_IMPL_H */
