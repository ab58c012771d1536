/*
 * hpo_muon_device.h -- device helpers shared by the Muon kernel files
 * (hpo_muon.hip, hpo_gram.hip).  Not part of the public ABI.
 *
 * Source: [OPT-INFRA] "02 · Optimizer：算法与 infra" (llm-infra-atlas, train/02_optimizer).
 */
#ifndef HPO_MUON_DEVICE_H
#define HPO_MUON_DEVICE_H

#include <hip/hip_runtime.h>

#include <cfloat>

#include "hpo_device.h"
#include "hpo_stack_impl.h"

namespace hpo {
namespace {

/* ---------------------------------------------------------------------- */
/* gates and per-step values                                              */
/* ---------------------------------------------------------------------- */
__device__ __forceinline__ bool gate_open(const MuonGate& g)
{
    if (g.dev) {
        /* the finalize has decided and counted the step (t = applied_steps, in the window) */
        if (!g.st->applied)
            return false;
        const int64_t j = g.st->applied_steps - g.t_first;
        return j >= 0 && j < g.window;
    }
    return !(g.d_found != nullptr && *g.d_found != 0);
}

struct GradVals {
    float inv_scale;
    float C;
    bool clip;
};

/* Unscale factor and clip coefficient ([OPT-INFRA] §11.1): the same global
 * norm and rule as the AdamW update of the same step. */
__device__ __forceinline__ GradVals grad_vals(const MuonScalars& sc)
{
    GradVals v;
    float norm = 0.0f;
    if (sc.gate.dev) {
        v.inv_scale = sc.gate.st->step_inv_scale;
        norm = sc.gate.st->grad_norm;
    } else {
        v.inv_scale = sc.inv_scale;
        if (sc.max_norm > 0.0)
            norm = *sc.d_norm;
    }
    v.clip = false;
    v.C = 1.0f;
    if (sc.max_norm > 0.0) {
        const double c = sc.max_norm / (static_cast<double>(norm) + 1e-6);
        if (c < 1.0) {
            v.clip = true;
            v.C = static_cast<float>(c);
        }
    }
    return v;
}

/* ---------------------------------------------------------------------- */
/* a stack's gradient and momentum                                         */
/* ---------------------------------------------------------------------- */
struct OrthoSrc {
    const void* G;
    int64_t gbs, grs;
    float* M;
    int64_t mbs, mrs;
    int64_t rows, cols;
    MuonScalars sc;
};

/* The matrices of a stack from z0 on. */
inline OrthoSrc slice_of(const OrthoArgs& a, int64_t z0)
{
    OrthoSrc s{};
    s.G = static_cast<const char*>(a.G.data) + (a.g_bf16 ? 2 : 4) * z0 * a.G.bs;
    s.gbs = a.G.bs;
    s.grs = a.G.rs;
    s.M = a.M.data ? static_cast<float*>(a.M.data) + z0 * a.M.bs : nullptr;
    s.mbs = a.M.bs;
    s.mrs = a.M.rs;
    s.rows = a.rows;
    s.cols = a.cols;
    s.sc = a.sc;
    return s;
}

template <bool BF16>
__device__ __forceinline__ float src_at(const OrthoSrc& s, int64_t off)
{
    if constexpr (BF16)
        return bf16_to_f32(static_cast<const uint16_t*>(s.G)[off]);
    else
        return static_cast<const float*>(s.G)[off];
}

/* g~ of one element from the stored grad and, when there is one, the momentum
 * after this step's update. */
__device__ __forceinline__ float nesterov_of(float g, float M, const MuonScalars& sc)
{
    if (!sc.nesterov)
        return M;
    return sc.form == HPO_MUON_MOMENTUM_SUM ? g + sc.mu * M : sc.omu * g + sc.mu * M;
}

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
/* four elements at any element's address (one instruction in global memory) */
typedef f32x4_t f32x4_any __attribute__((aligned(4)));
typedef u32x2_t u32x2_any __attribute__((aligned(2)));

/* Where X0 is held larger than it is: under 2^-10 of eps the iteration's cubic terms are under
 * 2^-18 of its linear ones.  An eps beyond fp32 came here as infinity and gives zeros. */
__device__ __forceinline__ bool far_below_eps(double norm, float eps)
{
    return norm > 0.0 && eps <= FLT_MAX && norm < 0x1p-10 * static_cast<double>(eps);
}

/* Four consecutive stored elements: n of them are there (the others read as 0). */
template <bool BF16>
__device__ __forceinline__ f32x4_t grad4(const OrthoSrc& s, int64_t at, int64_t n)
{
    f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n >= 4) {
        if constexpr (BF16) {
            const u32x2_t t = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(s.G) + at);
            x[0] = bf16_to_f32(t.x & 0xffffu);
            x[1] = bf16_to_f32(t.x >> 16);
            x[2] = bf16_to_f32(t.y & 0xffffu);
            x[3] = bf16_to_f32(t.y >> 16);
        } else {
            x = *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(s.G) + at);
        }
        return x;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n)
            x[e] = src_at<BF16>(s, at + e);
    return x;
}

__device__ __forceinline__ f32x4_t momentum4(const OrthoSrc& s, int64_t at, int64_t n)
{
    f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n >= 4)
        return *reinterpret_cast<const f32x4_any*>(s.M + at);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n)
            x[e] = s.M[at + e];
    return x;
}

__device__ __forceinline__ void put_momentum4(const OrthoSrc& s, int64_t at, int64_t n, f32x4_t x)
{
    if (n >= 4) {
        *reinterpret_cast<f32x4_any*>(s.M + at) = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n)
            s.M[at + e] = x[e];
}

__device__ __forceinline__ uint32_t f16_bits(float x)
{
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

__device__ __forceinline__ float f16v(uint16_t b) { return static_cast<float>(__builtin_bit_cast(_Float16, b)); }

}  // namespace
}  // namespace hpo

#endif /* HPO_MUON_DEVICE_H */
