/*
 * hpo_model_device.h -- device helpers shared by the model operators' kernel
 * files (hpo_embed.hip, hpo_mx8.hip): runs of elements of a row in fp32, and
 * the 8-bit block format.  Not part of the public ABI.
 */
#ifndef HPO_MODEL_DEVICE_H
#define HPO_MODEL_DEVICE_H

#include "hpo_device.h"
#include "hpo_model_impl.h"

namespace hpo {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
/* Vectors at any element's address: global memory takes such an access in one
 * instruction, a line more where it straddles one. */
typedef f32x4_t f32x4_any __attribute__((aligned(4)));
typedef u32x4_t u32x4_any4 __attribute__((aligned(4)));
typedef u32x4_t u32x4_any2 __attribute__((aligned(2)));
typedef u32x2_t u32x2_any2 __attribute__((aligned(2)));
typedef u32x4_t u32x4_any __attribute__((aligned(1)));
typedef u32x2_t u32x2_any __attribute__((aligned(1)));

constexpr int kMxBlock = 32;

__device__ __forceinline__ float f16_to_f32(uint32_t b)
{
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(b)));
}

__device__ __forceinline__ uint32_t f16_bits(float x)
{
    return __builtin_bit_cast(uint16_t, static_cast<_Float16>(x));
}

/* A 16-bit value of type DT in fp32, and back (round to nearest even). */
template <int DT>
__device__ __forceinline__ float widen(uint32_t b)
{
    return DT == HPO_PARAM_BF16 ? bf16_to_f32(b & 0xffffu) : f16_to_f32(b);
}

template <int DT>
__device__ __forceinline__ uint32_t narrow(float x)
{
    return DT == HPO_PARAM_BF16 ? bf16_rne_bits(x) : f16_bits(x);
}

/* Two neighbours of type DT, rounded to nearest even by the hardware's conversion (a NaN stays one). */
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    if constexpr (DT == HPO_PARAM_BF16)
        return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
    else
        return f16_bits(a) | (f16_bits(b) << 16);
}

/* n of eight 16-bit elements (n <= 0: none) as they are. */
__device__ __forceinline__ void store_raw8(uint16_t* p, int n, u32x4_t x)
{
    if (n >= 8) {
        *reinterpret_cast<u32x4_any2*>(p) = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n)
            p[e] = static_cast<uint16_t>(x[e >> 1] >> (16 * (e & 1)));
}

/* Eight consecutive elements of type DT as they are stored: loads that nothing waits for yet. */
template <int DT>
struct Raw8 {
    u32x4_t v[DT == HPO_PARAM_FP32 ? 2 : 1];
};

/* From element `at` on, n of them in the row (n <= 0: none; the others come as 0). */
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const void* base, int64_t at, int n)
{
    Raw8<DT> r;
    if constexpr (DT == HPO_PARAM_FP32) {
        const uint32_t* p = static_cast<const uint32_t*>(base) + at;
        if (n >= 8) {
            r.v[0] = *reinterpret_cast<const u32x4_any4*>(p);
            r.v[1] = *reinterpret_cast<const u32x4_any4*>(p + 4);
        } else {
            r.v[0] = u32x4_t{0, 0, 0, 0};
            r.v[1] = u32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n)
                    r.v[e >> 2][e & 3] = p[e];
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(base) + at;
        if (n >= 8) {
            r.v[0] = *reinterpret_cast<const u32x4_any2*>(p);
        } else {
            r.v[0] = u32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n)
                    r.v[0][e >> 1] |= static_cast<uint32_t>(p[e]) << (16 * (e & 1));
        }
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void unpack8(const Raw8<DT>& r, float (&x)[8])
{
    if constexpr (DT == HPO_PARAM_FP32) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] = __uint_as_float(r.v[e >> 2][e & 3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = widen<DT>(r.v[0][e] & 0xffffu);
            x[2 * e + 1] = widen<DT>(r.v[0][e] >> 16);
        }
    }
}

template <int DT>
__device__ __forceinline__ void load8(const void* base, int64_t at, int n, float (&x)[8])
{
    unpack8<DT>(load_raw8<DT>(base, at, n), x);
}

template <int DT>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, const float (&x)[8])
{
    if constexpr (DT == HPO_PARAM_FP32) {
        float* p = static_cast<float*>(base) + at;
        if (n >= 8) {
            *reinterpret_cast<f32x4_any*>(p) = f32x4_t{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<f32x4_any*>(p + 4) = f32x4_t{x[4], x[5], x[6], x[7]};
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n)
                    p[e] = x[e];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(base) + at;
        if (n >= 8) {
            u32x4_t t;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                t[e] = narrow<DT>(x[2 * e]) | (narrow<DT>(x[2 * e + 1]) << 16);
            *reinterpret_cast<u32x4_any2*>(p) = t;
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n)
                    p[e] = static_cast<uint16_t>(narrow<DT>(x[e]));
        }
    }
}

/* HPO_WEIGHT_MX8's scale byte of a block whose largest magnitude has the bits `m` (inf and NaN come
 * out above the finite values): floor(log2) of a normal value is its exponent field - 127; the byte is
 * that field - 8, 0 from 2^-118 down, 255 for a block that is not finite. */
__device__ __forceinline__ uint32_t mx8_byte(uint32_t m)
{
    const uint32_t field = m >> 23;
    return m >= 0x7f800000u ? 255u : (field > 8u ? field - 8u : 0u);
}

/* Four values at such a scale: multiplying by 2^-e is exact or below e4m3's smallest half step, the
 * conversion rounds to nearest even. */
__device__ __forceinline__ uint32_t mx8_pack(float a, float b, float c, float d, uint32_t byte)
{
    if (byte == 255u)
        return 0x7f7f7f7fu;
    const float inv = __uint_as_float((254u - byte) << 23);
    const float lim = 448.0f;
    int t = __builtin_amdgcn_cvt_pk_fp8_f32(fminf(fmaxf(a * inv, -lim), lim), fminf(fmaxf(b * inv, -lim), lim), 0, false);
    t = __builtin_amdgcn_cvt_pk_fp8_f32(fminf(fmaxf(c * inv, -lim), lim), fminf(fmaxf(d * inv, -lim), lim), t, true);
    return static_cast<uint32_t>(t);
}

template <typename... Args>
hipError_t launch(void (*kernel)(Args...), dim3 grid, int block, hipStream_t stream, Args... args)
{
    void* argv[] = {static_cast<void*>(&args)...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(block), argv, 0, stream);
}

}  // namespace
}  // namespace hpo

#endif /* HPO_MODEL_DEVICE_H */
