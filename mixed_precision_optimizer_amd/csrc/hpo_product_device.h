/*
 * hpo_product_device.h -- device code shared by the 8-bit products' kernel
 * files (hpo_mx8.hip: Y = X^ W^T; hpo_mx8_grad.hip: dX = dY W^, G += scale * dY^T X^):
 * tiles, the order of the work, staging in LDS, and what becomes of the sums.
 * Not part of the public ABI.
 */
#ifndef HPO_PRODUCT_DEVICE_H
#define HPO_PRODUCT_DEVICE_H

#include <type_traits>

#include "hpo_model_device.h"

namespace hpo {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

/* ---------------------------------------------------------------------- */
/* products: tiles                                                         */
/* ---------------------------------------------------------------------- */
/* A workgroup of WM x WN wavefronts computes BM x BN of C, each wavefront TM x TN blocks of 32 x 32. */
template <int WM_, int WN_, int TM_, int TN_>
struct Tile {
    static constexpr int WM = WM_, WN = WN_, TM = TM_, TN = TN_;
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int BM = WM * TM * 32, BN = WN * TN * 32;
};
using Tile256 = Tile<2, 4, 4, 2>;   /* of the gradients; hpo_mx8_linear's is Big */
using Tile128 = Tile<2, 2, 2, 2>;
using Tile64 = Tile<2, 2, 1, 1>;

constexpr int kRowBytes = 128;   /* of an operand row in a stage: 128 8-bit elements, or 64 16-bit ones */
constexpr int kStepK = 64;        /* 16-bit elements of k in a stage */
/* Tile rows that neighbouring workgroups share: 32 CUs of an XCD take 4 x 8 tiles of 256, and a gradient's row of A is
 * twice as many bytes as its column of B (2, 4, 8, 16: G of 14336 x 4096 over 8192 tokens 896, 908, 925, 936 us, Y of
 * 8192 x 14336 407, 400, 403, 414). */
constexpr uint32_t kGroup = 4;

/* Workgroups go to the 8 XCDs round-robin: each XCD gets one contiguous run of the work. */
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t n)
{
    constexpr uint32_t kXcd = 8;
    const uint32_t x = b % kXcd, k = b / kXcd, q = n / kXcd, r = n % kXcd;
    return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + k;
}

struct Work {
    int64_t z;
    int tm, tn, split;
};

/* Item b of n (at most INT32_MAX): the b-th workgroup's, or what a workgroup in its place takes. */
__device__ __forceinline__ Work work_of(const ProductArgs& p, uint32_t b, uint32_t n)
{
    Work w;
    uint32_t t = xcd_run(b, n);
    const uint32_t tiles_n = p.tiles_n, per = p.tiles_m * tiles_n, part = t / per;
    w.z = part / p.splits;
    w.split = static_cast<int>(part % p.splits);
    const uint32_t i = t % per, first = i / (kGroup * tiles_n) * kGroup, left = p.tiles_m - first;
    const uint32_t rows = left < kGroup ? left : kGroup, j = i - first * tiles_n;
    w.tm = static_cast<int>(first + j % rows);
    w.tn = static_cast<int>(j / rows);
    return w;
}

/* The same in every lane: kept in scalar registers. */
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p)
{
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
    return reinterpret_cast<const uint8_t*>(lo | static_cast<uint64_t>(hi) << 32);
}

/* 64 x 16 bytes from a buffer straight into LDS: lane l's lands at dst + 16 l; what lies behind the
 * descriptor's end comes as 0. */
__device__ __forceinline__ void buffer_load_lds16(__amdgpu_buffer_rsrc_t rs, char* dst, int voff, int soff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}

constexpr int kNowhere = 0x7ffffff0;   /* an offset behind every descriptor's end */

/* Byte offset of 16-byte piece p of a 128-byte LDS row: the pieces are permuted by the row, so that the
 * 16 rows a fragment read serves at a time lie in distinct banks. */
__device__ __forceinline__ int row_swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }
__device__ __forceinline__ int piece_at(int r, int p) { return r * kRowBytes + ((p ^ row_swizzle(r)) << 4); }

/* The same for slices of 64 bytes a row. */
constexpr int kSliceBytes = 64;
__device__ __forceinline__ int slice_swizzle(int r) { return (r >> 2) & 3; }
__device__ __forceinline__ int slice_at(int r, int p) { return r * kSliceBytes + ((p ^ slice_swizzle(r)) << 4); }

/* Rows that run along C's side (W elements of 16 bits, one row per k): their 32-byte pairs of pieces are
 * permuted by the row, so that the four rows (twice) a transposing read takes 32 bytes each of lie in
 * distinct banks. */
template <int W>
__device__ __forceinline__ int pair_swizzle(int k)
{
    if constexpr (W >= 128)
        return ((k & 3) << 1) ^ ((k >> 3) & 1);
    else
        return (k & 2) ^ ((k >> 3) & 1);
}

/* v without its first `bits` bits (whole bytes, less than 16 of them); 0 comes in behind. */
__device__ __forceinline__ u32x4_t drop_bytes(u32x4_t v, int bits)
{
    if (bits == 0)
        return v;
    uint64_t lo = v[0] | (static_cast<uint64_t>(v[1]) << 32), hi = v[2] | (static_cast<uint64_t>(v[3]) << 32);
    lo = bits < 64 ? (lo >> bits) | (hi << (64 - bits)) : hi >> (bits - 64);
    hi = bits < 64 ? hi >> bits : 0;
    return u32x4_t{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                   static_cast<uint32_t>(hi >> 32)};
}

/* 16 bytes of a row from `at` on, `left` of them (<= 0: none) inside it; 0 behind.  `before` bytes of the row lie before
 * `at`: a row's end is read as the 16 bytes that end there, in one load. */
__device__ __forceinline__ u32x4_t load16(const uint8_t* at, int64_t left, int64_t before)
{
    u32x4_t v = {0, 0, 0, 0};
    if (left > 0 && (left >= 16 || before + left >= 16)) {
        const int back = left < 16 ? 16 - static_cast<int>(left) : 0;
        return drop_bytes(*reinterpret_cast<const u32x4_any*>(at - back), 8 * back);
    }
    for (int e = 0; e < left; ++e)
        v[e >> 2] |= static_cast<uint32_t>(at[e]) << (8 * (e & 3));
    return v;
}

/* s_waitcnt's operand (gfx9 encoding): at most `loads` in flight, no LDS access. */
constexpr int waitcnt(int loads) { return (loads & 15) | 0x70 | (loads >> 4) << 14; }

/* Waits for this wavefront's loads and LDS accesses, then for the workgroup.  Nothing else makes
 * loads into LDS land before the barrier. */
__device__ __forceinline__ void land()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(waitcnt(0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

template <int DT>
__device__ __forceinline__ void store4(void* c, int64_t at, int n, f32x4_t x)
{
    if constexpr (DT == HPO_PARAM_FP32) {
        float* p = static_cast<float*>(c) + at;
        if (n >= 4) {
            *reinterpret_cast<f32x4_any*>(p) = x;
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < n)
                    p[e] = x[e];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(c) + at;
        if (n >= 4) {
            *reinterpret_cast<u32x2_any2*>(p) = u32x2_t{pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3])};
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < n)
                    p[e] = static_cast<uint16_t>(narrow<DT>(x[e]));
        }
    }
}

template <int DT>
__device__ __forceinline__ f32x4_t load4(const void* c, int64_t at, int n)
{
    f32x4_t x = {0, 0, 0, 0};
    if constexpr (DT == HPO_PARAM_FP32) {
        const float* p = static_cast<const float*>(c) + at;
        if (n >= 4)
            return *reinterpret_cast<const f32x4_any*>(p);
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n)
                x[e] = p[e];
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(c) + at;
        if (n >= 4) {
            const u32x2_t t = *reinterpret_cast<const u32x2_any2*>(p);
            return f32x4_t{widen<DT>(t.x), widen<DT>(t.x >> 16), widen<DT>(t.y), widen<DT>(t.y >> 16)};
        }
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n)
                x[e] = widen<DT>(p[e]);
    }
    return x;
}

/* What becomes of the sums, wavefront by wavefront through LDS (`lds`: the stages', done with), so that
 * whole rows of the wavefront's block leave in runs of 128 bytes and more: straight from the
 * registers, every store would touch 32 rows for 16 bytes each.
 * acc[i][j][r] of a lane: row 32 i + lane % 32, column 32 j + 8 (r / 4) + 4 (lane / 32) + r % 4. */
template <typename T, int DT, bool ADD>
__device__ __forceinline__ void write_block(char* mine, void* c, int64_t at, int64_t rs, int64_t rows, int64_t cols, float scale,
                                            const f32x16_t (&acc)[T::TM][T::TN])
{
    constexpr int P = T::TN * 8;          /* 16-byte pieces of a row */
    constexpr int kTurns = 32 * P / 64;   /* pieces of a lane in a block of 32 rows */
    const int lane = threadIdx.x & 63, frow = lane & 31, fh = lane >> 5;
    const int pc = lane % P, r0 = lane / P;
    const int n = cols - 4 * pc > 4 ? 4 : static_cast<int>(cols - 4 * pc);
#pragma unroll
    for (int i = 0; i < T::TM; ++i) {
        f32x4_t before[ADD ? kTurns : 1];
        if constexpr (ADD) {
#pragma unroll
            for (int t = 0; t < kTurns; ++t) {
                const int r = 32 * i + t * (64 / P) + r0;
                before[t] = load4<DT>(c, at + r * rs + 4 * pc, r < rows ? n : 0);
            }
        }
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4_t*>(mine + frow * (P * 16) + (((8 * j + 2 * g + fh) ^ (frow & (P - 1))) << 4)) =
                    f32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int t = 0; t < kTurns; ++t) {
            const int q = t * (64 / P) + r0, r = 32 * i + q;
            f32x4_t x = *reinterpret_cast<const f32x4_t*>(mine + q * (P * 16) + ((pc ^ (q & (P - 1))) << 4));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = x[e] * scale;
                if constexpr (ADD)
                    x[e] = before[t][e] + x[e];
            }
            if (r < rows)
                store4<DT>(c, at + r * rs + 4 * pc, n, x);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <typename T, bool GRAD>
__device__ __forceinline__ void epilogue(const ProductArgs& p, const Work& w, char* lds, const f32x16_t (&acc)[T::TM][T::TN])
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m0 = static_cast<int64_t>(w.tm) * T::BM + wave / T::WN * (T::TM * 32);
    const int64_t n0 = static_cast<int64_t>(w.tn) * T::BN + wave % T::WN * (T::TN * 32);
    const int64_t rows = p.m - m0, cols = p.n - n0;
    char* mine = lds + wave * (32 * T::TN * 128);
    __syncthreads();
    if (rows <= 0 || cols <= 0)
        return;
    if (p.splits > 1) {
        write_block<T, HPO_PARAM_FP32, false>(mine, p.part, ((w.z * p.splits + w.split) * p.m + m0) * p.n + n0, p.n, rows, cols,
                                              1.0f, acc);
        return;
    }
    const int64_t at = w.z * p.c_bs + m0 * p.c_rs + n0;
    auto put = [&](auto dt, auto add) {
        write_block<T, decltype(dt)::value, decltype(add)::value>(mine, p.c, at, p.c_rs, rows, cols, p.scale, acc);
    };
    using bf16 = std::integral_constant<int, HPO_PARAM_BF16>;
    using fp16 = std::integral_constant<int, HPO_PARAM_FP16>;
    using fp32 = std::integral_constant<int, HPO_PARAM_FP32>;
    if constexpr (GRAD) {   /* a main grad: fp32 or bf16 */
        if (p.c_dtype == HPO_PARAM_FP32)
            p.accumulate ? put(fp32{}, std::true_type{}) : put(fp32{}, std::false_type{});
        else
            p.accumulate ? put(bf16{}, std::true_type{}) : put(bf16{}, std::false_type{});
    } else {
        if (p.c_dtype == HPO_PARAM_BF16)
            put(bf16{}, std::false_type{});
        else if (p.c_dtype == HPO_PARAM_FP16)
            put(fp16{}, std::false_type{});
        else
            put(fp32{}, std::false_type{});
    }
}

}  // namespace
}  // namespace hpo

#endif /* HPO_PRODUCT_DEVICE_H */
