/*
 * hpo_mx8.hip -- gfx950 kernels of activations and weights in 8 bits with block
 * scales: the quantisation (hpo_mx8_save) and the products of a linear layer,
 * Y = X^ W^T, dX = dY W^, G += scale * dY^T X^ (hpo_mx8_linear, _dgrad, _wgrad).
 */
#include <hip/hip_runtime.h>

#include <algorithm>
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
/* hpo_mx8_save                                                            */
/* ---------------------------------------------------------------------- */
constexpr int kSaveThreads = 256;

/* LANES lanes take a row, eight elements each a step; four neighbours hold a scale block. */
template <int XT, int LANES>
__global__ __launch_bounds__(kSaveThreads) void k_mx8_save(SaveArgs a)
{
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (kSaveThreads / LANES) + threadIdx.x / LANES, z = blockIdx.y;
    if (i >= a.rows)
        return;
    const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock, src = z * a.x.bs + i * a.x.rs;
    uint8_t* q = static_cast<uint8_t*>(a.q.data) + z * a.q.bs + i * a.q.rs;
    uint8_t* sc = a.scales + (z * a.rows + i) * nb;
#pragma unroll 2
    for (int64_t c0 = 0; c0 < a.cols; c0 += 8 * LANES) {   /* all lanes of a block take part to the end */
        const int64_t c = c0 + 8 * (threadIdx.x % LANES);
        const int n = a.cols - c > 8 ? 8 : static_cast<int>(a.cols - c);
        float x[8];
        load8<XT>(a.x.data, src + c, n, x);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t u = __float_as_uint(x[e]) & 0x7fffffffu;
            m = u > m ? u : m;
        }
#pragma unroll
        for (int d = 1; d < kMxBlock / 8; d <<= 1) {
            const uint32_t o = __shfl_xor(m, d, 64);
            m = o > m ? o : m;
        }
        const uint32_t byte = mx8_byte(m);
        const uint32_t lo = mx8_pack(x[0], x[1], x[2], x[3], byte), hi = mx8_pack(x[4], x[5], x[6], x[7], byte);
        if (n >= 8) {
            *reinterpret_cast<u32x2_any*>(q + c) = u32x2_t{lo, hi};
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n)
                    q[c + e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
        }
        if (n > 0 && (threadIdx.x & 3) == 0)
            sc[c / kMxBlock] = static_cast<uint8_t>(byte);
    }
}

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
using Tile256 = Tile<2, 4, 4, 2>;
using Tile128 = Tile<2, 2, 2, 2>;
using Tile64 = Tile<2, 2, 1, 1>;

constexpr int kRowBytes = 128;   /* of an operand row in a stage: 128 8-bit elements, or 64 16-bit ones */
constexpr int kGroup = 8;        /* tile rows that neighbouring workgroups share */

/* Workgroups go to the 8 XCDs round-robin: each XCD gets one contiguous run of the work. */
__device__ __forceinline__ int64_t xcd_run(int64_t b, int64_t n)
{
    constexpr int64_t kXcd = 8;
    const int64_t x = b % kXcd, k = b / kXcd, q = n / kXcd, r = n % kXcd;
    return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + k;
}

struct Work {
    int64_t z;
    int tm, tn, split;
};

__device__ __forceinline__ Work work_of(const ProductArgs& p)
{
    Work w;
    int64_t t = xcd_run(blockIdx.x, gridDim.x);
    w.split = static_cast<int>(t % p.splits);
    t /= p.splits;
    const int64_t per = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
    w.z = t / per;
    const int i = static_cast<int>(t % per), g = i / (kGroup * p.tiles_n), first = g * kGroup;
    const int rows = p.tiles_m - first < kGroup ? p.tiles_m - first : kGroup, j = i - first * p.tiles_n;
    w.tm = first + j % rows;
    w.tn = j / rows;
    return w;
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

/* 16 bytes of a row from `at` on, `left` of them (<= 0: none) inside it; 0 behind. */
__device__ __forceinline__ u32x4_t load16(const uint8_t* at, int64_t left)
{
    u32x4_t v = {0, 0, 0, 0};
    if (left >= 16)
        return *reinterpret_cast<const u32x4_any*>(at);
    for (int e = 0; e < left; ++e)
        v[e >> 2] |= static_cast<uint32_t>(at[e]) << (8 * (e & 3));
    return v;
}

/* Waits for this wavefront's loads and LDS accesses, then for the workgroup.  Nothing else makes
 * loads into LDS land before the barrier. */
__device__ __forceinline__ void land()
{
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0x0070);   /* gfx9 encoding: vmcnt(0) lgkmcnt(0) */
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
            *reinterpret_cast<u32x2_any2*>(p) = u32x2_t{narrow<DT>(x[0]) | (narrow<DT>(x[1]) << 16),
                                                        narrow<DT>(x[2]) | (narrow<DT>(x[3]) << 16)};
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

/* Four neighbouring sums of row m become results. */
template <int DT>
__device__ __forceinline__ void finish4(const ProductArgs& p, int64_t z, int64_t m, int64_t n, f32x4_t x)
{
    const int64_t at = z * p.c_bs + m * p.c_rs + n;
    const int left = p.n - n > 4 ? 4 : static_cast<int>(p.n - n);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        x[e] = x[e] * p.scale;
    if (p.accumulate) {
        const f32x4_t g = load4<DT>(p.c, at, left);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = g[e] + x[e];
    }
    store4<DT>(p.c, at, left, x);
}

/* acc[i][j][r] of a lane: row 32 i + lane % 32, column 32 j + 8 (r / 4) + 4 (lane / 32) + r % 4. */
template <typename T>
__device__ __forceinline__ void epilogue(const ProductArgs& p, const Work& w, const f32x16_t (&acc)[T::TM][T::TN])
{
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t m0 = static_cast<int64_t>(w.tm) * T::BM + wave / T::WN * (T::TM * 32) + (lane & 31);
    const int64_t n0 = static_cast<int64_t>(w.tn) * T::BN + wave % T::WN * (T::TN * 32) + 4 * (lane >> 5);
    auto each = [&](auto&& put) {
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int64_t m = m0 + 32 * i, n = n0 + 32 * j + 8 * g;
                    if (m < p.m && n < p.n)
                        put(m, n, f32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]});
                }
    };
    if (p.splits > 1) {
        float* part = p.part + (w.z * p.splits + w.split) * p.m * p.n;
        each([&](int64_t m, int64_t n, f32x4_t x) {
            store4<HPO_PARAM_FP32>(part, m * p.n + n, p.n - n > 4 ? 4 : static_cast<int>(p.n - n), x);
        });
    } else if (p.c_dtype == HPO_PARAM_FP32) {
        each([&](int64_t m, int64_t n, f32x4_t x) { finish4<HPO_PARAM_FP32>(p, w.z, m, n, x); });
    } else if (p.c_dtype == HPO_PARAM_BF16) {
        each([&](int64_t m, int64_t n, f32x4_t x) { finish4<HPO_PARAM_BF16>(p, w.z, m, n, x); });
    } else {
        each([&](int64_t m, int64_t n, f32x4_t x) { finish4<HPO_PARAM_FP16>(p, w.z, m, n, x); });
    }
}

/* Adds the splits' sums, in order.  Grid: (pieces of a row's 1024 columns, rows in turn, batch in turn). */
constexpr int kJoinThreads = 256;
template <int DT>
__global__ __launch_bounds__(kJoinThreads) void k_product_join(ProductArgs p)
{
    const int64_t quads = (p.n + 3) / 4, all = p.batch * p.m * quads;
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kJoinThreads + threadIdx.x; t < all;
         t += static_cast<int64_t>(gridDim.x) * kJoinThreads) {
        const int64_t n = t % quads * 4, row = t / quads, z = row / p.m, m = row % p.m;
        const int left = p.n - n > 4 ? 4 : static_cast<int>(p.n - n);
        const float* part = p.part + z * p.splits * p.m * p.n;
        f32x4_t x = {0, 0, 0, 0};
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            const f32x4_t y = load4<HPO_PARAM_FP32>(part, (s * p.m + m) * p.n + n, left);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] += y[e];
        }
        finish4<DT>(p, z, m, n, x);
    }
}

/* ---------------------------------------------------------------------- */
/* Y = X^ W^T                                                              */
/* ---------------------------------------------------------------------- */
/* The matrix cores take blocks of 32 x 32 x 64 with a scale for each row and 32 elements of k.  Lane
 * (r, h) = (lane % 32, lane / 32) holds of row r bytes 16 h .. 16 h + 15 of the first block of 32 and
 * of the second, and the scale of block h. */
template <typename T, bool DIRECT>
__global__ __launch_bounds__(T::kThreads) void k_mx8_linear(ProductArgs p)
{
    constexpr int kRows = T::BM + T::BN;
    constexpr int kStage = kRows * kRowBytes;
    constexpr int kScales = 2 * kStage;              /* behind the stages: 16 scale bytes a row, twice */
    constexpr int kScaleStage = kRows * 16;
    constexpr int kChunks = kRows / 8 / T::kWaves;   /* 1 KB loads of a wavefront per stage */
    constexpr int kPieces = kRows * 8 / T::kThreads;
    constexpr int kScaleRows = (kRows + T::kThreads - 1) / T::kThreads;
    __shared__ __attribute__((aligned(16))) char lds[2 * kStage + 2 * kScaleStage];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int frow = lane & 31, fh = lane >> 5;
    const Work w = work_of(p);
    const int64_t m0 = static_cast<int64_t>(w.tm) * T::BM, n0 = static_cast<int64_t>(w.tn) * T::BN;
    const int rows_m = p.m - m0 < T::BM ? static_cast<int>(p.m - m0) : T::BM;
    const int rows_n = p.n - n0 < T::BN ? static_cast<int>(p.n - n0) : T::BN;
    const uint8_t* A = static_cast<const uint8_t*>(p.a) + w.z * p.a_bs + m0 * p.a_rs;
    const uint8_t* B = p.b + w.z * p.b_bs + n0 * p.b_rs;
    const int64_t nb = (p.k + kMxBlock - 1) / kMxBlock;
    const uint8_t* SA = p.a_scales + (w.z * p.m + m0) * nb;
    const uint8_t* SB = p.b_scales + (w.z * p.n + n0) * nb;
    const int steps = static_cast<int>((p.k + kRowBytes - 1) / kRowBytes);
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * w.split / p.splits);
    const int k1 = static_cast<int>(static_cast<int64_t>(steps) * (w.split + 1) / p.splits);

    /* tile row -> source row; rows behind C's sides hold copies of the last and their sums are not kept */
    auto clamp = [&](int r) { return r < T::BM ? (r < rows_m ? r : rows_m - 1) : (r - T::BM < rows_n ? r - T::BM : rows_n - 1); };

    __amdgpu_buffer_rsrc_t rsA, rsB;
    int voff[DIRECT ? kChunks : 1], piece[DIRECT ? kChunks : 1];
    u32x4_t held[DIRECT ? 1 : kPieces];
    if constexpr (DIRECT) {
        rsA = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(A), 0,
                                                static_cast<int>((rows_m - 1) * p.a_rs + p.k), 0x00020000);
        rsB = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(B), 0,
                                                static_cast<int>((rows_n - 1) * p.b_rs + p.k), 0x00020000);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int r = (wave * kChunks + c) * 8 + (lane >> 3);
            piece[c] = (lane & 7) ^ row_swizzle(r);
            voff[c] = clamp(r) * static_cast<int>(r < T::BM ? p.a_rs : p.b_rs) + piece[c] * 16;
        }
    }
    auto fetch = [&](int kt, int buf) {
        const int64_t left = p.k - static_cast<int64_t>(kt) * kRowBytes;   /* bytes of the row from here */
        if constexpr (DIRECT) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int idx = wave * kChunks + c;
                const int v = left >= kRowBytes || piece[c] * 16 < left ? voff[c] : kNowhere;
                buffer_load_lds16(idx < T::BM / 8 ? rsA : rsB, lds + buf * kStage + idx * 1024, v, kt * kRowBytes);
            }
        } else {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int i = c * T::kThreads + tid, r = i >> 3, at = (i & 7) * 16;
                const uint8_t* row = r < T::BM ? A + clamp(r) * p.a_rs : B + clamp(r) * p.b_rs;
                held[c] = load16(row + static_cast<int64_t>(kt) * kRowBytes + at, left - at);
            }
        }
    };
    auto put = [&](int buf) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int i = c * T::kThreads + tid;
                *reinterpret_cast<u32x4_t*>(lds + buf * kStage + piece_at(i >> 3, i & 7)) = held[c];
            }
        }
    };
    /* Scales of four steps at a time; a byte behind the row's end reads as 0, never as a neighbour's NaN. */
    u32x4_t sheld[kScaleRows];
    auto fetch_scales = [&](int kt) {
#pragma unroll
        for (int c = 0; c < kScaleRows; ++c) {
            const int r = c * T::kThreads + tid;
            if (r < kRows)
                sheld[c] = load16((r < T::BM ? SA : SB) + clamp(r) * nb + 4 * kt, nb - 4 * static_cast<int64_t>(kt));
        }
    };
    auto put_scales = [&](int buf) {
#pragma unroll
        for (int c = 0; c < kScaleRows; ++c) {
            const int r = c * T::kThreads + tid;
            if (r < kRows)
                *reinterpret_cast<u32x4_t*>(lds + kScales + buf * kScaleStage + r * 16) = sheld[c];
        }
    };

    f32x16_t acc[T::TM][T::TN];
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            acc[i][j] = f32x16_t{};
    const int am = wave / T::WN * (T::TM * 32) + frow, bn = T::BM + wave % T::WN * (T::TN * 32) + frow;

    auto compute = [&](int buf, int sbuf, int word) {
        const char* src = lds + buf * kStage;
        const char* scl = lds + kScales + sbuf * kScaleStage + word * 4;
        int sa[T::TM], sb[T::TN];
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
            sa[i] = static_cast<int>(*reinterpret_cast<const uint32_t*>(scl + (am + 32 * i) * 16) >> (8 * fh));
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            sb[j] = static_cast<int>(*reinterpret_cast<const uint32_t*>(scl + (bn + 32 * j) * 16) >> (8 * fh));
        auto frag = [&](int r, int s) {
            const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(src + piece_at(r, 4 * s + fh));
            const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(src + piece_at(r, 4 * s + 2 + fh));
            return i32x8_t{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]),
                           static_cast<int>(hi[0]), static_cast<int>(hi[1]), static_cast<int>(hi[2]), static_cast<int>(hi[3])};
        };
        auto slice = [&](auto S) {
            i32x8_t fa[T::TM], fb[T::TN];
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
                fb[j] = frag(bn + 32 * j, S.value);
#pragma unroll
            for (int i = 0; i < T::TM; ++i)
                fa[i] = frag(am + 32 * i, S.value);
#pragma unroll
            for (int i = 0; i < T::TM; ++i)
#pragma unroll
                for (int j = 0; j < T::TN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], 0, 0, 2 * S.value,
                                                                                sb[j], 2 * S.value, sa[i]);
        };
        slice(std::integral_constant<int, 0>{});
        slice(std::integral_constant<int, 1>{});
    };

    if (k0 < k1) {
        fetch_scales(k0);
        fetch(k0, 0);
        put_scales(0);
        put(0);
        for (int kt = k0; kt < k1; ++kt) {
            const int at = kt - k0, buf = at & 1, sbuf = (at >> 2) & 1;
            land();
            if (kt + 1 < k1)
                fetch(kt + 1, buf ^ 1);
            if ((at & 3) == 0 && kt + 4 < k1)
                fetch_scales(kt + 4);
            __builtin_amdgcn_sched_barrier(0);
            compute(buf, sbuf, at & 3);
            if (kt + 1 < k1)
                put(buf ^ 1);
            if ((at & 3) == 3 && kt + 1 < k1)
                put_scales(sbuf ^ 1);
        }
    }
    epilogue<T>(p, w, acc);
}

/* ---------------------------------------------------------------------- */
/* dX = dY W^ and G += scale * dY^T X^                                     */
/* ---------------------------------------------------------------------- */
/* Eight bits become 16 exactly (bf16), or rounded (fp16): two neighbours at a time, at 2^(byte - 127). */
template <bool FP16, bool HIGH>
__device__ __forceinline__ uint32_t widen_pair(uint32_t v, float scale)
{
    if constexpr (FP16) {
        const f16x2_t r = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, scale, HIGH);
        return __builtin_bit_cast(uint32_t, r);
    } else {
        const bf16x2_t r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, HIGH);
        return __builtin_bit_cast(uint32_t, r);
    }
}

template <bool FP16>
__device__ __forceinline__ f32x16_t mfma16(u32x4_t a, u32x4_t b, f32x16_t c)
{
    if constexpr (FP16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

/* Eight k of 32 neighbouring columns from rows along C's side: lane (r, h) gets k = 8 h .. 8 h + 7 of column
 * r.  A transposing read gives each of 16 lanes four rows of one column; `at` is this lane's source. */
template <int W>
__device__ __forceinline__ u32x4_t transposed(const char* at)
{
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
    const u32x2_t lo = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at)));
    const u32x2_t hi = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * W * 2)));
    return u32x4_t{lo.x, lo.y, hi.x, hi.y};
}

constexpr int kStepK = 64;

template <typename T, bool WGRAD, bool FP16, bool DIRECT>
__global__ __launch_bounds__(T::kThreads) void k_mx8_grad(ProductArgs p)
{
    constexpr int kA = T::BM * kRowBytes, kB = T::BN * kRowBytes, kStage = kA + kB;
    constexpr int kChunks = T::BM / 8 / T::kWaves;                  /* 1 KB loads of a wavefront per stage of A */
    constexpr int kPieces = T::BM * 8 / T::kThreads;                /* 16-byte pieces of a lane */
    constexpr int kCols16 = T::BN / 16, kBPieces = kStepK * kCols16 / T::kThreads;
    static_assert(kChunks >= 1 && kBPieces >= 1, "every wavefront stages");
    __shared__ __attribute__((aligned(16))) char lds[2 * kStage];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int frow = lane & 31, fh = lane >> 5;
    const Work w = work_of(p);
    const int64_t m0 = static_cast<int64_t>(w.tm) * T::BM, n0 = static_cast<int64_t>(w.tn) * T::BN;
    const int rows_m = p.m - m0 < T::BM ? static_cast<int>(p.m - m0) : T::BM;
    const int rows_n = p.n - n0 < T::BN ? static_cast<int>(p.n - n0) : T::BN;
    const uint16_t* A = static_cast<const uint16_t*>(p.a) + w.z * p.a_bs + (WGRAD ? m0 : m0 * p.a_rs);
    const uint8_t* B = p.b + w.z * p.b_bs + n0;
    const int64_t nb = (p.n + kMxBlock - 1) / kMxBlock;
    const uint8_t* SB = p.b_scales + w.z * p.k * nb;
    const int steps = static_cast<int>((p.k + kStepK - 1) / kStepK);
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * w.split / p.splits);
    const int k1 = static_cast<int>(static_cast<int64_t>(steps) * (w.split + 1) / p.splits);

    __amdgpu_buffer_rsrc_t rsA;
    int voff[DIRECT ? kChunks : 1], piece[DIRECT ? kChunks : 1];
    u32x4_t held[DIRECT ? 1 : kPieces];
    if constexpr (DIRECT) {
        if constexpr (!WGRAD)
            rsA = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(A), 0,
                                                    static_cast<int>(((rows_m - 1) * p.a_rs + p.k) * 2), 0x00020000);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            const int idx = wave * kChunks + c;
            if constexpr (WGRAD) {
                constexpr int kSlots = T::BM / 8;
                const int r = idx * (64 / kSlots) + lane / kSlots, s = lane % kSlots;
                piece[c] = (((s >> 1) ^ pair_swizzle<T::BM>(r)) << 1) | (s & 1);
                voff[c] = (r * static_cast<int>(p.a_rs) + piece[c] * 8) * 2;
            } else {
                const int r = idx * 8 + (lane >> 3);
                piece[c] = (lane & 7) ^ row_swizzle(r);
                voff[c] = ((r < rows_m ? r : rows_m - 1) * static_cast<int>(p.a_rs) + piece[c] * 8) * 2;
            }
        }
    }
    auto fetch_a = [&](int kt, int buf) {
        const int64_t k = static_cast<int64_t>(kt) * kStepK, left = p.k - k;
        if constexpr (DIRECT && WGRAD) {
            /* rows behind the last token lie behind the descriptor's end, and columns behind C's side are
             * copies of what follows them; their sums are not kept.  The end is that of an aligned word:
             * a word that is only partly inside would read as 0. */
            const int rows = left < kStepK ? static_cast<int>(left) : kStepK;
            const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                const_cast<uint16_t*>(A + k * p.a_rs), 0, static_cast<int>((((rows - 1) * p.a_rs + rows_m) * 2 + 3) & ~3),
                0x00020000);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                buffer_load_lds16(rs, lds + buf * kStage + (wave * kChunks + c) * 1024, voff[c], 0);
        } else if constexpr (DIRECT) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int v = left >= kStepK || piece[c] * 8 < left ? voff[c] : kNowhere;
                buffer_load_lds16(rsA, lds + buf * kStage + (wave * kChunks + c) * 1024, v, kt * kRowBytes);
            }
        } else {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int i = c * T::kThreads + tid;
                if constexpr (WGRAD) {
                    const int r = i / (T::BM / 8), at = i % (T::BM / 8) * 8;
                    held[c] = load16(reinterpret_cast<const uint8_t*>(A + (k + r) * p.a_rs + at), r < left ? 2 * (rows_m - at) : 0);
                } else {
                    const int r = i >> 3, at = (i & 7) * 8;
                    held[c] = load16(reinterpret_cast<const uint8_t*>(A + (r < rows_m ? r : rows_m - 1) * p.a_rs + k + at),
                                     2 * (left - at));
                }
            }
        }
    };
    auto put_a = [&](int buf) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int i = c * T::kThreads + tid;
                int at;
                if constexpr (WGRAD) {
                    const int r = i / (T::BM / 8), s = i % (T::BM / 8);
                    at = r * (T::BM * 2) + ((((s >> 1) ^ pair_swizzle<T::BM>(r)) << 1) | (s & 1)) * 16;
                } else {
                    at = piece_at(i >> 3, i & 7);
                }
                *reinterpret_cast<u32x4_t*>(lds + buf * kStage + at) = held[c];
            }
        }
    };
    u32x4_t bheld[kBPieces];
    uint32_t bscale[kBPieces];
    auto fetch_b = [&](int kt) {
#pragma unroll
        for (int c = 0; c < kBPieces; ++c) {
            const int i = c * T::kThreads + tid, r = i / kCols16, at = i % kCols16 * 16;
            const int64_t k = static_cast<int64_t>(kt) * kStepK + r;
            const bool in = k < p.k && at < rows_n;
            bheld[c] = load16(B + k * p.b_rs + at, in ? rows_n - at : 0);
            bscale[c] = in ? SB[k * nb + (n0 + at) / kMxBlock] : 127u;
        }
    };
    auto put_b = [&](int buf) {
#pragma unroll
        for (int c = 0; c < kBPieces; ++c) {
            const int i = c * T::kThreads + tid, r = i / kCols16, pair = i % kCols16;
            const float s = __uint_as_float(bscale[c] << 23);
            char* dst = lds + buf * kStage + kA + r * (T::BN * 2) + (pair ^ pair_swizzle<T::BN>(r)) * 32;
            u32x4_t lo, hi;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                lo[2 * e] = widen_pair<FP16, false>(bheld[c][e], s);
                lo[2 * e + 1] = widen_pair<FP16, true>(bheld[c][e], s);
                hi[2 * e] = widen_pair<FP16, false>(bheld[c][2 + e], s);
                hi[2 * e + 1] = widen_pair<FP16, true>(bheld[c][2 + e], s);
            }
            *reinterpret_cast<u32x4_t*>(dst) = lo;
            *reinterpret_cast<u32x4_t*>(dst + 16) = hi;
        }
    };

    f32x16_t acc[T::TM][T::TN];
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            acc[i][j] = f32x16_t{};
    const int am = wave / T::WN * (T::TM * 32), bn = wave % T::WN * (T::TN * 32);
    /* this lane's place in a transposing read: row 8 h + q of a slice, pair g, 8 bytes c */
    const int tq = (lane & 15) >> 2, tg = (lane >> 4) & 1, tc = lane & 3, tk = 8 * fh + tq;

    auto compute = [&](int buf) {
        const char* src = lds + buf * kStage;
#pragma unroll
        for (int s = 0; s < kStepK / 16; ++s) {
            u32x4_t fa[T::TM], fb[T::TN];
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
                fb[j] = transposed<T::BN>(src + kA + (16 * s + tk) * (T::BN * 2) +
                                          (((bn + 32 * j) / 16 + tg) ^ pair_swizzle<T::BN>(tk)) * 32 + tc * 8);
#pragma unroll
            for (int i = 0; i < T::TM; ++i) {
                if constexpr (WGRAD)
                    fa[i] = transposed<T::BM>(src + (16 * s + tk) * (T::BM * 2) +
                                              (((am + 32 * i) / 16 + tg) ^ pair_swizzle<T::BM>(tk)) * 32 + tc * 8);
                else
                    fa[i] = *reinterpret_cast<const u32x4_t*>(src + piece_at(am + 32 * i + frow, 2 * s + fh));
            }
#pragma unroll
            for (int i = 0; i < T::TM; ++i)
#pragma unroll
                for (int j = 0; j < T::TN; ++j)
                    acc[i][j] = mfma16<FP16>(fb[j], fa[i], acc[i][j]);
        }
    };

    if (k0 < k1) {
        fetch_b(k0);
        fetch_a(k0, 0);
        put_a(0);
        put_b(0);
        for (int kt = k0; kt < k1; ++kt) {
            const int buf = (kt - k0) & 1;
            land();
            if (kt + 1 < k1) {
                fetch_b(kt + 1);
                fetch_a(kt + 1, buf ^ 1);
            }
            __builtin_amdgcn_sched_barrier(0);
            compute(buf);
            if (kt + 1 < k1) {
                put_a(buf ^ 1);
                put_b(buf ^ 1);
            }
        }
    }
    epilogue<T>(p, w, acc);
}

/* ---------------------------------------------------------------------- */
/* launches                                                                */
/* ---------------------------------------------------------------------- */
template <int XT>
hipError_t save(const SaveArgs& a, hipStream_t stream)
{
    int lanes = 8;
    while (lanes < 256 && lanes * 8 < a.cols)
        lanes *= 2;
    const int64_t per = kSaveThreads / lanes;
    const dim3 grid(static_cast<uint32_t>((a.rows + per - 1) / per), static_cast<uint32_t>(a.batch));
    switch (lanes) {
    case 8: return launch(k_mx8_save<XT, 8>, grid, kSaveThreads, stream, a);
    case 16: return launch(k_mx8_save<XT, 16>, grid, kSaveThreads, stream, a);
    case 32: return launch(k_mx8_save<XT, 32>, grid, kSaveThreads, stream, a);
    case 64: return launch(k_mx8_save<XT, 64>, grid, kSaveThreads, stream, a);
    case 128: return launch(k_mx8_save<XT, 128>, grid, kSaveThreads, stream, a);
    default: return launch(k_mx8_save<XT, 256>, grid, kSaveThreads, stream, a);
    }
}

/* How a product is cut. */
struct Cut {
    int tile;      /* 256, 128 or 64 */
    int64_t tiles_m, tiles_n;
    int splits;
};

Cut cut_of(ProductKind kind, int64_t batch, int64_t m, int64_t n, int64_t k)
{
    constexpr int64_t kCus = 256;
    Cut c{};
    const int64_t steps = (k + (kind == kLinear ? kRowBytes : kStepK) - 1) / (kind == kLinear ? kRowBytes : kStepK);
    for (int t : {256, 128, 64}) {
        c.tile = t;
        c.tiles_m = (m + t - 1) / t;
        c.tiles_n = (n + t - 1) / t;
        if (batch * c.tiles_m * c.tiles_n >= kCus / (t == 64 ? 1 : 2))
            break;
    }
    const int64_t tiles = batch * c.tiles_m * c.tiles_n;
    const int64_t want = tiles >= kCus ? 1 : (2 * kCus + tiles - 1) / tiles, most = std::max<int64_t>(1, steps / 8);
    c.splits = static_cast<int>(std::min<int64_t>({want, most, 64}));
    return c;
}

template <typename T, typename... Flags>
hipError_t linear_tile(const ProductArgs& p, bool direct, uint32_t grid, hipStream_t stream)
{
    return direct ? launch(k_mx8_linear<T, true>, dim3(grid), T::kThreads, stream, p)
                  : launch(k_mx8_linear<T, false>, dim3(grid), T::kThreads, stream, p);
}

template <typename T, bool WGRAD>
hipError_t grad_tile(const ProductArgs& p, bool direct, uint32_t grid, hipStream_t stream)
{
    if (p.fp16)
        return direct ? launch(k_mx8_grad<T, WGRAD, true, true>, dim3(grid), T::kThreads, stream, p)
                      : launch(k_mx8_grad<T, WGRAD, true, false>, dim3(grid), T::kThreads, stream, p);
    return direct ? launch(k_mx8_grad<T, WGRAD, false, true>, dim3(grid), T::kThreads, stream, p)
                  : launch(k_mx8_grad<T, WGRAD, false, false>, dim3(grid), T::kThreads, stream, p);
}

template <typename T>
hipError_t product_tile(ProductKind kind, const ProductArgs& p, bool direct, uint32_t grid, hipStream_t stream)
{
    if (kind == kLinear)
        return linear_tile<T>(p, direct, grid, stream);
    return kind == kDgrad ? grad_tile<T, false>(p, direct, grid, stream) : grad_tile<T, true>(p, direct, grid, stream);
}

bool on16(const void* p, int64_t stride_bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride_bytes % 16 == 0; }

/* Whether the operands go straight into LDS: 16-byte pieces that lie whole in a row, at addresses that
 * 32-bit offsets from a tile's first row reach. */
bool is_direct(ProductKind kind, const ProductArgs& p, int tile)
{
    constexpr int64_t kReach = int64_t{1} << 30;
    if (kind == kLinear)
        return p.k % 16 == 0 && on16(p.a, p.a_rs) && on16(p.a, p.a_bs) && on16(p.b, p.b_rs) && on16(p.b, p.b_bs) &&
               tile * p.a_rs + p.k < kReach && tile * p.b_rs + p.k < kReach;
    if (kind == kDgrad)
        return p.k % 8 == 0 && on16(p.a, 2 * p.a_rs) && on16(p.a, 2 * p.a_bs) && 2 * (tile * p.a_rs + p.k) < kReach;
    return on16(p.a, 2 * p.a_rs) && on16(p.a, 2 * p.a_bs) && 2 * (kStepK * p.a_rs + p.m) < kReach;
}

}  // namespace

hipError_t launch_mx8_save(const SaveArgs& a, hipStream_t stream)
{
    if (a.x_dtype == HPO_PARAM_BF16)
        return save<HPO_PARAM_BF16>(a, stream);
    if (a.x_dtype == HPO_PARAM_FP16)
        return save<HPO_PARAM_FP16>(a, stream);
    return save<HPO_PARAM_FP32>(a, stream);
}

int64_t product_workspace(ProductKind kind, int64_t batch, int64_t m, int64_t n, int64_t k)
{
    const Cut c = cut_of(kind, batch, m, n, k);
    return c.splits > 1 ? 4 * batch * c.splits * m * n : 0;
}

hipError_t launch_product(ProductKind kind, ProductArgs p, hipStream_t stream)
{
    const Cut c = cut_of(kind, p.batch, p.m, p.n, p.k);
    const int64_t grid = p.batch * c.tiles_m * c.tiles_n * c.splits;
    if (grid > INT32_MAX)
        return hipErrorInvalidConfiguration;
    p.tiles_m = static_cast<int32_t>(c.tiles_m);
    p.tiles_n = static_cast<int32_t>(c.tiles_n);
    p.splits = c.splits;
    const bool direct = is_direct(kind, p, c.tile);
    const uint32_t g = static_cast<uint32_t>(grid);
    hipError_t e = c.tile == 256   ? product_tile<Tile256>(kind, p, direct, g, stream)
                   : c.tile == 128 ? product_tile<Tile128>(kind, p, direct, g, stream)
                                   : product_tile<Tile64>(kind, p, direct, g, stream);
    if (e != hipSuccess || p.splits == 1)
        return e;
    const int64_t quads = p.batch * p.m * ((p.n + 3) / 4);
    const dim3 jgrid(static_cast<uint32_t>(std::min<int64_t>((quads + kJoinThreads - 1) / kJoinThreads, 1 << 16)));
    if (p.c_dtype == HPO_PARAM_FP32)
        return launch(k_product_join<HPO_PARAM_FP32>, jgrid, kJoinThreads, stream, p);
    if (p.c_dtype == HPO_PARAM_BF16)
        return launch(k_product_join<HPO_PARAM_BF16>, jgrid, kJoinThreads, stream, p);
    return launch(k_product_join<HPO_PARAM_FP16>, jgrid, kJoinThreads, stream, p);
}

}  // namespace hpo
