/*
 * hpo_gram.hip -- gfx950 kernels of hpo_orthogonalize for matrices whose short
 * side m is at most 128 (the heads of a projection, thin or tiny matrices).
 *
 * Every step of Newton-Schulz multiplies X from the left by a polynomial of
 * A = X X^T, so with S = X0 X0^T all of them act in the m x m space:
 *     A_0 = S;   Q_k = a I + b A_k + c A_k^2;   A_{k+1} = Q_k A_k Q_k;
 *     O = (Q_last ... Q_1 Q_0) X0 = P X0
 * and the long side n is touched twice (S, then P X0) instead of twice a step.
 *   gram     one pass over the gradient (and the momentum, updated in place):
 *            partial S of a run of columns on the matrix cores
 *   iterate  one workgroup per matrix: S, its trace (the norm), the steps in LDS
 *   apply    O = P X0 in a second pass
 * P grows to a^steps in the directions of the small singular values, so every
 * product carries 22 bits: x = h + l with h = f16(x), l = f16(x - h) at a
 * power-of-two scale, and x y = h h + h l + l h (the dropped l l is 2^-22 of it) with
 * fp32 sums.  In the Gram product the two mixed terms are transposes of each other:
 * h (h + 2 l)^T, made symmetric afterwards, is the same sum in two products.
 * The scale of the raw gradient is not known before the norm is: a workgroup
 * keeps a running exponent of its largest magnitude and, when it grows, scales its
 * sums down (an exact power of two), as an online softmax does with its maximum.
 *
 * Measured on 32 x 128 x 4096 fp32 with momentum (192 MB read and written in the first pass, 128 MB
 * read and 34 MB written in the last): gram 40 us (HBM: 5.6 TB/s with its partial results), their
 * sum 7 us, iterate 47 us (32 of 256 CUs, one matrix each; matrix cores busy 41 %: the splits
 * and barriers between its 17 products of 128^3 are the rest), apply 39 us.  The form with two
 * products of the long side a step takes 1227 us there.  Tiny matrices (5 x 2 x 15) take 23 us,
 * a chain of latencies.
 *
 * Source: [HANDBOOK] "优化器：AdamW、Muon 与分布式优化器" (ai-infra-handbooks,
 * train/algo/optimizer), section on Muon: the iteration and its coefficients.
 *
 * Floating point: built with -ffp-contract=off; every elementwise operation
 * rounds on its own, in the order written.
 */
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>

#include "hpo_muon_device.h"

namespace hpo {
namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kTileElems = 8192;   /* elements of a column tile: 32 per thread */
constexpr int kTop = 14;           /* values are scaled to at most 2^14 */

struct GramArgs {
    OrthoSrc s;
    int64_t m, n;        /* short and long side */
    int64_t run;         /* columns (of the wide form) a workgroup takes in either pass, whole tiles */
    int32_t chunks;      /* workgroups per matrix */
    int32_t summed;      /* k_gram_sum has added the parts up */
    float* part;         /* [batch][chunks][MP][MP] */
    int32_t* part_exp;   /* [batch][chunks] */
    uint16_t* P;         /* [batch][2][MP][MP]: h and l of P * 2^p_exp */
    float* inv;          /* [batch][3]: 1 / d as (mantissa, exponent of X0's scale), and the result's exponent */
    uint16_t* out;
    int64_t obs, ors;
    int32_t steps;
    int32_t p_exp;       /* exponent of the final P */
    GramStep step[HPO_NS_MAX_STEPS];
};

__device__ __forceinline__ f32x16_t mfma(u32x4_t a, u32x4_t b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

/* Byte offset of 16-byte piece p of an LDS row of ROW elements, the pieces
 * permuted by the row so that a fragment's 16 rows meet distinct banks; the row's higher
 * bits spread the writes of every fourth row that a tile laid across memory makes. */
template <int ROW>
__device__ __forceinline__ int piece_at(int r, int p)
{
    int f;
    if constexpr (ROW >= 128)
        f = (r & 15) ^ ((r >> 4) & 3);
    else if constexpr (ROW == 64)
        f = (r & 7) ^ ((r >> 3) & 1) ^ ((r >> 3) & 2);
    else
        f = (r ^ (r >> 2)) & 3;
    return r * (ROW * 2) + ((p ^ f) << 4);
}

template <int ROW>
__device__ __forceinline__ u32x4_t fragment(const char* base, int row0, int slice)
{
    const int lane = threadIdx.x & 63;
    return *reinterpret_cast<const u32x4_t*>(base + piece_at<ROW>(row0 + (lane & 31), 2 * slice + (lane >> 5)));
}

/* A thread's share of one column tile, as eight runs of four elements that lie
 * together in memory.  ALONG: the eight consecutive elements of an LDS piece run
 * along memory (two runs a piece, four pieces); else across it (eight memory rows,
 * four pieces side by side).
 * LROW x LCOL is the LDS tile (LCOL consecutive elements per row). */
template <int LROW, int LCOL, bool ALONG>
struct Share {
    /* LDS row and first LDS column of piece q (0..3) */
    __device__ static __forceinline__ void piece(int q, int& r, int& c)
    {
        const int t = threadIdx.x;
        if constexpr (ALONG) {
            const int p = t + q * kThreads;
            r = p / (LCOL / 8);
            c = (p % (LCOL / 8)) * 8;
        } else {
            r = (t % (LROW / 4)) * 4 + q;
            c = (t / (LROW / 4)) * 8;
        }
    }
    /* run j (0..7): its LDS coordinates (first element) */
    __device__ static __forceinline__ void run(int j, int& r, int& c)
    {
        if constexpr (ALONG) {
            piece(j >> 1, r, c);
            c += 4 * (j & 1);
        } else {
            piece(0, r, c);
            c += j;
        }
    }
    /* element e (0..7) of piece q among the runs' values */
    __device__ static __forceinline__ float at(const f32x4_t (&v)[8], int q, int e)
    {
        return ALONG ? v[2 * q + (e >> 2)][e & 3] : v[e][q];
    }
};

/* The stored elements of a share. */
struct Raw {
    f32x4_t g[8], m[8];
};

/* One matrix: a scalar base and 32-bit element offsets (the host sends matrices that
 * span more than 2^30 elements elsewhere), or the addresses alone would take a
 * quarter of the registers. */
struct Mat {
    const char* g;
    float* m;
    uint32_t grs, mrs;
};

template <bool BF16>
__device__ __forceinline__ Mat matrix_of(const OrthoSrc& s, int64_t z)
{
    Mat x;
    x.g = static_cast<const char*>(s.G) + z * s.gbs * (BF16 ? 2 : 4);
    x.m = s.M != nullptr ? s.M + z * s.mbs : nullptr;
    x.grs = static_cast<uint32_t>(s.grs);
    x.mrs = static_cast<uint32_t>(s.mrs);
    return x;
}

template <bool BF16>
__device__ __forceinline__ f32x4_t grad_at(const char* base, uint32_t at, int n)
{
    f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (BF16) {
        const char* p = base + at * 2u;
        if (n >= 4) {
            const u32x2_t t = *reinterpret_cast<const u32x2_any*>(p);
            x[0] = bf16_to_f32(t.x & 0xffffu);
            x[1] = bf16_to_f32(t.x >> 16);
            x[2] = bf16_to_f32(t.y & 0xffffu);
            x[3] = bf16_to_f32(t.y >> 16);
            return x;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n)
                x[e] = bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[e]);
    } else {
        const char* p = base + at * 4u;
        if (n >= 4)
            return *reinterpret_cast<const f32x4_any*>(p);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n)
                x[e] = reinterpret_cast<const float*>(p)[e];
    }
    return x;
}

/* A share's elements in memory: LDS row = short side (GRAM) or long side
 * (apply), columns of the wide form from k0 on. */
template <bool TALL, bool GRAM, int LROW, int LCOL>
__device__ __forceinline__ void place(const OrthoSrc& s, int64_t k0, int j, uint32_t& row, uint32_t& col, int& cnt)
{
    int r, c;
    Share<LROW, LCOL, GRAM != TALL>::run(j, r, c);
    const int i = GRAM ? r : c, kk = static_cast<int>(k0) + (GRAM ? c : r);   /* short, long coordinate */
    const int y = TALL ? kk : i, x = TALL ? i : kk;
    row = static_cast<uint32_t>(y);
    col = static_cast<uint32_t>(x);
    const int left = y < static_cast<int>(s.rows) ? static_cast<int>(s.cols) - x : 0;
    cnt = left >= 4 ? 4 : (left > 0 ? left : 0);
}

template <bool BF16, bool TALL, bool GRAM, int LROW, int LCOL>
__device__ __forceinline__ void fetch(const GramArgs& a, const Mat& t, int64_t k0, Raw& x)
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t row, col;
        int cnt;
        place<TALL, GRAM, LROW, LCOL>(a.s, k0, j, row, col, cnt);
        x.g[j] = grad_at<BF16>(t.g, row * t.grs + col, cnt);
        if (t.m != nullptr)
            x.m[j] = grad_at<false>(reinterpret_cast<const char*>(t.m), row * t.mrs + col, cnt);
    }
}

/* g~ of a fetched share in x.g.  The first pass (GRAM) updates the momentum in
 * memory; the second reads it as it is after the update. */
template <bool TALL, bool GRAM, int LROW, int LCOL>
__device__ __forceinline__ void finish(const GramArgs& a, const Mat& t, const GradVals& k, int64_t k0, Raw& x)
{
    const MuonScalars& sc = a.s.sc;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t row, col;
        int cnt;
        place<TALL, GRAM, LROW, LCOL>(a.s, k0, j, row, col, cnt);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float g = x.g[j][e] * k.inv_scale;
            if (k.clip)
                g = g * k.C;
            x.g[j][e] = g;
        }
        if (t.m != nullptr) {
            if constexpr (GRAM) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x.m[j][e] = sc.form == HPO_MUON_MOMENTUM_SUM ? sc.mu * x.m[j][e] + x.g[j][e]
                                                                  : sc.mu * x.m[j][e] + sc.omu * x.g[j][e];
                char* p = reinterpret_cast<char*>(t.m) + (row * t.mrs + col) * 4u;
                if (cnt >= 4) {
                    *reinterpret_cast<f32x4_any*>(p) = x.m[j];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (e < cnt)
                            reinterpret_cast<float*>(p)[e] = x.m[j][e];
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x.g[j][e] = nesterov_of(x.g[j][e], x.m[j][e], sc);
        }
        /* behind the edge 0 * C is 0 or, with a clip that is not a number, not one: edges are zeros */
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e >= cnt)
                x.g[j][e] = 0.0f;
    }
}

/* h and LO * l of two values as packed pairs, both rounded to nearest even: l is
 * as often of the other sign as h, so the dropped l l does not add up. */
template <int LO>
__device__ __forceinline__ void split2(float a, float b, uint32_t& h, uint32_t& l)
{
    const f32x2_t x = {a, b};
    const f16x2_t hv = __builtin_convertvector(x, f16x2_t);
    const f32x2_t r = {static_cast<float>(LO) * (a - static_cast<float>(hv[0])),
                       static_cast<float>(LO) * (b - static_cast<float>(hv[1]))};
    h = __builtin_bit_cast(uint32_t, hv);
    l = __builtin_bit_cast(uint32_t, __builtin_convertvector(r, f16x2_t));
}

template <int LO>
__device__ __forceinline__ void split8(const float (&y)[8], u32x4_t& h, u32x4_t& l)
{
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        uint32_t hb, lb;
        split2<LO>(y[2 * w], y[2 * w + 1], hb, lb);
        h[w] = hb;
        l[w] = lb;
    }
}

/* Where the four values of rows 32 bi + 8 q + 4 (lane / 32) .. + 3, column 32 bj +
 * lane % 32 of a partial S lie, in units of four. */
template <int MP>
__device__ __forceinline__ int part_at(int bi, int bj, int q, int lane)
{
    return ((bi * (MP / 32) + bj) * 4 + q) * 64 + lane;
}

/* ---------------------------------------------------------------------- */
/* S in parts                                                              */
/* ---------------------------------------------------------------------- */
/* One workgroup's run of columns (c0 .. c1 - 1).  LDS: h and 2 l of an [MP][KC] tile.  MP = 128, 64:
 * 2 x 2 wavefronts over the MP x MP result; MP = 32: every wavefront takes a
 * quarter of the tile's columns for the whole result. */
constexpr int kTileBytes = 2 * kTileElems * 2;   /* both halves of a column tile */

template <bool BF16, int MP, bool TALL>
__device__ __forceinline__ void gram_part(const GramArgs& a, int64_t z, int64_t chunk, char* lds, uint32_t* wave_top)
{
    constexpr int KC = kTileElems / MP;
    constexpr int kBytes = kTileElems * 2;
    constexpr int kB = MP == 128 ? 2 : 1;               /* 32 x 32 blocks per wavefront and side */
    constexpr bool kSplitK = MP == 32;
    constexpr int kSlices = KC / 16 / (kSplitK ? 4 : 1);
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const GradVals gv = grad_vals(a.s.sc);
    const int64_t c0 = chunk * a.run;
    const int64_t c1 = c0 + a.run < a.n ? c0 + a.run : a.n;
    const int r0 = kSplitK ? 0 : (wave >> 1) * 32 * kB, q0 = kSplitK ? 0 : (wave & 1) * 32 * kB;
    const int s0 = kSplitK ? wave * kSlices : 0;
    f32x16_t acc[kB][kB];
#pragma unroll
    for (int i = 0; i < kB; ++i)
#pragma unroll
        for (int j = 0; j < kB; ++j)
            acc[i][j] = f32x16_t{};
    int top = -1000;   /* the sums are scaled by 2^(2 (kTop - top)) */
    using Sh = Share<MP, KC, !TALL>;
    const Mat mat = matrix_of<BF16>(a.s, z);
    Raw x;
    fetch<BF16, TALL, true, MP, KC>(a, mat, c0, x);
    for (int64_t k0 = c0; k0 < c1; k0 += KC) {
        finish<TALL, true, MP, KC>(a, mat, gv, k0, x);
        const f32x4_t(&v)[8] = x.g;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t u = __float_as_uint(v[j][e]) & 0x7fffffffu;
                m = u > m ? u : m;
            }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_xor(m, d, 64);
            m = o > m ? o : m;
        }
        if (lane == 0)
            wave_top[wave] = m;
        __syncthreads();   /* also: the previous tile's fragments are read */
        m = wave_top[0];
#pragma unroll
        for (int w = 1; w < 4; ++w)
            m = wave_top[w] > m ? wave_top[w] : m;
        /* every magnitude is under 2^e; inf and NaN stay what they are */
        int e = -1000;
        if (m >= 0x7f800000u)
            e = 128;
        else if (m != 0)
            e = m >= 0x00800000u ? static_cast<int>(m >> 23) - 126 : -117 - __clz(static_cast<int>(m));
        if (e > top) {
            if (top > -1000) {
                const int d = 2 * (top - e);
#pragma unroll
                for (int i = 0; i < kB; ++i)
#pragma unroll
                    for (int j = 0; j < kB; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            acc[i][j][r] = __builtin_ldexpf(acc[i][j][r], d);
            }
            top = e;
        }
        const int up = kTop - top;   /* no element is non-zero where top is still -1000 */
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[8];
#pragma unroll
            for (int t = 0; t < 8; ++t)
                y[t] = __builtin_ldexpf(Sh::at(v, q, t), up);
            u32x4_t h, l;
            split8<2>(y, h, l);
            int r, c;
            Sh::piece(q, r, c);
            const int off = piece_at<KC>(r, c / 8);
            *reinterpret_cast<u32x4_t*>(lds + off) = h;
            *reinterpret_cast<u32x4_t*>(lds + kBytes + off) = l;
        }
        __syncthreads();
        if (k0 + KC < c1)   /* the next tile arrives under this one's products */
            fetch<BF16, TALL, true, MP, KC>(a, mat, k0 + KC, x);
#pragma unroll
        for (int s = 0; s < kSlices; ++s) {
            u32x4_t fa[kB], fb[kB], fl[kB];
#pragma unroll
            for (int i = 0; i < kB; ++i) {
                fa[i] = fragment<KC>(lds, r0 + 32 * i, s0 + s);
                fb[i] = fragment<KC>(lds, q0 + 32 * i, s0 + s);
                fl[i] = fragment<KC>(lds + kBytes, q0 + 32 * i, s0 + s);
            }
#pragma unroll
            for (int i = 0; i < kB; ++i)
#pragma unroll
                for (int j = 0; j < kB; ++j) {
                    acc[i][j] = mfma(fa[i], fb[j], acc[i][j]);
                    acc[i][j] = mfma(fa[i], fl[j], acc[i][j]);
                }
        }
    }
    float* out = a.part + (z * a.chunks + chunk) * (MP * MP);
    if (tid == 0)
        a.part_exp[z * a.chunks + chunk] = top;
    /* in the order of the registers that the next kernel sums them in: four rows of one column
     * a lane, 1 KB an access */
    if constexpr (kSplitK) {
        /* the four wavefronts' quarters, in order */
        float* buf = reinterpret_cast<float*>(lds);
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 16; ++r)
            buf[(wave * 16 + r) * 64 + lane] = acc[0][0][r];
        __syncthreads();
        f32x4_t t;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = wave * 4 + e;
            t[e] = ((buf[r * 64 + lane] + buf[(16 + r) * 64 + lane]) + buf[(32 + r) * 64 + lane]) +
                   buf[(48 + r) * 64 + lane];
        }
        reinterpret_cast<f32x4_t*>(out)[part_at<MP>(0, 0, wave, lane)] = t;
    } else {
#pragma unroll
        for (int i = 0; i < kB; ++i)
#pragma unroll
            for (int j = 0; j < kB; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    f32x4_t t;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        t[e] = acc[i][j][4 * q + e];
                    reinterpret_cast<f32x4_t*>(out)[part_at<MP>(r0 / 32 + i, q0 / 32 + j, q, lane)] = t;
                }
    }
}

/* grid (chunks, batch) */
template <bool BF16, int MP, bool TALL>
__global__ __launch_bounds__(kThreads, 2) void k_gram(GramArgs a)
{
    if (!gate_open(a.s.sc.gate))
        return;
    __shared__ __attribute__((aligned(16))) char lds[kTileBytes];
    __shared__ uint32_t wave_top[4];
    gram_part<BF16, MP, TALL>(a, blockIdx.y, blockIdx.x, lds, wave_top);
}

/* Sums the parts of S where they are many: a workgroup takes 1024 of each matrix's values
 * (grid: MP^2 / 1024, batch) and leaves the sum, at the largest part's exponent, in the
 * first part. */
template <int MP>
__global__ __launch_bounds__(kThreads) void k_gram_sum(GramArgs a)
{
    if (!gate_open(a.s.sc.gate))
        return;
    const int64_t z = blockIdx.y;
    const int32_t* pe = a.part_exp + z * a.chunks;
    int top = -1000;
    for (int c = 0; c < a.chunks; ++c)
        top = pe[c] > top ? pe[c] : top;
    f32x4_t* part = reinterpret_cast<f32x4_t*>(a.part + z * a.chunks * (MP * MP)) + blockIdx.x * kThreads + threadIdx.x;
    f32x4_t t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int c = 0; c < a.chunks; ++c) {
        const f32x4_t x = part[c * (MP * MP / 4)];
        const int d = 2 * (pe[c] - top);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            t[e] += __builtin_ldexpf(x[e], d);
    }
    part[0] = t;
}

/* ---------------------------------------------------------------------- */
/* the steps in the m x m space                                            */
/* ---------------------------------------------------------------------- */
/* One workgroup per matrix (grid: batch), WM x WN wavefronts of BM x BN blocks.
 * All operands are symmetric, so a matrix in LDS (rows of MP, h then l) serves
 * as left and as right operand, and a lane's four consecutive rows of one
 * column are stored as four consecutive columns of one row: mul(x, y) is x^T y.
 * A is formed as Q^T A Q, from both sides: where roundings leave A and Q not quite symmetric,
 * a one-sided A^T Q Q grows that part by Q^2 a step (2 x 2 with singular values 1 and 0.02:
 * 6e-2 off after five).  Products stay at the
 * scale of their operands' exponents; the next split or sum takes that in (an
 * exact power of two). */
template <int MP>
struct Iter {
    static constexpr int WM = MP / 32, WN = MP == 32 ? 1 : 2;
    static constexpr int BN = MP / 32 / WN;   /* blocks of a wavefront: one row, BN columns */
    static constexpr int kThreads = 64 * WM * WN;
    static constexpr int kMatBytes = 2 * 2 * 2 * MP * MP, kRawBytes = MP * (MP + 1) * 4;
    static constexpr int kLds = kMatBytes > kRawBytes ? kMatBytes : kRawBytes;
};

__device__ __forceinline__ float pow2f(int e) { return __builtin_ldexpf(1.0f, e); }

/* `wave`: the wavefront's place; wavefronts that share one do the same work and store the
 * same values. */
template <int MP>
__device__ __forceinline__ void iterate(const GramArgs& a, int64_t z, int wave, char* lds)
{
    constexpr int WN = Iter<MP>::WN, BN = Iter<MP>::BN;
    constexpr int kPlane = MP * MP * 2, kBuf = 2 * kPlane;
    const int tid = threadIdx.x, lane = tid & 63;
    const int r0 = (wave / WN) * 32, q0 = (wave % WN) * 32 * BN;
    typedef f32x16_t Block[BN];
    const int lrow = r0 + 4 * (lane >> 5), lcol = q0 + (lane & 31);
    auto row_of = [&](int r) { return lrow + 8 * (r >> 2) + (r & 3); };
    auto col_of = [&](int j) { return lcol + 32 * j; };

    /* S: the parts at their largest exponent, in order */
    const int32_t* pe = a.part_exp + z * a.chunks;
    int top = -1000;
    for (int c = 0; c < a.chunks; ++c)
        top = pe[c] > top ? pe[c] : top;
    Block A, P, Q, acc;
#pragma unroll
    for (int j = 0; j < BN; ++j)
        A[j] = f32x16_t{};
    for (int c = 0; c < (a.summed ? 1 : a.chunks); ++c) {
        const f32x4_t* part = reinterpret_cast<const f32x4_t*>(a.part + (z * a.chunks + c) * (MP * MP));
        const int d = a.summed ? 0 : 2 * (pe[c] - top);
        f32x4_t t[BN][4];
#pragma unroll
        for (int j = 0; j < BN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                t[j][q] = part[part_at<MP>(r0 / 32, q0 / 32 + j, q, lane)];
#pragma unroll
        for (int j = 0; j < BN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                A[j][r] += __builtin_ldexpf(t[j][r >> 2][r & 3], d);
    }
    /* (S + S^T) / 2 and the trace */
    float* raw = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int j = 0; j < BN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            raw[row_of(r) * (MP + 1) + col_of(j)] = A[j][r];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < BN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            A[j][r] = 0.5f * (A[j][r] + raw[col_of(j) * (MP + 1) + row_of(r)]);
    /* every lane of every wavefront sums the same diagonal in the same order */
    double trace = 0.0;
    for (int i = lane; i < MP; i += 64)
        trace += static_cast<double>(raw[i * (MP + 1) + i]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        trace += __shfl_xor(trace, off, 64);
    __syncthreads();
    /* d = ||g~|| + eps; the sums are at scale 2^(2 (kTop - top)) */
    const double unit = ldexp(1.0, top > -1000 ? top - kTop : 0), norm = sqrt(trace) * unit;
    const float df = static_cast<float>(norm) + a.s.sc.eps;
    /* under fp32's normal numbers the sum stays in binary64: a subnormal keeps few bits, or none */
    const double d = df < FLT_MIN ? norm + static_cast<double>(a.s.sc.eps) : static_cast<double>(df);
    const double id = d == 0.0 ? 0.0 : 1.0 / d;
    /* A norm far under eps leaves X0 far under 1, and its two fp16 values would keep few bits: X0 and
     * the result are held 2^lift larger (P does not depend on X0's scale). */
    const int lift = far_below_eps(norm, a.s.sc.eps) ? -1 - ilogb(norm * id) : 0;
    /* the factor of A as a value in [1/2, 1) and an exponent */
    int fe = 0;
    const float fm = static_cast<float>(frexp(trace == 0.0 ? 0.0 : (unit * id) * (unit * id), &fe));
    if (tid == 0) {
        /* 1 / d as mantissa and exponent: it may lie beyond fp32's range.  0 (d beyond it) takes no
         * scale, which would make an infinity of large elements. */
        int e = 0;
        const double mant = frexp(id, &e);
        a.inv[3 * z] = static_cast<float>(mant);
        a.inv[3 * z + 1] = id == 0.0 ? 0.0f : static_cast<float>(e + kTop + lift);
        a.inv[3 * z + 2] = static_cast<float>(-(a.p_exp + kTop + lift));
    }
#pragma unroll
    for (int j = 0; j < BN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            A[j][r] = __builtin_ldexpf(A[j][r] * fm, fe);

    char* b0 = lds;
    char* b1 = lds + kBuf;
    /* x * 2^e, split, into buf */
    auto put = [&](char* buf, const Block& x, int e) {
        const float s = pow2f(e);
#pragma unroll
        for (int j = 0; j < BN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                /* rows row_of(4 q) + 0..3 of column col_of(j), stored as that row's columns */
                u32x2_t h, l;
                uint32_t hb, lb;
                split2<1>(x[j][4 * q] * s, x[j][4 * q + 1] * s, hb, lb);
                h.x = hb;
                l.x = lb;
                split2<1>(x[j][4 * q + 2] * s, x[j][4 * q + 3] * s, hb, lb);
                h.y = hb;
                l.y = lb;
                const int c = lrow + 8 * q;
                const int off = piece_at<MP>(col_of(j), c >> 3) + ((c >> 2) & 1) * 8;
                *reinterpret_cast<u32x2_t*>(buf + off) = h;
                *reinterpret_cast<u32x2_t*>(buf + kPlane + off) = l;
            }
    };
    /* One slice's fragments are read under the last one's products (one scheduling region per
     * slice: left alone the compiler reads far ahead and spills). */
    auto mul = [&](const char* x, const char* y, Block& out) {
#pragma unroll
        for (int j = 0; j < BN; ++j)
            out[j] = f32x16_t{};
        u32x4_t xh[2], xl[2], yh[2][BN], yl[2][BN];
        auto read = [&](int s) {
            xh[s & 1] = fragment<MP>(x, r0, s);
            xl[s & 1] = fragment<MP>(x + kPlane, r0, s);
#pragma unroll
            for (int j = 0; j < BN; ++j) {
                yh[s & 1][j] = fragment<MP>(y, q0 + 32 * j, s);
                yl[s & 1][j] = fragment<MP>(y + kPlane, q0 + 32 * j, s);
            }
        };
        read(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int s = 0; s < MP / 16; ++s) {
            if (s + 1 < MP / 16)
                read(s + 1);
#pragma unroll
            for (int j = 0; j < BN; ++j)
                out[j] = mfma(xh[s & 1], yh[s & 1][j], out[j]);
#pragma unroll
            for (int j = 0; j < BN; ++j)
                out[j] = mfma(xh[s & 1], yl[s & 1][j], out[j]);
#pragma unroll
            for (int j = 0; j < BN; ++j)
                out[j] = mfma(xl[s & 1], yh[s & 1][j], out[j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    int ae = 0, pq = 0;   /* A's and P's registers hold A 2^ae and P 2^pq */
    put(b0, A, a.step[0].a_exp);
    __syncthreads();
    for (int k = 0; k < a.steps; ++k) {
        const GramStep& g = a.step[k];
        const bool first = k == 0, last = k + 1 == a.steps;
        mul(b0, b0, acc);
        const float fb = g.b * pow2f(-ae), fc = g.c * pow2f(-2 * g.a_exp);
#pragma unroll
        for (int j = 0; j < BN; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float diag = row_of(r) == col_of(j) ? g.a : 0.0f;
                Q[j][r] = diag + (fb * A[j][r] + fc * acc[j][r]);
            }
        if (first) {
#pragma unroll
            for (int j = 0; j < BN; ++j)
                P[j] = Q[j];
        }
        if (first && last)
            break;
        put(b1, Q, g.q_exp);
        __syncthreads();
        if (!last)
            mul(b0, b1, acc);   /* T = A^T Q */
        if (!first) {
            __syncthreads();
            put(b0, P, g.p_exp - pq);
            __syncthreads();
            mul(b1, b0, P);
            pq = g.q_exp + g.p_exp;
        }
        if (!last) {
            __syncthreads();
            put(b0, acc, g.t_exp - g.q_exp - g.a_exp);
            __syncthreads();
            mul(b0, b1, A);     /* A = T^T Q = Q^T A Q */
            ae = g.t_exp + g.q_exp;
            __syncthreads();
            put(b0, A, a.step[k + 1].a_exp - ae);
            __syncthreads();
        }
    }
    /* P for the last pass: rows of 16-bit values, h then l.  Row by row as it is, not transposed:
     * roundings leave P = Q_last ... Q_0 not quite symmetric, and what they put into the block that takes a strong
     * direction of X0 to its small ones is grown by every later Q, the other block's by every
     * earlier one, and only the first meets large elements of X0 (one direction over 0.1 % of
     * noise: 1e-2 of the result with P^T, 4e-4 with P). */
    uint16_t* out = a.P + z * (2 * MP * MP);
    const float s = pow2f(a.p_exp - pq);
#pragma unroll
    for (int j = 0; j < BN; ++j)
#pragma unroll
        for (int r = 0; r < 16; r += 2) {
            uint32_t h, l;
            split2<1>(P[j][r] * s, P[j][r + 1] * s, h, l);
            const int at = row_of(r) * MP + col_of(j);
            out[at] = static_cast<uint16_t>(h & 0xffffu);
            out[at + MP] = static_cast<uint16_t>(h >> 16);
            out[MP * MP + at] = static_cast<uint16_t>(l & 0xffffu);
            out[MP * MP + at + MP] = static_cast<uint16_t>(l >> 16);
        }
}

template <int MP>
__global__ __launch_bounds__(Iter<MP>::kThreads) void k_gram_iterate(GramArgs a)
{
    if (!gate_open(a.s.sc.gate))
        return;
    __shared__ __attribute__((aligned(16))) char lds[Iter<MP>::kLds];
    iterate<MP>(a, blockIdx.x, threadIdx.x >> 6, lds);
}

/* ---------------------------------------------------------------------- */
/* O = P X0                                                                */
/* ---------------------------------------------------------------------- */
/* One workgroup's run of columns.  LDS: h and l of a [KC][MP] tile (X0's columns).  Each
 * wavefront takes 32 rows of P (its fragments in registers) and two blocks of 32
 * columns; the result of a tall matrix comes out transposed, so that lanes always
 * run along its rows. */
template <bool BF16, int MP, bool TALL>
__device__ __forceinline__ void apply(const GramArgs& a, int64_t z, int64_t chunk, char* lds)
{
    constexpr int KC = kTileElems / MP;
    constexpr int kBytes = kTileElems * 2;
    constexpr int kSlices = MP / 16;
    constexpr int kRowBlocks = MP / 32;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const GradVals gv = grad_vals(a.s.sc);
    const int64_t c0 = chunk * a.run;
    const int64_t c1 = c0 + a.run < a.n ? c0 + a.run : a.n;
    const float mant = a.inv[3 * z];
    const int ex = static_cast<int>(a.inv[3 * z + 1]), down = static_cast<int>(a.inv[3 * z + 2]);
    const int i0 = (wave % kRowBlocks) * 32, j0 = (wave / kRowBlocks) * 64;
    u32x4_t ph[kSlices], pl[kSlices];
    const uint16_t* P = a.P + z * (2 * MP * MP);
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
        const int at = (i0 + (lane & 31)) * MP + 16 * s + 8 * (lane >> 5);
        ph[s] = *reinterpret_cast<const u32x4_t*>(P + at);
        pl[s] = *reinterpret_cast<const u32x4_t*>(P + MP * MP + at);
    }
    using Sh = Share<KC, MP, TALL>;
    const Mat mat = matrix_of<BF16>(a.s, z);
    Raw x;
    fetch<BF16, TALL, false, KC, MP>(a, mat, c0, x);
    for (int64_t k0 = c0; k0 < c1; k0 += KC) {
        finish<TALL, false, KC, MP>(a, mat, gv, k0, x);
        const f32x4_t(&v)[8] = x.g;
        __syncthreads();   /* the previous tile's fragments are read */
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[8];
#pragma unroll
            for (int t = 0; t < 8; ++t)
                y[t] = __builtin_ldexpf(Sh::at(v, q, t), ex) * mant;   /* scaled first: it may be subnormal */
            u32x4_t h, l;
            split8<1>(y, h, l);
            int r, c;
            Sh::piece(q, r, c);
            const int off = piece_at<MP>(r, c / 8);
            *reinterpret_cast<u32x4_t*>(lds + off) = h;
            *reinterpret_cast<u32x4_t*>(lds + kBytes + off) = l;
        }
        __syncthreads();
        if (k0 + KC < c1)
            fetch<BF16, TALL, false, KC, MP>(a, mat, k0 + KC, x);
        f32x16_t acc[2] = {f32x16_t{}, f32x16_t{}};
#pragma unroll
        for (int s = 0; s < kSlices; ++s) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u32x4_t xh = fragment<MP>(lds, j0 + 32 * j, s);
                const u32x4_t xl = fragment<MP>(lds + kBytes, j0 + 32 * j, s);
                if constexpr (TALL) {
                    acc[j] = mfma(xh, ph[s], acc[j]);
                    acc[j] = mfma(xl, ph[s], acc[j]);
                    acc[j] = mfma(xh, pl[s], acc[j]);
                } else {
                    acc[j] = mfma(ph[s], xh, acc[j]);
                    acc[j] = mfma(ph[s], xl, acc[j]);
                    acc[j] = mfma(pl[s], xh, acc[j]);
                }
            }
        }
        char* out = reinterpret_cast<char*>(a.out + z * a.obs);
        const uint32_t ors = static_cast<uint32_t>(a.ors);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int reg = 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                const int i = i0 + (TALL ? lane & 31 : reg);
                const int kk = static_cast<int>(k0) + j0 + 32 * j + (TALL ? reg : lane & 31);
                if (i < static_cast<int>(a.m) && kk < static_cast<int>(a.n)) {
                    const uint32_t at = TALL ? static_cast<uint32_t>(kk) * ors + i : static_cast<uint32_t>(i) * ors + kk;
                    *reinterpret_cast<uint16_t*>(out + at * 2u) =
                        static_cast<uint16_t>(bf16_rne_bits(__builtin_ldexpf(acc[j][r], down)));
                }
            }
    }
}

/* grid (chunks, batch) */
template <bool BF16, int MP, bool TALL>
__global__ __launch_bounds__(kThreads, 2) void k_gram_apply(GramArgs a)
{
    if (!gate_open(a.s.sc.gate))
        return;
    __shared__ __attribute__((aligned(16))) char lds[kTileBytes];
    apply<BF16, MP, TALL>(a, blockIdx.y, blockIdx.x, lds);
}

/* All three where one workgroup takes a whole matrix (grid: batch): what a
 * workgroup wrote to its own scratch it reads behind a barrier. */
template <bool BF16, int MP, bool TALL>
__global__ __launch_bounds__(kThreads, 2) void k_gram_whole(GramArgs a)
{
    if (!gate_open(a.s.sc.gate))
        return;
    static_assert(Iter<MP>::kLds <= kTileBytes && Iter<MP>::kThreads <= kThreads, "the steps fit the tile's LDS");
    __shared__ __attribute__((aligned(16))) char lds[kTileBytes];
    __shared__ uint32_t wave_top[4];
    const int64_t z = blockIdx.x;
    gram_part<BF16, MP, TALL>(a, z, 0, lds, wave_top);
    __syncthreads();
    iterate<MP>(a, z, (threadIdx.x >> 6) % (Iter<MP>::kThreads / 64), lds);
    __syncthreads();
    apply<BF16, MP, TALL>(a, z, 0, lds);
}

template <typename... Args>
hipError_t launch(void (*kernel)(Args...), dim3 grid, int block, hipStream_t stream, Args... args)
{
    void* argv[] = {static_cast<void*>(&args)...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(block), argv, 0, stream);
}

int mp_of(int64_t m) { return m <= 32 ? 32 : (m <= 64 ? 64 : 128); }

struct GramPlan {
    int mp;
    int64_t m, n, run, chunks, count;
    int64_t slot;   /* bytes of one matrix */
};

GramPlan gram_plan(int64_t batch, int64_t rows, int64_t cols)
{
    GramPlan p{};
    p.m = rows > cols ? cols : rows;
    p.n = rows > cols ? rows : cols;
    p.mp = mp_of(p.m);
    const int64_t kc = kTileElems / p.mp, tiles = (p.n + kc - 1) / kc;
    /* both passes: one round of two workgroups a CU */
    int64_t per = std::max<int64_t>((tiles * batch + 511) / 512, 1);
    p.chunks = (tiles + per - 1) / per;
    per = (tiles + p.chunks - 1) / p.chunks;
    p.chunks = (tiles + per - 1) / per;
    p.run = per * kc;
    p.slot = (4 * p.chunks + 4) * p.mp * p.mp + 4 * p.chunks + 12;
    constexpr int64_t kCap = int64_t{4} << 30;
    const int64_t most = kCap / p.slot > 1 ? kCap / p.slot : 1;
    const int64_t slices = (batch + most - 1) / most;
    p.count = (batch + slices - 1) / slices;
    return p;
}

template <bool BF16, int MP, bool TALL>
hipError_t run(const GramArgs& a, uint32_t count, hipStream_t stream)
{
    if constexpr (MP <= 64) {
        if (a.chunks == 1)
            return launch(k_gram_whole<BF16, MP, TALL>, dim3(count), kThreads, stream, a);
    }
    const dim3 grid(static_cast<uint32_t>(a.chunks), count);
    hipError_t e = launch(k_gram<BF16, MP, TALL>, grid, kThreads, stream, a);
    if (e != hipSuccess)
        return e;
    if (a.summed) {
        e = launch(k_gram_sum<MP>, dim3(MP * MP / 4 / kThreads, count), kThreads, stream, a);
        if (e != hipSuccess)
            return e;
    }
    e = launch(k_gram_iterate<MP>, dim3(count), Iter<MP>::kThreads, stream, a);
    if (e != hipSuccess)
        return e;
    return launch(k_gram_apply<BF16, MP, TALL>, grid, kThreads, stream, a);
}

template <bool BF16, int MP>
hipError_t run_tall(const GramArgs& a, bool tall, uint32_t count, hipStream_t stream)
{
    return tall ? run<BF16, MP, true>(a, count, stream) : run<BF16, MP, false>(a, count, stream);
}

template <bool BF16>
hipError_t run_mp(const GramArgs& a, int mp, bool tall, uint32_t count, hipStream_t stream)
{
    if (mp == 32)
        return run_tall<BF16, 32>(a, tall, count, stream);
    if (mp == 64)
        return run_tall<BF16, 64>(a, tall, count, stream);
    return run_tall<BF16, 128>(a, tall, count, stream);
}

}  // namespace

int64_t gram_workspace(int64_t batch, int64_t rows, int64_t cols)
{
    const GramPlan p = gram_plan(batch, rows, cols);
    return p.count * p.slot;
}

hipError_t launch_gram(const OrthoArgs& o, hipStream_t stream)
{
    const GramPlan p = gram_plan(o.batch, o.rows, o.cols);
    const bool tall = o.rows > o.cols;
    for (int64_t z0 = 0; z0 < o.batch; z0 += p.count) {
        const int64_t count = o.batch - z0 < p.count ? o.batch - z0 : p.count;
        GramArgs a{};
        a.s = slice_of(o, z0);
        a.m = p.m;
        a.n = p.n;
        a.run = p.run;
        a.chunks = static_cast<int32_t>(p.chunks);
        /* one workgroup reads about 256 KB in the time that another launch costs */
        a.summed = p.chunks * p.mp * p.mp * 4 > (int64_t{1} << 18) ? 1 : 0;
        char* at = static_cast<char*>(o.ws);
        a.part = reinterpret_cast<float*>(at);
        at += 4 * p.count * p.chunks * p.mp * p.mp;
        a.P = reinterpret_cast<uint16_t*>(at);
        at += 4 * p.count * p.mp * p.mp;
        a.inv = reinterpret_cast<float*>(at);
        at += 12 * p.count;
        a.part_exp = reinterpret_cast<int32_t*>(at);
        a.out = static_cast<uint16_t*>(o.out.data) + z0 * o.out.bs;
        a.obs = o.out.bs;
        a.ors = o.out.rs;
        a.steps = o.steps;
        a.p_exp = o.p_exp;
        for (int k = 0; k < o.steps; ++k)
            a.step[k] = o.gram[k];
        const hipError_t e = o.g_bf16 ? run_mp<true>(a, p.mp, tall, static_cast<uint32_t>(count), stream)
                                      : run_mp<false>(a, p.mp, tall, static_cast<uint32_t>(count), stream);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

}  // namespace hpo
