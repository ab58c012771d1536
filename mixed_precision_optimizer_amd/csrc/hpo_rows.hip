/*
 * hpo_rows.hip -- gfx950 kernels that update the fp32 master of a stack of
 * matrices row by row and write the model weight: the row-normalised update
 * (hpo_rms_update) and QK-clip (hpo_qk_clip).
 *
 * Both are bound by HBM: the update moves 2 (or 4) bytes of O, 8 of the master
 * and 2 (bf16) or 1 + 1/32 (8 bits) of the weight per element.  A wavefront
 * takes pieces of 256 consecutive elements of one row, four per lane, so that
 * every master access is one whole 1 KB run, and a scale block of 32 elements
 * lies in eight neighbouring lanes.
 *
 * Measured: 4096 x 14336, bf16 O and weight: statistics 24 us (4.9 TB/s of O), update 108 us
 * (6.5 TB/s of its 12 bytes per element); 16 x 1024 x 2048 with 8-bit weights 16 and 59 us; 129 x 257:
 * 4 and 4 us, 11 us with the binding.  Rows under 256 columns leave lanes of their piece idle: 65536 x 64
 * takes 61 us (50 MB), 32768 x 128 38 us, 16384 x 256 26 us.  Clip of one layer (4096 x 4096 and 1024 x 4096
 * rows, nearly all clipped): 37 to 40 us, 5.3 to 5.7 TB/s.
 *
 * Floating point: built with -ffp-contract=off; every elementwise operation
 * rounds on its own, in the order written.
 */
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>

#include "hpo_device.h"
#include "hpo_stack_impl.h"

namespace hpo {
namespace {

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
/* Four elements at any element's address: global memory takes such an access in one
 * instruction, a line more where it straddles one. */
typedef f32x4_t f32x4_any __attribute__((aligned(4)));
typedef u32x2_t u32x2_any __attribute__((aligned(2)));
typedef uint32_t u32_any __attribute__((aligned(1)));

constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kPiece = 256;        /* elements of a row that one wavefront takes at a time */
constexpr int kUnroll = 2;         /* pieces in flight at a time, where there is much to do */
constexpr int kMxBlock = 32;

/* ---------------------------------------------------------------------- */
/* four consecutive elements of a row                                      */
/* ---------------------------------------------------------------------- */
/* n of them are in the row (n <= 0: none); the others read as 0 and are not written. */
/* NT: an access that goes around the caches, for arrays that do not fit them. */
template <typename V, bool NT, typename T>
__device__ __forceinline__ V get(const T* p)
{
    if constexpr (NT)
        return __builtin_nontemporal_load(reinterpret_cast<const V*>(p));
    else
        return *reinterpret_cast<const V*>(p);
}

template <typename V, bool NT, typename T, typename X>
__device__ __forceinline__ void set(T* p, X x)
{
    if constexpr (NT)
        __builtin_nontemporal_store(x, reinterpret_cast<V*>(p));
    else
        *reinterpret_cast<V*>(p) = x;
}

template <bool NT = false>
__device__ __forceinline__ f32x4_t load4(const float* p, int n)
{
    f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n >= 4)
        return get<f32x4_any, NT>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n)
            x[e] = p[e];
    return x;
}

__device__ __forceinline__ f32x4_t load4(const uint16_t* p, int n)
{
    f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
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
            x[e] = bf16_to_f32(p[e]);
    return x;
}

template <bool NT = false>
__device__ __forceinline__ void store4(float* p, f32x4_t x, int n)
{
    if (n >= 4) {
        set<f32x4_any, NT>(p, x);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n)
            p[e] = x[e];
}

template <bool NT>
__device__ __forceinline__ void store_bf16(uint16_t* p, f32x4_t x, int n)
{
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        b[e] = bf16_rne_bits(x[e]);
    if (n >= 4) {
        u32x2_t t;
        t.x = b[0] | (b[1] << 16);
        t.y = b[2] | (b[3] << 16);
        set<u32x2_any, NT>(p, t);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n)
            p[e] = static_cast<uint16_t>(b[e]);
}

/* HPO_WEIGHT_MX8.  All 64 lanes take part (eight lanes hold one scale block);
 * elements behind the row's end come in as 0 and do not count.  The largest
 * magnitude is compared as bits: of finite values it orders them, and inf and
 * NaN come out above.  floor(log2) of a normal value is its exponent field - 127;
 * the scale byte is that field - 8, and 0 from 2^-118 down.  Multiplying by
 * 2^-e is exact or below e4m3's smallest half step; the conversion rounds to
 * nearest even. */
template <bool NT>
__device__ __forceinline__ void store_mx8(uint8_t* p, uint8_t* scale, f32x4_t x, int n)
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t u = __float_as_uint(x[e]) & 0x7fffffffu;
        m = u > m ? u : m;
    }
#pragma unroll
    for (int d = 1; d < kMxBlock / 4; d <<= 1) {
        const uint32_t o = __shfl_xor(m, d, 64);
        m = o > m ? o : m;
    }
    const bool bad = m >= 0x7f800000u;
    const uint32_t field = m >> 23;
    const uint32_t byte = bad ? 255u : (field > 8u ? field - 8u : 0u);
    uint32_t v = 0x7f7f7f7fu;
    if (!bad) {
        const float inv = __uint_as_float((254u - byte) << 23);
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = fminf(fmaxf(x[e] * inv, -448.0f), 448.0f);
        int t = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        t = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], t, true);
        v = static_cast<uint32_t>(t);
    }
    if (n > 0 && (threadIdx.x & 7) == 0)
        *scale = static_cast<uint8_t>(byte);
    if (n >= 4) {
        set<u32_any, NT>(p, v);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n)
            p[e] = static_cast<uint8_t>(v >> (8 * e));
}

/* Where a lane's four elements of one piece lie. */
struct Spot {
    int64_t row;
    int64_t col;
    int n;   /* elements inside the row */
};

__device__ __forceinline__ Spot spot_of(int64_t row, int64_t piece, int64_t cols)
{
    Spot s;
    s.row = row;
    s.col = piece * kPiece + 4 * (threadIdx.x & 63);
    const int64_t left = cols - s.col;
    s.n = left > 4 ? 4 : static_cast<int>(left);
    return s;
}

template <int PT, bool NT = false>
__device__ __forceinline__ void store_weight(const WeightView& w, int64_t z, const Spot& s, f32x4_t x)
{
    if constexpr (PT == HPO_PARAM_BF16) {
        store_bf16<NT>(static_cast<uint16_t*>(w.param.data) + z * w.param.bs + s.row * w.param.rs + s.col, x, s.n);
    } else if constexpr (PT == HPO_WEIGHT_MX8) {
        const int64_t nb = (w.cols + kMxBlock - 1) / kMxBlock;
        store_mx8<NT>(static_cast<uint8_t*>(w.param.data) + z * w.param.bs + s.row * w.param.rs + s.col,
                  w.scales + (z * w.rows + s.row) * nb + s.col / kMxBlock, x, s.n);
    }
}

__device__ __forceinline__ bool skipped(const int32_t* d_found) { return d_found != nullptr && *d_found != 0; }

/* ---------------------------------------------------------------------- */
/* hpo_rms_update                                                          */
/* ---------------------------------------------------------------------- */
constexpr int kStatRows = 4;    /* rows of a workgroup, one wavefront each */

/* x, the largest finite value in place of an infinity. */
__device__ __forceinline__ float finite(float x) { return __builtin_isinf(x) ? __builtin_copysignf(FLT_MAX, x) : x; }
__device__ __forceinline__ double finite(double x) { return __builtin_isinf(x) ? __builtin_copysign(DBL_MAX, x) : x; }

/* Squares of eight consecutive elements, n of them in the row. */
template <typename OT>
__device__ __forceinline__ float square8(const OT* p, int64_t n)
{
    const int m = n > 8 ? 8 : static_cast<int>(n);
    const f32x4_t x = load4(p, m), y = load4(p + 4, m - 4);
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        s += x[e] * x[e];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        s += y[e] * y[e];
    return s;
}

/* Row statistics from the row's sum of squares: the running v, r, and the row's part of N^2. */
__device__ __forceinline__ double finish_row(const RmsArgs& a, int64_t idx, double tot)
{
    const double ms = tot / static_cast<double>(a.w.cols);
    float v = static_cast<float>(ms);
    if (a.v != nullptr) {
        if (a.beta2 > 0.0)
            v = static_cast<float>(a.beta2 * static_cast<double>(a.v[idx]) + (1.0 - a.beta2) * ms);
        a.v[idx] = v;
    }
    const double den = sqrt(static_cast<double>(v)) + a.eps;
    /* Finite in fp32: only a row with v = 0 comes to the limit, and every such row comes to the same
     * 1 / eps; its ratio to the rows with v > 0 (at most 2^75) is beyond binary64's bits either way. */
    const double r = den == 0.0 ? 0.0 : (den * FLT_MAX < 1.0 ? FLT_MAX : 1.0 / den);
    a.r[idx] = static_cast<float>(r);
    return tot * r * r;
}

/* Sum of squares of each row; a part of N^2 per workgroup (grid: parts, batch).  A
 * wavefront takes a row (4 a workgroup); few long rows take a workgroup each, which
 * then is a part of its own. */
template <typename OT>
__global__ __launch_bounds__(64 * kStatRows) void k_row_stats(RmsArgs a)
{
    if (skipped(a.d_found))
        return;
    __shared__ double part[kStatRows];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t z = blockIdx.y, rows = a.w.rows, cols = a.w.cols;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kStatRows + wave;
    double q = 0.0;
    if (i < rows) {
        const OT* __restrict__ o = static_cast<const OT*>(a.O.data) + z * a.O.bs + i * a.O.rs;
        float acc = 0.0f;
#pragma unroll 4
        for (int64_t c = 8 * lane; c < cols; c += 8 * 64)
            acc += square8(o + c, cols - c);
        double tot = static_cast<double>(acc);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            tot += __shfl_down(tot, off, 64);
        if (lane == 0)
            q = finish_row(a, z * rows + i, tot);
    }
    if (lane == 0)
        part[wave] = q;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = 0.0;
#pragma unroll
        for (int w = 0; w < kStatRows; ++w)
            t += part[w];
        a.q[z * a.parts + blockIdx.x] = t;
    }
}

template <typename OT>
__global__ __launch_bounds__(kRowThreads) void k_long_row_stats(RmsArgs a)
{
    if (skipped(a.d_found))
        return;
    const int64_t z = blockIdx.y, i = blockIdx.x, cols = a.w.cols;
    const OT* __restrict__ o = static_cast<const OT*>(a.O.data) + z * a.O.bs + i * a.O.rs;
    float acc = 0.0f;
#pragma unroll 4
    for (int64_t c = 8 * threadIdx.x; c < cols; c += 8 * kRowThreads)
        acc += square8(o + c, cols - c);
    const double tot = block_sum<kRowThreads>(static_cast<double>(acc));
    if (threadIdx.x == 0)
        a.q[z * a.parts + i] = finish_row(a, z * a.w.rows + i, tot);
}

/* N^2 of each matrix from very many parts: one workgroup, fixed order. */
__global__ __launch_bounds__(kRowThreads) void k_row_fold(RmsArgs a)
{
    if (skipped(a.d_found))
        return;
    const double* q = a.q + static_cast<int64_t>(blockIdx.x) * a.parts;
    double acc = 0.0;
    for (int64_t i = threadIdx.x; i < a.parts; i += kRowThreads)
        acc += q[i];
    const double tot = block_sum<kRowThreads>(acc);
    if (threadIdx.x == 0)
        a.norm2[blockIdx.x] = tot;
}

/* The pieces of one workgroup, U at a time: fn(spots) gets U spots of which the
 * first `n` are in the matrix.  Wavefronts take runs of consecutive pieces. */
template <int U, typename F>
__device__ __forceinline__ void each_piece(int64_t rows, int64_t cols, int64_t block, int32_t rounds, F&& fn)
{
    const int64_t pieces = (cols + kPiece - 1) / kPiece;
    const int wave = threadIdx.x >> 6;
    const int64_t t = (block * kRowWaves + wave) * rounds * U;
    int64_t row = t / pieces, piece = t % pieces;
    for (int k = 0; k < rounds && row < rows; ++k) {
        Spot s[U];
        int n = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = spot_of(row < rows ? row : rows - 1, piece, cols);
            if (row < rows)
                n = u + 1;
            else
                s[u].n = 0;
            if (++piece == pieces) {
                piece = 0;
                ++row;
            }
        }
        fn(s, n);
    }
}

/* W <- W keep - (s r_i) O_i, and the model weight.  FOLDED: N^2 was summed by
 * k_row_fold; else every workgroup sums the matrix's parts itself. */
template <typename OT, int PT, bool FOLDED, int U, bool NT>
__global__ __launch_bounds__(kRowThreads) void k_rms_apply(RmsArgs a)
{
    if (skipped(a.d_found))
        return;
    const int64_t z = blockIdx.y, rows = a.w.rows, cols = a.w.cols;
    double n2;
    if constexpr (FOLDED) {
        n2 = a.norm2[z];
    } else {
        __shared__ double total;
        double acc = 0.0;
        for (int64_t i = threadIdx.x; i < a.parts; i += kRowThreads)
            acc += a.q[z * a.parts + i];
        acc = block_sum<kRowThreads>(acc);
        if (threadIdx.x == 0)
            total = acc;
        __syncthreads();
        n2 = total;
    }
    /* finite, as the coefficients are: a row of zeros, or one with r = 0, stays where it is */
    const double s = n2 > 0.0 ? finite(a.gain / sqrt(n2)) : 0.0;
    each_piece<U>(rows, cols, blockIdx.x, a.rounds, [&](const Spot(&p)[U], int n) {
        f32x4_t o[U], x[U];
        float c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            c[u] = finite(static_cast<float>(s * static_cast<double>(a.r[z * rows + p[u].row])));
            o[u] = load4(static_cast<const OT*>(a.O.data) + z * a.O.bs + p[u].row * a.O.rs + p[u].col, p[u].n);
            x[u] = load4<NT>(static_cast<const float*>(a.w.master.data) + z * a.w.master.bs + p[u].row * a.w.master.rs +
                                 p[u].col,
                             p[u].n);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u >= n)
                break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float kept = x[u][e] * a.keep;
                const float d = c[u] * o[u][e];
                x[u][e] = kept - d;
            }
            store4<NT>(static_cast<float*>(a.w.master.data) + z * a.w.master.bs + p[u].row * a.w.master.rs + p[u].col,
                       x[u], p[u].n);
            store_weight<PT, NT>(a.w, z, p[u], x[u]);
        }
    });
}

/* ---------------------------------------------------------------------- */
/* hpo_qk_clip                                                             */
/* ---------------------------------------------------------------------- */
template <bool NT>
__global__ __launch_bounds__(kRowThreads) void k_qk_clip(ClipArgs a)
{
    if (skipped(a.d_found))
        return;
    const int64_t b = blockIdx.x;
    int k = 0;
    while (k + 1 < a.n && b >= a.item[k + 1].first_block)
        ++k;
    const ClipItem& it = a.item[k];
    const int64_t z = (b - it.first_block) / it.blocks, part = (b - it.first_block) % it.blocks;
    /* the largest finite logit over the threshold among the heads that share this gamma */
    const int per = a.heads / a.kv_heads;
    int h0 = static_cast<int>(z), h1 = h0 + 1;
    if (it.heads != a.heads) {
        h0 = static_cast<int>(z) * per;
        h1 = h0 + per;
    } else if (it.per_group) {
        h0 = static_cast<int>(z) / per * per;
        h1 = h0 + per;
    }
    double top = a.tau;
    for (int h = h0; h < h1; ++h) {
        const float s = a.d_max[h];
        if (isfinite(s) && static_cast<double>(s) > top)
            top = static_cast<double>(s);
    }
    if (!(top > a.tau))
        return;
    const float f = static_cast<float>(it.power == 0.5 ? sqrt(a.tau / top) : pow(a.tau / top, it.power));
    const WeightView& wv = it.w;
    each_piece<kUnroll>(wv.rows, wv.cols, part, it.rounds, [&](const Spot(&p)[kUnroll], int n) {
        f32x4_t x[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
            x[u] = load4<NT>(static_cast<const float*>(wv.master.data) + z * wv.master.bs + p[u].row * wv.master.rs +
                                 p[u].col,
                             p[u].n);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (u >= n)
                break;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[u][e] = x[u][e] * f;
            store4<NT>(static_cast<float*>(wv.master.data) + z * wv.master.bs + p[u].row * wv.master.rs + p[u].col, x[u],
                       p[u].n);
            if (wv.param_dtype == HPO_PARAM_BF16)
                store_weight<HPO_PARAM_BF16, NT>(wv, z, p[u], x[u]);
            else if (wv.param_dtype == HPO_WEIGHT_MX8)
                store_weight<HPO_WEIGHT_MX8, NT>(wv, z, p[u], x[u]);
        }
    });
}

template <typename... Args>
hipError_t launch(void (*kernel)(Args...), dim3 grid, int block, hipStream_t stream, Args... args)
{
    void* argv[] = {static_cast<void*>(&args)...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(block), argv, 0, stream);
}

template <typename OT, bool FOLDED, int U, bool NT>
hipError_t launch_apply(const RmsArgs& a, dim3 grid, hipStream_t stream)
{
    if (a.w.param_dtype == HPO_PARAM_BF16)
        return launch(k_rms_apply<OT, HPO_PARAM_BF16, FOLDED, U, NT>, grid, kRowThreads, stream, a);
    if (a.w.param_dtype == HPO_WEIGHT_MX8)
        return launch(k_rms_apply<OT, HPO_WEIGHT_MX8, FOLDED, U, NT>, grid, kRowThreads, stream, a);
    return launch(k_rms_apply<OT, HPO_PARAM_FP32, FOLDED, U, NT>, grid, kRowThreads, stream, a);
}

/* Workgroups that cover one matrix of a stack, `run` pieces per wavefront. */
int64_t blocks_of(const WeightView& w, int64_t run)
{
    const int64_t pieces = (w.cols + kPiece - 1) / kPiece;
    return (w.rows * pieces + kRowWaves * run - 1) / (kRowWaves * run);
}

/* Bytes of master and model weight per element (8-bit scales left out). */
int64_t bytes_of(const WeightView& w)
{
    return w.param_dtype == HPO_PARAM_FP32 ? 4 : (w.param_dtype == HPO_PARAM_BF16 ? 6 : 5);
}

constexpr int64_t kStreamBytes = int64_t{64} << 20;

template <typename OT>
hipError_t rms_update(RmsArgs a, hipStream_t stream)
{
    const int64_t rows = a.w.rows;
    /* few long rows: a workgroup each, or most of the chip would wait for single wavefronts */
    const bool wg = a.batch * rows <= 2048 && a.w.cols > 4096;
    a.parts = wg ? rows : (rows + kStatRows - 1) / kStatRows;
    const dim3 sgrid(static_cast<uint32_t>(a.parts), static_cast<uint32_t>(a.batch));
    hipError_t e = wg ? launch(k_long_row_stats<OT>, sgrid, kRowThreads, stream, a)
                      : launch(k_row_stats<OT>, sgrid, 64 * kStatRows, stream, a);
    if (e != hipSuccess)
        return e;
    /* Little to do: one piece a wavefront, as many workgroups as there are; much: runs of eight,
     * two in flight (one, four and eight in flight are 2 to 10 % slower). */
    const bool small = a.batch * blocks_of(a.w, 1) <= 2048;
    constexpr int32_t kRounds = 4;
    a.rounds = small ? 1 : kRounds;
    const dim3 grid(static_cast<uint32_t>(blocks_of(a.w, small ? 1 : kRounds * kUnroll)), static_cast<uint32_t>(a.batch));
    /* Larger masters and weights go around the caches, which leaves these to O between the two passes:
     * 4096 x 14336 takes 135 us so and 165 us through them; with other states in between (as in a step
     * over a whole model) 16 x 1024 x 2048 takes 77 and 90 us, half of it 44 and 49, a quarter 26 and
     * 25; a lone state that stays in the cache loses 2 %. */
    const bool nt = a.batch * rows * a.w.cols * bytes_of(a.w) > kStreamBytes;
    /* every workgroup sums the parts itself (and one launch is saved) unless they are very many */
    constexpr int64_t kFoldParts = 1024;
    const bool fold = a.parts > kFoldParts;
    if (fold) {
        e = launch(k_row_fold, dim3(static_cast<uint32_t>(a.batch)), kRowThreads, stream, a);
        if (e != hipSuccess)
            return e;
    }
    if (small)
        return fold ? launch_apply<OT, true, 1, false>(a, grid, stream) : launch_apply<OT, false, 1, false>(a, grid, stream);
    if (nt)
        return fold ? launch_apply<OT, true, kUnroll, true>(a, grid, stream)
                    : launch_apply<OT, false, kUnroll, true>(a, grid, stream);
    return fold ? launch_apply<OT, true, kUnroll, false>(a, grid, stream)
                : launch_apply<OT, false, kUnroll, false>(a, grid, stream);
}

}  // namespace

hipError_t launch_rms_update(const RmsArgs& a, hipStream_t stream)
{
    return a.o_fp32 ? rms_update<float>(a, stream) : rms_update<uint16_t>(a, stream);
}

hipError_t launch_qk_clip(ClipArgs& a, hipStream_t stream)
{
    int64_t total = 0, bytes = 0;
    for (int32_t k = 0; k < a.n; ++k) {
        const ClipItem& it = a.item[k];
        total += it.heads * blocks_of(it.w, kUnroll);
        bytes += it.heads * it.w.rows * it.w.cols * bytes_of(it.w);
    }
    /* most workgroups of a wide layer only find that their head is not clipped: above 4096 of them,
     * longer runs */
    const int32_t rounds = static_cast<int32_t>(std::min<int64_t>(4, (total + 4095) / 4096));
    total = 0;
    for (int32_t k = 0; k < a.n; ++k) {
        a.item[k].rounds = rounds;
        a.item[k].blocks = static_cast<int32_t>(blocks_of(a.item[k].w, kUnroll * rounds));
        a.item[k].first_block = total;
        total += static_cast<int64_t>(a.item[k].heads) * a.item[k].blocks;
    }
    if (total == 0)
        return hipSuccess;
    const dim3 grid(static_cast<uint32_t>(total));
    return bytes > kStreamBytes ? launch(k_qk_clip<true>, grid, kRowThreads, stream, a)
                                : launch(k_qk_clip<false>, grid, kRowThreads, stream, a);
}

}  // namespace hpo
