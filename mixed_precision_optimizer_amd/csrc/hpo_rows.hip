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
 * Floating point: built with -ffp-contract=off; every elementwise operation
 * rounds on its own, in the order written.
 */
#include <hip/hip_runtime.h>

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
constexpr int kPiecesPerWave = 8;  /* consecutive pieces of one wavefront */
constexpr int kMxBlock = 32;

/* ---------------------------------------------------------------------- */
/* four consecutive elements of a row                                      */
/* ---------------------------------------------------------------------- */
/* n of them are in the row (n <= 0: none); the others read as 0 and are not written. */
__device__ __forceinline__ f32x4_t load4(const float* p, int n)
{
    f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n >= 4)
        return *reinterpret_cast<const f32x4_any*>(p);
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

__device__ __forceinline__ void store4(float* p, f32x4_t x, int n)
{
    if (n >= 4) {
        *reinterpret_cast<f32x4_any*>(p) = x;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < n)
            p[e] = x[e];
}

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
        *reinterpret_cast<u32x2_any*>(p) = t;
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
        *reinterpret_cast<u32_any*>(p) = v;
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

template <int PT>
__device__ __forceinline__ void store_weight(const WeightView& w, int64_t z, const Spot& s, f32x4_t x)
{
    if constexpr (PT == HPO_PARAM_BF16) {
        store_bf16(static_cast<uint16_t*>(w.param.data) + z * w.param.bs + s.row * w.param.rs + s.col, x, s.n);
    } else if constexpr (PT == HPO_WEIGHT_MX8) {
        const int64_t nb = (w.cols + kMxBlock - 1) / kMxBlock;
        store_mx8(static_cast<uint8_t*>(w.param.data) + z * w.param.bs + s.row * w.param.rs + s.col,
                  w.scales + (z * w.rows + s.row) * nb + s.col / kMxBlock, x, s.n);
    }
}

__device__ __forceinline__ bool skipped(const int32_t* d_found) { return d_found != nullptr && *d_found != 0; }

/* ---------------------------------------------------------------------- */
/* hpo_rms_update                                                          */
/* ---------------------------------------------------------------------- */
/* Mean square of each row, the running v, r and the row's part of N^2.
 * WG: a workgroup per row (long rows), else a wavefront per row. */
template <typename OT, bool WG>
__global__ __launch_bounds__(kRowThreads) void k_row_stats(RmsArgs a)
{
    if (skipped(a.d_found))
        return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t rows = a.w.rows, cols = a.w.cols;
    const int64_t idx = WG ? static_cast<int64_t>(blockIdx.x) : static_cast<int64_t>(blockIdx.x) * kRowWaves + wave;
    if (idx >= a.batch * rows)
        return;   /* whole wavefronts; no barrier follows in that form */
    const int64_t z = idx / rows, i = idx % rows;
    const OT* __restrict__ o = static_cast<const OT*>(a.O.data) + z * a.O.bs + i * a.O.rs;
    float acc = 0.0f;
    const int64_t step = WG ? 4 * kRowThreads : 4 * 64;
#pragma unroll 4
    for (int64_t c = 4 * (WG ? static_cast<int>(threadIdx.x) : lane); c < cols; c += step) {
        const int64_t left = cols - c;
        const f32x4_t x = load4(o + c, left > 4 ? 4 : static_cast<int>(left));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            acc += x[e] * x[e];
    }
    double tot = static_cast<double>(acc);
    if constexpr (WG) {
        tot = block_sum<kRowThreads>(tot);
    } else {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1)
            tot += __shfl_down(tot, off, 64);
    }
    if ((WG ? static_cast<int>(threadIdx.x) : lane) == 0) {
        const double ms = tot / static_cast<double>(cols);
        float v = static_cast<float>(ms);
        if (a.v != nullptr) {
            if (a.beta2 > 0.0)
                v = static_cast<float>(a.beta2 * static_cast<double>(a.v[idx]) + (1.0 - a.beta2) * ms);
            a.v[idx] = v;
        }
        const double den = sqrt(static_cast<double>(v)) + a.eps;
        const double r = den == 0.0 ? 0.0 : 1.0 / den;
        a.r[idx] = static_cast<float>(r);
        a.q[idx] = tot * r * r;
    }
}

/* N^2 of each matrix: one workgroup, fixed order. */
__global__ __launch_bounds__(kRowThreads) void k_row_fold(RmsArgs a)
{
    if (skipped(a.d_found))
        return;
    const double* q = a.q + static_cast<int64_t>(blockIdx.x) * a.w.rows;
    double acc = 0.0;
    for (int64_t i = threadIdx.x; i < a.w.rows; i += kRowThreads)
        acc += q[i];
    const double tot = block_sum<kRowThreads>(acc);
    if (threadIdx.x == 0)
        a.norm2[blockIdx.x] = tot;
}

/* W <- W keep - (s r_i) O_i, and the model weight.  FOLDED: N^2 was summed by
 * k_row_fold; else every workgroup sums the matrix's rows itself. */
template <typename OT, int PT, bool FOLDED>
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
        for (int64_t i = threadIdx.x; i < rows; i += kRowThreads)
            acc += a.q[z * rows + i];
        acc = block_sum<kRowThreads>(acc);
        if (threadIdx.x == 0)
            total = acc;
        __syncthreads();
        n2 = total;
    }
    const double s = n2 > 0.0 ? a.gain / sqrt(n2) : 0.0;
    const int64_t pieces = (cols + kPiece - 1) / kPiece;
    const int wave = threadIdx.x >> 6;
    int64_t t = (static_cast<int64_t>(blockIdx.x) * kRowWaves + wave) * kPiecesPerWave;
    int64_t row = t / pieces, piece = t % pieces;
    for (int k = 0; k < kPiecesPerWave && row < rows; ++k) {
        const Spot p = spot_of(row, piece, cols);
        const float c = static_cast<float>(s * static_cast<double>(a.r[z * rows + row]));
        const f32x4_t o = load4(static_cast<const OT*>(a.O.data) + z * a.O.bs + row * a.O.rs + p.col, p.n);
        float* w = static_cast<float*>(a.w.master.data) + z * a.w.master.bs + row * a.w.master.rs + p.col;
        f32x4_t x = load4(w, p.n);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float kept = x[e] * a.keep;
            const float u = c * o[e];
            x[e] = kept - u;
        }
        store4(w, x, p.n);
        store_weight<PT>(a.w, z, p, x);
        if (++piece == pieces) {
            piece = 0;
            ++row;
        }
    }
}

/* ---------------------------------------------------------------------- */
/* hpo_qk_clip                                                             */
/* ---------------------------------------------------------------------- */
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
    const int64_t rows = wv.rows, cols = wv.cols, pieces = (cols + kPiece - 1) / kPiece;
    const int wave = threadIdx.x >> 6;
    int64_t t = (part * kRowWaves + wave) * kPiecesPerWave;
    int64_t row = t / pieces, piece = t % pieces;
    for (int q = 0; q < kPiecesPerWave && row < rows; ++q) {
        const Spot p = spot_of(row, piece, cols);
        float* w = static_cast<float*>(wv.master.data) + z * wv.master.bs + row * wv.master.rs + p.col;
        f32x4_t x = load4(w, p.n);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            x[e] = x[e] * f;
        store4(w, x, p.n);
        if (wv.param_dtype == HPO_PARAM_BF16)
            store_weight<HPO_PARAM_BF16>(wv, z, p, x);
        else if (wv.param_dtype == HPO_WEIGHT_MX8)
            store_weight<HPO_WEIGHT_MX8>(wv, z, p, x);
        if (++piece == pieces) {
            piece = 0;
            ++row;
        }
    }
}

template <typename... Args>
hipError_t launch(void (*kernel)(Args...), dim3 grid, hipStream_t stream, Args... args)
{
    void* argv[] = {static_cast<void*>(&args)...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(kRowThreads), argv, 0, stream);
}

template <typename OT, bool FOLDED>
hipError_t launch_apply(const RmsArgs& a, dim3 grid, hipStream_t stream)
{
    if (a.w.param_dtype == HPO_PARAM_BF16)
        return launch(k_rms_apply<OT, HPO_PARAM_BF16, FOLDED>, grid, stream, a);
    if (a.w.param_dtype == HPO_WEIGHT_MX8)
        return launch(k_rms_apply<OT, HPO_WEIGHT_MX8, FOLDED>, grid, stream, a);
    return launch(k_rms_apply<OT, HPO_PARAM_FP32, FOLDED>, grid, stream, a);
}

/* Workgroups that cover one matrix of a stack. */
int64_t blocks_of(const WeightView& w)
{
    const int64_t pieces = (w.cols + kPiece - 1) / kPiece;
    return (w.rows * pieces + kRowWaves * kPiecesPerWave - 1) / (kRowWaves * kPiecesPerWave);
}

template <typename OT>
hipError_t rms_update(const RmsArgs& a, hipStream_t stream)
{
    const int64_t total = a.batch * a.w.rows;
    const bool wg = a.w.cols > 2048;
    const int64_t blocks = wg ? total : (total + kRowWaves - 1) / kRowWaves;
    hipError_t e = wg ? launch(k_row_stats<OT, true>, dim3(static_cast<uint32_t>(blocks)), stream, a)
                      : launch(k_row_stats<OT, false>, dim3(static_cast<uint32_t>(blocks)), stream, a);
    if (e != hipSuccess)
        return e;
    const dim3 grid(static_cast<uint32_t>(blocks_of(a.w)), static_cast<uint32_t>(a.batch));
    /* Few rows: every workgroup sums them itself and one launch is saved; many rows are summed once. */
    constexpr int64_t kFoldRows = 1024;
    if (a.w.rows <= kFoldRows)
        return launch_apply<OT, false>(a, grid, stream);
    e = launch(k_row_fold, dim3(static_cast<uint32_t>(a.batch)), stream, a);
    if (e != hipSuccess)
        return e;
    return launch_apply<OT, true>(a, grid, stream);
}

}  // namespace

hipError_t launch_rms_update(const RmsArgs& a, hipStream_t stream)
{
    return a.o_fp32 ? rms_update<float>(a, stream) : rms_update<uint16_t>(a, stream);
}

hipError_t launch_qk_clip(ClipArgs& a, hipStream_t stream)
{
    int64_t total = 0;
    for (int32_t k = 0; k < a.n; ++k) {
        a.item[k].blocks = static_cast<int32_t>(blocks_of(a.item[k].w));
        a.item[k].first_block = total;
        total += static_cast<int64_t>(a.item[k].heads) * a.item[k].blocks;
    }
    if (total == 0)
        return hipSuccess;
    return launch(k_qk_clip, dim3(static_cast<uint32_t>(total)), stream, a);
}

}  // namespace hpo
