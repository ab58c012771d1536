/*
 * hpo_qk.hip -- gfx950 kernels of hpo_qk_max_logits: the largest attention
 * logit of each head, S_h = max over the seen pairs of scale * (q . k).
 *
 * Source: [OPT-INFRA] "02 · Optimizer：算法与 infra" (llm-infra-atlas,
 * train/02_optimizer), §6: the S_max^h that QK-clip compares with its threshold.
 *
 * The logits are a matrix product of which only the maximum leaves the chip,
 * so the work is bound by the matrix cores.  A workgroup of four wavefronts
 * takes 256 queries of one head (64 per wavefront, their fragments in
 * registers for the whole pass) against key tiles of 64, staged in LDS in two
 * buffers; a key tile is the MFMA's row operand, so a lane's 16 results of one
 * 32 x 32 block are keys of one query, and its limits (causal, window,
 * lengths) are two numbers.  Tiles that every query of the wavefront sees whole skip
 * the mask, tiles none sees skip the products.  The maximum needs no state per query:
 * each lane keeps one number, folded with v_maximum3 (two logits an
 * instruction, NaN stays NaN).
 *
 * Measured: 8192 causal tokens, 32 heads over 8, dim 128, bf16: 206 to 216 us from box to box, 1.27
 * to 1.33 PFLOP/s of the seen pairs (a large library product reaches 1.20 here); the matrix cores are busy 65 % of the
 * cycles at the 1.85 GHz that this load leaves, LDS free of bank conflicts.  4096 tokens, 8 heads:
 * dim 64 18 us, 128 24 us, 192 32 us, 256 39 us.  Dims that are not multiples of 16 pass through
 * registers and are bound by that (64-bit shifts beside the queries' fragments): 57 30 us,
 * 72 36 us, 136 67 us, 200 98 us; over 192 they also spill (165 registers).  One or few queries: a head's
 * workgroups each stage the keys of its group for one row in 64, so 4 x 1 on 9000 keys, 32 heads
 * over 8, read 74 MB of keys in 38 us (16 at the rate of a large copy).  Short sequences
 * are bound by the two launches (about 9 us with the binding).
 */
#include <hip/hip_runtime.h>

#include <type_traits>

#include "hpo_device.h"
#include "hpo_stack_impl.h"

namespace hpo {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
/* eight elements at any element's address (one instruction in global memory) */
typedef u32x4_t u32x4_any __attribute__((aligned(2)));

constexpr int kQkThreads = 256;
constexpr int kQkWaves = 4;
constexpr int kWaveRows = 64;                      /* queries of a wavefront */
constexpr int kTileQ = kWaveRows * kQkWaves;       /* queries of a workgroup */
constexpr int kTileK = 64;                         /* keys of a stage */

template <bool FP16>
__device__ __forceinline__ f32x16_t mfma(u32x4_t a, u32x4_t b, f32x16_t c)
{
    if constexpr (FP16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c,
                                                      0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                       __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

/* Byte offset of 16-byte piece p of LDS row r (rows of DP elements).  The
 * pieces of a row are permuted by an XOR of the row, so that the 16 rows a
 * fragment read serves at a time lie in distinct banks. */
template <int DP>
__device__ __forceinline__ int swizzle(int r)
{
    if constexpr (DP % 128 == 0)
        return r & 15;
    else
        return (r & 7) ^ ((r >> 3) & 1);
}

template <int DP>
__device__ __forceinline__ int piece_at(int r, int p)
{
    return r * (DP * 2) + ((p ^ swizzle<DP>(r)) << 4);
}

/* 64 x 16 bytes from a buffer straight into LDS: lane l's lands at dst + 16 l. */
__device__ __forceinline__ void buffer_load_lds16(__amdgpu_buffer_rsrc_t rs, char* dst, int voff)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)dst, 16, voff, 0, 0, 0);
}

/* Eight elements of a row of `dim`, from element d on; 0 behind its end.  Rows of
 * eight and more take one access, moved back to end with the row where it would pass
 * it, and a shift. */
__device__ __forceinline__ u32x4_t load8(const uint16_t* row, int d, int dim)
{
    if (dim < 8) {
        u32x4_t v = {0, 0, 0, 0};
        for (int e = 0; e < dim - d; ++e)
            v[e >> 1] |= static_cast<uint32_t>(row[d + e]) << (16 * (e & 1));
        return v;
    }
    const int start = d < dim - 8 ? d : dim - 8;
    const u32x4_t x = *reinterpret_cast<const u32x4_any*>(row + start);
    const int by = (d - start) * 16;   /* bits; 128 and more: nothing is left */
    uint64_t lo = x[0] | (static_cast<uint64_t>(x[1]) << 32), hi = x[2] | (static_cast<uint64_t>(x[3]) << 32);
    if (by >= 64) {
        lo = by < 128 ? hi >> (by - 64) : 0;
        hi = 0;
    } else if (by > 0) {
        lo = (lo >> by) | (hi << (64 - by));
        hi >>= by;
    }
    return u32x4_t{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                   static_cast<uint32_t>(hi >> 32)};
}

__device__ __forceinline__ float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }

/* Work of one workgroup in dispatch order.  Workgroups go to the 8 XCDs
 * round-robin: each XCD gets one contiguous run, so the heads and query tiles
 * that read one key head meet in its L2. */
__device__ __forceinline__ int64_t xcd_run(int64_t b, int64_t n)
{
    constexpr int64_t kXcd = 8;
    const int64_t x = b % kXcd, k = b / kXcd, q = n / kXcd, r = n % kXcd;
    return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + k;
}

/* One sequence: its first token and its length, cut to what is there. */
__device__ __forceinline__ void extent(const int32_t* cu, const int32_t* len, int b, int seq, int& start, int& n)
{
    start = 0;
    n = seq;
    if (cu != nullptr) {
        const int lo = cu[b], hi = cu[b + 1];
        start = lo < 0 ? 0 : (lo > seq ? seq : lo);
        const int end = hi < start ? start : (hi > seq ? seq : hi);
        n = end - start;
    } else if (len != nullptr) {
        const int l = len[b];
        n = l < 0 ? 0 : (l > seq ? seq : l);
    }
}

/* How key tiles come into LDS (rows of DP elements there):
 *   kWhole    dim == DP, every row 16-byte aligned: straight from global memory;
 *   kSlices16 dim a multiple of 16, aligned: the same, the slices behind dim hold copies of its
 *             last piece and are not multiplied;
 *   kAny      through registers, zero-filled to whole slices. */
enum Mode : int { kWhole = 0, kSlices16 = 1, kAny = 2 };

template <bool FP16, int DP, int MODE>
__global__ __launch_bounds__(kQkThreads, 2) void k_qk_max(QkArgs a)
{
    constexpr int kSlices = DP / 16;
    constexpr bool DIRECT = MODE != kAny;
    constexpr int kPieces = DP / 8;
    constexpr int kStageBytes = kTileK * DP * 2;
    constexpr int kChunks = kStageBytes / 1024 / kQkWaves;   /* 1 KB loads of a wavefront per stage */
    __shared__ __attribute__((aligned(16))) char lds[2 * kStageBytes];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int per = a.heads / a.kv_heads;
    int64_t t = xcd_run(blockIdx.x, gridDim.x);
    const int split = static_cast<int>(t % a.splits);
    t /= a.splits;
    const int hg = static_cast<int>(t % per);
    t /= per;
    const int tile0 = a.q_tiles - 1 - static_cast<int>(t % a.q_tiles);   /* the longest causal rows first */
    t /= a.q_tiles;
    const int hk = static_cast<int>(t % a.kv_heads), b = static_cast<int>(t / a.kv_heads);
    const int h = hk * per + hg;
    int q_start, len_q, k_start, len_k;
    extent(a.cu_q, a.len_q, b, a.seq_q, q_start, len_q);
    extent(a.cu_k, a.len_k, b, a.seq_k, k_start, len_k);
    if (len_q == 0 || len_k == 0)
        return;
    const int off = len_k - len_q;
    const uint16_t* __restrict__ Q = a.q + (a.cu_q ? 0 : b * a.qsb) + q_start * a.qst + h * a.qsh;
    const uint16_t* __restrict__ K = a.k + (a.cu_k ? 0 : b * a.ksb) + k_start * a.kst + hk * a.ksh;
    const int nks = MODE == kWhole ? kSlices : (a.dim + 15) / 16;   /* slices that are not all padding */
    const int last_piece = a.dim / 8 - 1;
    const int frow = lane & 31, fhalf = lane >> 5;
    float best = -INFINITY;
    /* one lane's pieces of a stage: byte offsets from its first key */
    int voff[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
        const int at = (wave * kChunks + c) * 64 + lane;
        const int r = at / kPieces;
        int p = (at % kPieces) ^ swizzle<DP>(r);
        if constexpr (MODE == kSlices16)
            p = p < last_piece ? p : last_piece;
        voff[c] = (r * static_cast<int>(a.kst) + p * 8) * 2;
    }

    for (int qt = tile0; static_cast<int64_t>(qt) * kTileQ < len_q; qt += a.q_tiles) {
        const int q0 = qt * kTileQ;
        const int q1 = q0 + kTileQ < len_q ? q0 + kTileQ : len_q;
        /* keys that some query of the tile sees */
        int lo = 0, hi = len_k - 1;
        if (a.causal) {
            hi = q1 - 1 + off < hi ? q1 - 1 + off : hi;
            if (a.window >= 0 && q0 + off - a.window > 0)
                lo = q0 + off - a.window;
        }
        if (hi < lo)
            continue;
        const int first = lo / kTileK, count = hi / kTileK - first + 1;
        const int t0 = first + static_cast<int>(static_cast<int64_t>(count) * split / a.splits);
        const int t1 = first + static_cast<int>(static_cast<int64_t>(count) * (split + 1) / a.splits);
        if (t0 >= t1)
            continue;

        /* this wavefront's queries: fragments and each lane's key limits */
        const int w0 = q0 + wave * kWaveRows;
        u32x4_t fq[2][kSlices];
        int klo[2], khi[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = w0 + 32 * j + frow;
            const uint16_t* row = Q + static_cast<int64_t>(i < len_q ? i : len_q - 1) * a.qst;
#pragma unroll
            for (int s = 0; s < kSlices; ++s) {
                if constexpr (MODE == kWhole)
                    fq[j][s] = *reinterpret_cast<const u32x4_t*>(row + 16 * s + 8 * fhalf);
                else if constexpr (MODE == kSlices16)
                    fq[j][s] = s < nks ? *reinterpret_cast<const u32x4_t*>(row + 16 * s + 8 * fhalf) : u32x4_t{0, 0, 0, 0};
                else if (16 * s + 16 <= a.dim)
                    fq[j][s] = *reinterpret_cast<const u32x4_any*>(row + 16 * s + 8 * fhalf);
                else if (s < nks)
                    fq[j][s] = load8(row, 16 * s + 8 * fhalf, a.dim);
                else
                    fq[j][s] = u32x4_t{0, 0, 0, 0};
            }
            khi[j] = len_k - 1;
            klo[j] = 0;
            if (a.causal) {
                khi[j] = i + off < khi[j] ? i + off : khi[j];
                if (a.window >= 0 && i + off - a.window > 0)
                    klo[j] = i + off - a.window;
            }
            if (i >= len_q)
                khi[j] = -1;
        }
        /* the wavefront's limits: seen by some query, seen by every query */
        const int wlast = w0 + kWaveRows - 1 < len_q ? w0 + kWaveRows - 1 : len_q - 1;
        int some_hi = w0 < len_q ? len_k - 1 : -1, every_hi = w0 + kWaveRows <= len_q ? len_k - 1 : -1;
        int some_lo = 0, every_lo = 0;
        if (a.causal) {
            some_hi = wlast + off < some_hi ? wlast + off : some_hi;
            every_hi = w0 + off < every_hi ? w0 + off : every_hi;
            if (a.window >= 0) {
                some_lo = w0 + off - a.window > 0 ? w0 + off - a.window : 0;
                every_lo = wlast + off - a.window > 0 ? wlast + off - a.window : 0;
            }
        }

        auto stage = [&](int kt, int buf) {
            const int k0 = kt * kTileK;
            const int left = len_k - k0;   /* >= 1 */
            const uint16_t* base = K + static_cast<int64_t>(k0) * a.kst;
            char* dst = lds + buf * kStageBytes;
            if constexpr (DIRECT) {
                /* rows behind the end are behind the descriptor's too: not read, and masked */
                const int rows = left < kTileK ? left : kTileK;
                const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
                    const_cast<uint16_t*>(base), 0, ((rows - 1) * static_cast<int>(a.kst) + a.dim) * 2, 0x00020000);
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    buffer_load_lds16(rs, dst + (wave * kChunks + c) * 1024, voff[c]);
            } else {
                /* two pieces at a time: all of them in flight spill beside the queries' registers */
#pragma unroll 2
                for (int c = 0; c < kChunks; ++c) {
                    const int at = c * kQkThreads + tid;
                    const int r = at / kPieces, p = at % kPieces;
                    const int rr = r < left ? r : left - 1;
                    const u32x4_t v = load8(base + static_cast<int64_t>(rr) * a.kst, p * 8, a.dim);
                    *reinterpret_cast<u32x4_t*>(dst + piece_at<DP>(r, p)) = v;
                }
            }
        };

        auto compute = [&](int kt, int buf) {
            const int k0 = kt * kTileK;
            if (k0 > some_hi || k0 + kTileK - 1 < some_lo)
                return;
            const char* src = lds + buf * kStageBytes;
            f32x16_t acc[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = f32x16_t{};
#pragma unroll
            for (int s = 0; s < kSlices; ++s) {
                if (MODE == kWhole || s < nks) {
                    u32x4_t fk[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        fk[i] = *reinterpret_cast<const u32x4_t*>(src + piece_at<DP>(32 * i + frow, 2 * s + fhalf));
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            acc[i][j] = mfma<FP16>(fk[i], fq[j][s], acc[i][j]);
                }
            }
            if (k0 >= every_lo && k0 + kTileK - 1 <= every_hi) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            best = maximum(best, acc[i][j][r]);
            } else {
                /* acc[i][j][r]: key k0 + 4 (lane / 32) + 32 i + 8 (r / 4) + r % 4, query of this lane;
                 * a tile at one of the two edges is compared with that one's limit only */
                auto masked = [&](auto lo_side, auto hi_side) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int l = klo[j] - k0 - 4 * fhalf, u = khi[j] - k0 - 4 * fhalf;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int r = 0; r < 16; ++r) {
                                const int key = 32 * i + 8 * (r >> 2) + (r & 3);
                                const bool seen = (!lo_side.value || key >= l) && (!hi_side.value || key <= u);
                                best = maximum(best, seen ? acc[i][j][r] : -INFINITY);
                            }
                    }
                };
                if (k0 >= every_lo)
                    masked(std::false_type{}, std::true_type{});
                else if (k0 + kTileK - 1 <= every_hi)
                    masked(std::true_type{}, std::false_type{});
                else
                    masked(std::true_type{}, std::true_type{});
            }
        };

        __syncthreads();   /* the buffers of the previous query tile */
        stage(t0, 0);
        for (int kt = t0; kt < t1; ++kt) {
            const int buf = (kt - t0) & 1;
            /* Behind the barrier every wavefront's part of stage kt is in LDS, and the other buffer is
             * no longer read.  The wait for this wavefront's own loads and LDS accesses is written
             * out: nothing else makes the loads into LDS land before it.  (Three and four buffers with
             * loads further ahead are no faster: 4096 tokens, dim 128, 23.0 and 23.6 us, two 22.4.) */
            if constexpr (DIRECT) {
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_waitcnt(0x0070);   /* gfx9 encoding: vmcnt(0) lgkmcnt(0) */
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            } else {
                __syncthreads();
            }
            if (kt + 1 < t1)
                stage(kt + 1, buf ^ 1);
            if constexpr (DIRECT)
                __builtin_amdgcn_sched_barrier(0);
            compute(kt, buf);
        }
    }

#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        best = maximum(best, __shfl_xor(best, d, 64));
    /* In the stages' array: beside a second LDS variable the compiler waits for all loads in flight
     * before a stage's first fragment read, and nothing overlaps (4096 tokens, dim 128: 26.7 us, so
     * 22.4). */
    float* wmax = reinterpret_cast<float*>(lds);
    __syncthreads();
    if (lane == 0)
        wmax[wave] = best;
    __syncthreads();
    if (tid == 0) {
        best = maximum(maximum(wmax[0], wmax[1]), maximum(wmax[2], wmax[3]));
        /* rounding is monotone: the largest product times scale is the largest logit.  Adding 0
         * turns -0 into 0.  As bits, non-negative values (and the positive NaN above
         * them) order as signed integers, negative ones fall as unsigned grow; each atomic
         * only ever raises the value, so their order does not matter.  A NaN of the caller's with
         * its sign set lies below everything: whoever replaces it puts a NaN back. */
        const float v = best * a.scale + 0.0f;
        float* out = a.out + h;
        uint32_t before = 0;
        if (v != v)
            atomicMax(reinterpret_cast<int*>(out), 0x7fc00000);
        else if (v >= 0.0f)
            before = static_cast<uint32_t>(atomicMax(reinterpret_cast<int*>(out), __float_as_int(v)));
        else if (v > -INFINITY)
            before = atomicMin(reinterpret_cast<unsigned int*>(out), __float_as_uint(v));
        if (a.accumulate && before > 0xff800000u)
            atomicMax(reinterpret_cast<int*>(out), 0x7fc00000);
    }
}

__global__ void k_fill(float* out, int n, float v)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < n)
        out[i] = v;
}

template <typename... Args>
hipError_t launch(void (*kernel)(Args...), dim3 grid, int block, hipStream_t stream, Args... args)
{
    void* argv[] = {static_cast<void*>(&args)...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(block), argv, 0, stream);
}

template <bool FP16, int DP>
hipError_t launch_dim(const QkArgs& a, bool aligned, uint32_t grid, hipStream_t stream)
{
    if (aligned && a.dim == DP)
        return launch(k_qk_max<FP16, DP, kWhole>, dim3(grid), kQkThreads, stream, a);
    if (aligned && a.dim % 16 == 0)
        return launch(k_qk_max<FP16, DP, kSlices16>, dim3(grid), kQkThreads, stream, a);
    return launch(k_qk_max<FP16, DP, kAny>, dim3(grid), kQkThreads, stream, a);
}

template <bool FP16>
hipError_t launch_type(const QkArgs& a, bool aligned, uint32_t grid, hipStream_t stream)
{
    if (a.dim <= 64)
        return launch_dim<FP16, 64>(a, aligned, grid, stream);
    if (a.dim <= 128)
        return launch_dim<FP16, 128>(a, aligned, grid, stream);
    if (a.dim <= 192)
        return launch_dim<FP16, 192>(a, aligned, grid, stream);
    return launch_dim<FP16, 256>(a, aligned, grid, stream);
}

}  // namespace

hipError_t launch_qk_max(QkArgs a, bool fp16, bool aligned, hipStream_t stream)
{
    if (!a.accumulate) {
        hipError_t e = launch(k_fill, dim3((a.heads + 255) / 256), 256, stream, a.out, static_cast<int>(a.heads), -INFINITY);
        if (e != hipSuccess)
            return e;
    }
    if (a.batch == 0 || a.seq_q == 0 || a.seq_k == 0)
        return hipSuccess;
    a.q_tiles = (a.max_q + kTileQ - 1) / kTileQ;
    const int64_t tiles = static_cast<int64_t>(a.batch) * a.heads * a.q_tiles;
    /* Few query tiles: the keys are split until the chip's 512 resident workgroups have work, with
     * four stages each at the least.  Up to 64 queries keep one wavefront of a workgroup busy, and dims
     * up to 128 leave room for a third one: 768.  4 x 1 query on 9000 keys, 32 heads over 8, dim 128:
     * 41 us, with 512 53, with 1024 55; over 14 shapes of 1 to 64 queries, 1 to 32 sequences, 2000 to
     * 100000 keys, dims 40 to 128 it takes 0.55 to 0.92 of the time with 512 on ten, the same on three,
     * and 1.14 on 64 queries of dim 64 (16 and 18 us).  Longer queries lose 3 to 12 % with it. */
    const int64_t wgs = a.max_q <= kWaveRows && a.dim <= 128 ? 768 : 512;
    const int64_t want = (wgs + tiles - 1) / tiles, most = (a.max_k + 4 * kTileK - 1) / (4 * kTileK);
    a.splits = static_cast<int32_t>(want < most ? want : most);
    if (a.splits < 1)
        a.splits = 1;
    const uint32_t grid = static_cast<uint32_t>(tiles * a.splits);
    return fp16 ? launch_type<true>(a, aligned, grid, stream) : launch_type<false>(a, aligned, grid, stream);
}

}  // namespace hpo
