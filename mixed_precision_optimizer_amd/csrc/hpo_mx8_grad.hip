/*
 * hpo_mx8_grad.hip -- gfx950 kernels of a linear layer's gradients beside 8-bit
 * operands: dX = dY W^ (hpo_mx8_dgrad) and G += scale * dY^T X^ (hpo_mx8_wgrad).
 *
 * dY stays in 16 bits, and a product of 16 and 8 bits does not exist: B (W or X) becomes 16 bits on its way
 * from registers into LDS, scaled by its blocks (exact in bf16, one rounding in fp16), in the kernel, so that HBM only
 * sees 8.  Both sums run over B's rows (dgrad over the outputs, wgrad over the tokens), along which nothing is
 * contiguous: the fragments come from LDS by transposing reads, for wgrad dY's as well.  The scale blocks lie along
 * the other side, so no scale could stay outside of the sum.
 *
 * Bound by the matrix cores (busy 55 % of dX's time, 46 % of G's) and the clock that the power leaves them (1.7 to 2.2
 * GHz under counters), wavefronts waiting for a third of the time.  dX of 8192 x 4096 from 14336 outputs takes 810 to
 * 867 us from box to box (1.11 to 1.19 PFLOP/s); G of 14336 x 4096 over 8192 tokens 908 to 961 (1.00 to 1.06; 3.5 rounds of
 * tiles on 256 CUs in the time of four); call after call 834 and 936, in the first ten on a card that was idle 920 to 1150 and
 * 1060 to 1330, while its clock swings.  A bf16 product of the library alone, without the widening, takes 729 and 971 us.
 * Eight wavefronts share a tile of 256, so that the widening of one runs beside the products of another; four of 128 x 128
 * each, as in hpo_mx8_linear, took 1568 and 1824 us with loads that the compiler waits for (see load_lds16), when eight took
 * 1028 and 1178.
 */
#include <hip/hip_runtime.h>

#include <type_traits>

#include "hpo_product_device.h"

namespace hpo {
namespace {

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

__device__ __forceinline__ u32x4_t descriptor(const void* base, int bytes)
{
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    return u32x4_t{static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32), static_cast<uint32_t>(bytes), 0x00020000u};
}

/* buffer_load_lds16 behind the compiler's back, which else lets every transposing read wait for all loads in flight
 * (8192 x 4096 x 14336: 920 us for dX, so 842).  It writes no register; the nops stand between the scalar
 * registers' writes and their use.  The waits that the compiler sets for other loads count these too, so they only wait
 * longer, and what it doesn't wait for wait_all does. */
__device__ __forceinline__ void load_lds16(u32x4_t rs, char* dst, int voff, int soff)
{
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) char*)dst));
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   /* m0 is a reserved register; nothing else here uses it */
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(at), "v"(voff), "s"(rs), "s"(soff)
                 : "m0", "memory");
#pragma clang diagnostic pop
}

__device__ __forceinline__ void wait_all() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_sched_barrier(0);
    wait_all();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

/* A stage of 64 k is four slices of 16, each TM groups of TN matrix instructions; fragments are read D groups
 * ahead and the barrier stands D groups before the stage's end, as in hpo_mx8_linear. */
template <typename T, bool WGRAD, bool FP16, bool DIRECT>
__global__ __launch_bounds__(T::kThreads) void k_mx8_grad(ProductArgs p)
{
    constexpr int kA = T::BM * kRowBytes, kB = T::BN * kRowBytes, kStage = kA + kB;
    constexpr int kChunks = T::BM / 8 / T::kWaves;                  /* 1 KB loads of a wavefront per stage of A */
    constexpr int kPieces = T::BM * 8 / T::kThreads;                /* 16-byte pieces of a lane */
    constexpr int kCols16 = T::BN / 16, kBPieces = kStepK * kCols16 / T::kThreads;
    constexpr int kSlices = kStepK / 16;
    constexpr int G = kSlices * T::TM, D = T::TM > 1 ? 2 : 1, S = 2 * D;
    static_assert(kChunks >= 1 && kBPieces >= 1, "every wavefront stages");
    static_assert(G % S == 0 && T::TM >= D, "fragment slots");
    __shared__ __attribute__((aligned(16))) char lds[2 * kStage];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int frow = lane & 31, fh = lane >> 5;
    const Work w = work_of(p, blockIdx.x, gridDim.x);
    const int64_t m0 = static_cast<int64_t>(w.tm) * T::BM, n0 = static_cast<int64_t>(w.tn) * T::BN;
    const int rows_m = p.m - m0 < T::BM ? static_cast<int>(p.m - m0) : T::BM;
    const int rows_n = p.n - n0 < T::BN ? static_cast<int>(p.n - n0) : T::BN;
    const uint16_t* A = static_cast<const uint16_t*>(p.a) + w.z * p.a_bs + (WGRAD ? m0 : m0 * p.a_rs);
    const uint8_t* B = p.b + w.z * p.b_bs + n0;
    const int64_t nb = (p.n + kMxBlock - 1) / kMxBlock;
    const uint8_t* SB = p.b_scales + w.z * p.k * nb;
    const int steps = static_cast<int>((p.k + kStepK - 1) / kStepK);
    const int tail = static_cast<int>(p.k - static_cast<int64_t>(steps - 1) * kStepK);
    auto rows_of = [&](int kt) { return kt + 1 < steps ? kStepK : kt < steps ? tail : 0; };
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * w.split / p.splits);
    const int k1 = static_cast<int>(static_cast<int64_t>(steps) * (w.split + 1) / p.splits);

    u32x4_t rsA;
    int voff[DIRECT ? kChunks : 1], piece[DIRECT ? kChunks : 1];
    u32x4_t held[DIRECT ? 1 : kPieces];
    if constexpr (DIRECT) {
        if constexpr (!WGRAD)
            rsA = descriptor(A, static_cast<int>(((rows_m - 1) * p.a_rs + p.k) * 2));
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
        const int left = rows_of(kt);
        const int64_t k = left > 0 ? static_cast<int64_t>(kt) * kStepK : 0;
        if constexpr (DIRECT && WGRAD) {
            /* rows behind the last token lie behind the descriptor's end, and columns behind C's side are
             * copies of what follows them; their sums are not kept.  The end is that of an aligned word:
             * a word that is only partly inside would read as 0. */
            const u32x4_t rs = descriptor(A + k * p.a_rs,
                                          left > 0 ? static_cast<int>((((left - 1) * p.a_rs + rows_m) * 2 + 3) & ~3) : 0);
#pragma unroll
            for (int c = 0; c < kChunks; ++c)
                load_lds16(rs, lds + buf * kStage + (wave * kChunks + c) * 1024, voff[c], 0);
        } else if constexpr (DIRECT) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                const int v = left >= kStepK || piece[c] * 8 < left ? voff[c] : kNowhere;
                load_lds16(rsA, lds + buf * kStage + (wave * kChunks + c) * 1024, v, left > 0 ? kt * kRowBytes : 0);
            }
        } else {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int i = c * T::kThreads + tid;
                if constexpr (WGRAD) {
                    const int r = i / (T::BM / 8), at = i % (T::BM / 8) * 8;
                    held[c] = load16(reinterpret_cast<const uint8_t*>(A + (k + r) * p.a_rs + at), r < left ? 2 * (rows_m - at) : 0,
                                     2 * (m0 + at));
                } else {
                    const int r = i >> 3, at = (i & 7) * 8;
                    held[c] = load16(reinterpret_cast<const uint8_t*>(A + (r < rows_m ? r : rows_m - 1) * p.a_rs + k + at),
                                     2 * (left - at), 2 * (k + at));
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
    const int brow = tid / kCols16, bcol = tid % kCols16 * 16;   /* piece c: kThreads / kCols16 rows further each */
    constexpr int kBRows = T::kThreads / kCols16;
    auto fetch_b = [&](int kt) {
        const int rows = rows_of(kt);
        const int64_t k = rows > 0 ? static_cast<int64_t>(kt) * kStepK : 0;
        if constexpr (DIRECT) {
            /* rows behind the last lie behind the descriptors' ends, stages behind the last wholly; columns behind C's side
             * are copies of what follows them, and their sums are not kept.  The end is that of an aligned word. */
            const int bytes = rows > 0 ? (static_cast<int>((rows - 1) * p.b_rs) + rows_n + 3) & ~3 : 0;
            const int sbytes = rows > 0 ? static_cast<int>((rows - 1) * nb) + (rows_n + kMxBlock - 1) / kMxBlock : 0;
            const __amdgpu_buffer_rsrc_t rs =
                __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(B + k * p.b_rs), 0, bytes, 0x00020000);
            const __amdgpu_buffer_rsrc_t ss =
                __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(SB + k * nb + n0 / kMxBlock), 0, sbytes, 0x00020000);
#pragma unroll
            for (int c = 0; c < kBPieces; ++c) {
                const int r = brow + c * kBRows;
                bheld[c] = __builtin_bit_cast(
                    u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, r * static_cast<int>(p.b_rs) + bcol, 0, 0));
                bscale[c] = __builtin_amdgcn_raw_buffer_load_b8(ss, r * static_cast<int>(nb) + bcol / kMxBlock, 0, 0);
            }
        } else {
#pragma unroll
            for (int c = 0; c < kBPieces; ++c) {
                const int r = brow + c * kBRows;
                const bool in = r < rows && bcol < rows_n;
                bheld[c] = load16(B + (k + r) * p.b_rs + bcol, in ? rows_n - bcol : 0, n0 + bcol);
                bscale[c] = in ? SB[(k + r) * nb + (n0 + bcol) / kMxBlock] : 127u;
            }
        }
    };
    auto put_b = [&](int c, int buf) {
        const int r = brow + c * kBRows;
        const float s = __uint_as_float(bscale[c] << 23);
        char* dst = lds + buf * kStage + kA + r * (T::BN * 2) + (bcol / 16 ^ pair_swizzle<T::BN>(r)) * 32;
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
    auto frag_a = [&](int buf, int i, int s) {
        const char* src = lds + buf * kStage;
        if constexpr (WGRAD)
            return transposed<T::BM>(src + (16 * s + tk) * (T::BM * 2) +
                                     (((am + 32 * i) / 16 + tg) ^ pair_swizzle<T::BM>(tk)) * 32 + tc * 8);
        else
            return *reinterpret_cast<const u32x4_t*>(src + piece_at(am + 32 * i + frow, 2 * s + fh));
    };
    auto frag_b = [&](int buf, int j, int s) {
        return transposed<T::BN>(lds + buf * kStage + kA + (16 * s + tk) * (T::BN * 2) +
                                 (((bn + 32 * j) / 16 + tg) ^ pair_swizzle<T::BN>(tk)) * 32 + tc * 8);
    };
    u32x4_t fa[S], fb[2][T::TN];
    /* Behind the barrier, D groups before the stage's end, nobody reads this stage's places any more, and the loads of
     * the stage after next go out: A's into LDS, B's into registers.  The groups before the barrier turn B's values of
     * the next stage into 16 bits, as late as they can: in the stage's first half they wait for their loads (860 us,
     * so 842). */
    auto stage = [&](int kt, auto MORE) {
        constexpr bool more = decltype(MORE)::value;
        const int buf = (kt - k0) & 1;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if constexpr (more) {
                if (g >= G - D - kBPieces && g < G - D)
                    put_b(g - (G - D - kBPieces), buf ^ 1);
                if (g == G - D) {
                    put_a(buf ^ 1);
                    meet();
                    fetch_a(kt + 2, buf);
                    fetch_b(kt + 2);
                }
            }
            const int h = (g + D) % G, s = h / T::TM;
            if (g + D < G || more) {
                const int from = g + D < G ? buf : buf ^ 1;
                if (h % T::TM == 0) {
#pragma unroll
                    for (int j = 0; j < T::TN; ++j)
                        fb[s & 1][j] = frag_b(from, j, s);
                }
                fa[(g + D) % S] = frag_a(from, h % T::TM, s);
            }
            __builtin_amdgcn_sched_barrier(0);
            const int i = g % T::TM;
#pragma unroll
            for (int j = 0; j < T::TN; ++j)
                acc[i][j] = mfma16<FP16>(fb[(g / T::TM) & 1][j], fa[g % S], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (k0 < k1) {
        fetch_b(k0);
        fetch_a(k0, 0);
        put_a(0);
#pragma unroll
        for (int c = 0; c < kBPieces; ++c)
            put_b(c, 0);
        meet();
        fetch_a(k0 + 1, 1);
        fetch_b(k0 + 1);
#pragma unroll
        for (int g = 0; g < D; ++g) {
            if (g % T::TM == 0) {
#pragma unroll
                for (int j = 0; j < T::TN; ++j)
                    fb[(g / T::TM) & 1][j] = frag_b(0, j, g / T::TM);
            }
            fa[g] = frag_a(0, g % T::TM, g / T::TM);
        }
        int kt = k0;
        for (; kt + 1 < k1; ++kt)
            stage(kt, std::true_type{});
        stage(kt, std::false_type{});
        wait_all();   /* what was fetched for stages that are not here */
    }
    epilogue<T, WGRAD>(p, w, lds, acc);
}

template <typename T, bool WGRAD, bool DIRECT>
hipError_t grad_tile(const ProductArgs& p, uint32_t grid, hipStream_t stream)
{
    return p.fp16 ? launch(k_mx8_grad<T, WGRAD, true, DIRECT>, dim3(grid), T::kThreads, stream, p)
                  : launch(k_mx8_grad<T, WGRAD, false, DIRECT>, dim3(grid), T::kThreads, stream, p);
}

template <bool WGRAD>
hipError_t grad_kind(const ProductArgs& p, int32_t tile, bool direct, uint32_t grid, hipStream_t stream)
{
    if (tile == 256)
        return grad_tile<Tile256, WGRAD, true>(p, grid, stream);
    if (tile == 128)
        return direct ? grad_tile<Tile128, WGRAD, true>(p, grid, stream) : grad_tile<Tile128, WGRAD, false>(p, grid, stream);
    return direct ? grad_tile<Tile64, WGRAD, true>(p, grid, stream) : grad_tile<Tile64, WGRAD, false>(p, grid, stream);
}

}  // namespace

hipError_t launch_mx8_grad(bool wgrad, const ProductArgs& p, int32_t tile, bool direct, uint32_t grid, hipStream_t stream)
{
    return wgrad ? grad_kind<true>(p, tile, direct, grid, stream) : grad_kind<false>(p, tile, direct, grid, stream);
}

}  // namespace hpo
