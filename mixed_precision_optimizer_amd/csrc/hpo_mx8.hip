/*
 * hpo_mx8.hip -- gfx950 kernels of activations and weights in 8 bits with block
 * scales: the quantisation (hpo_mx8_save) and the products of a linear layer,
 * Y = X^ W^T, dX = dY W^, G += scale * dY^T X^ (hpo_mx8_linear, _dgrad, _wgrad).
 */
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "hpo_product_device.h"

namespace hpo {
namespace {


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

/* Adds the splits' sums, in order.  Lanes take four neighbouring sums at a time. */
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
 * of the second, and the scale of block h.
 *
 * Slices of 64 k lie in a ring of four in LDS; one is TM groups of TN matrix instructions, and fragments are
 * read D groups ahead, across the slice's end too.  A barrier stands D groups before that end, where the next slice
 * must have landed and nobody reads this one any more: its place goes to the loads of the slice after next but
 * one, so that a load has the time of three slices (with two whole stages of 128 in LDS, one ahead, the loop waits
 * for loads: 8192 x 4096 x 14336 takes 467 us).  The loop's body is a stage of two slices, and the scale words are
 * read once for both. */
template <typename T, bool DIRECT>
__global__ __launch_bounds__(T::kThreads) void k_mx8_linear(ProductArgs p)
{
    constexpr int kRows = T::BM + T::BN;
    constexpr int kSlice = kRows * kSliceBytes;
    constexpr int kScales = 4 * kSlice;               /* behind the slices: 16 scale bytes a row, twice */
    constexpr int kScaleStage = kRows * 16;
    constexpr int kChunks = kRows / 16 / T::kWaves;   /* 1 KB loads of a wavefront per slice: all of A or all of B */
    constexpr int kPieces = kRows * 4 / T::kThreads;
    constexpr int kScaleRows = (kRows + T::kThreads - 1) / T::kThreads;
    constexpr int G = 2 * T::TM, D = T::TM > 1 ? 2 : 1, S = 2 * D;
    static_assert((T::BM / 16) % kChunks == 0, "a wavefront stages rows of one operand");
    static_assert(G % S == 0 && T::TM >= D, "fragment slots");
    __shared__ __attribute__((aligned(16))) char lds[4 * kSlice + 2 * kScaleStage];
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
    const int steps = static_cast<int>((p.k + 127) / 128);
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * w.split / p.splits);
    const int k1 = static_cast<int>(static_cast<int64_t>(steps) * (w.split + 1) / p.splits);

    /* tile row -> source row; rows behind C's sides hold copies of the last and their sums are not kept */
    auto clamp = [&](int r) { return r < T::BM ? (r < rows_m ? r : rows_m - 1) : (r - T::BM < rows_n ? r - T::BM : rows_n - 1); };

    /* straight into LDS: rows behind C's sides lie behind the descriptor's end, or (a lone row, stride
     * 0) hold copies of it */
    const bool side_b = wave * kChunks >= T::BM / 16;
    __amdgpu_buffer_rsrc_t rs;
    int ld = 0, voff = 0;
    const int piece = ((lane & 3) ^ slice_swizzle(lane >> 2)) * 16;
    u32x4_t held[DIRECT ? 1 : kPieces];
    if constexpr (DIRECT) {
        ld = static_cast<int>(side_b ? p.b_rs : p.a_rs);
        rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(side_b ? B : A), 0,
                                               static_cast<int>(((side_b ? rows_n : rows_m) - 1) * ld + p.k), 0x00020000);
        voff = (wave * kChunks * 16 - (side_b ? T::BM : 0) + (lane >> 2)) * ld + piece;
    }
    /* Loads first .. last - 1 of slice x, which goes to place `to`.  Slices behind the last are fetched too, as
     * zeros from nowhere: the loads in flight stay as many. */
    auto fetch = [&](int x, int to, int first, int last) {
        const int64_t k = static_cast<int64_t>(x) * 64, left = p.k - k;   /* bytes of the row from here */
        if constexpr (DIRECT) {
            const int v = left >= 64 || piece < left ? voff : kNowhere, soff = left > 0 ? static_cast<int>(k) : 0;
#pragma unroll
            for (int c = first; c < last; ++c)
                buffer_load_lds16(rs, lds + to * kSlice + (wave * kChunks + c) * 1024, v, soff + c * 16 * ld);
        } else {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int i = c * T::kThreads + tid, r = i >> 2, at = (i & 3) * 16;
                const uint8_t* row = r < T::BM ? A + clamp(r) * p.a_rs : B + clamp(r) * p.b_rs;
                held[c] = load16(row + k + at, left - at);
            }
        }
    };
    auto put = [&](int to) {
        if constexpr (!DIRECT) {
#pragma unroll
            for (int c = 0; c < kPieces; ++c) {
                const int i = c * T::kThreads + tid;
                *reinterpret_cast<u32x4_t*>(lds + to * kSlice + slice_at(i >> 2, i & 3)) = held[c];
            }
        }
    };
    /* The next slice has landed: the two behind it may still be in flight. */
    auto arrive = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(waitcnt(DIRECT ? 2 * kChunks : 63));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    /* Scales of four stages at a time; a byte behind the row's end reads as 0, never as a neighbour's NaN.
     * A row of fewer than 16 has only the first stages'; longer ones read their last 16 at their end. */
    u32x4_t sheld[kScaleRows];
    const uint8_t* srow[kScaleRows];
    int late = 0;   /* bits that the held scales lie too early */
#pragma unroll
    for (int c = 0; c < kScaleRows; ++c) {
        const int r = c * T::kThreads + tid;
        srow[c] = (r < T::BM ? SA : SB) + clamp(r < kRows ? r : 0) * nb;
    }
    auto fetch_scales = [&](int64_t at) {
        if (nb >= 16) {
            const int64_t start = at < nb - 16 ? at : nb - 16;
            late = at - start < 16 ? static_cast<int>(at - start) * 8 : 0;   /* 16 and more: behind the last stage */
#pragma unroll
            for (int c = 0; c < kScaleRows; ++c)
                sheld[c] = *reinterpret_cast<const u32x4_any*>(srow[c] + start);
        }
    };
    auto put_scales = [&](int at) {
        if (late > 0) {
#pragma unroll
            for (int c = 0; c < kScaleRows; ++c) {
                uint64_t lo = sheld[c][0] | (static_cast<uint64_t>(sheld[c][1]) << 32);
                uint64_t hi = sheld[c][2] | (static_cast<uint64_t>(sheld[c][3]) << 32);
                lo = late < 64 ? (lo >> late) | (hi << (64 - late)) : hi >> (late - 64);
                hi = late < 64 ? hi >> late : 0;
                sheld[c] = u32x4_t{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                                   static_cast<uint32_t>(hi >> 32)};
            }
        }
#pragma unroll
        for (int c = 0; c < kScaleRows; ++c) {
            const int r = c * T::kThreads + tid;
            if (kRows % T::kThreads == 0 || r < kRows)
                *reinterpret_cast<u32x4_t*>(lds + at + r * 16) = sheld[c];
        }
    };

    f32x16_t acc[T::TM][T::TN];
#pragma unroll
    for (int i = 0; i < T::TM; ++i)
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            acc[i][j] = f32x16_t{};
    const int am = wave / T::WN * (T::TM * 32) + frow, bn = T::BM + wave % T::WN * (T::TN * 32) + frow;
    /* pieces fh and 2 + fh of a lane's row: the second at the first's offset with bit 5 turned over */
    const int base_a = slice_at(am, fh), base_b = slice_at(bn, fh);
    auto frag = [&](int base, int block, int s) {
        const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(lds + base + s * kSlice + block * (32 * kSliceBytes));
        const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(lds + (base ^ 32) + s * kSlice + block * (32 * kSliceBytes));
        return i32x8_t{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]),
                       static_cast<int>(hi[0]), static_cast<int>(hi[1]), static_cast<int>(hi[2]), static_cast<int>(hi[3])};
    };
    i32x8_t fa[S], fb[2][T::TN];
    int sa[T::TM], sb[T::TN], na[T::TM], nb4[T::TN];
    /* the scale words of stage `at` from the first: block h of slice s in byte 2 s */
    auto read_scales = [&](unsigned at) {
        const char* scl = lds + kScales + (at >> 2 & 1) * kScaleStage + (at & 3) * 4;
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
            na[i] = static_cast<int>(*reinterpret_cast<const uint32_t*>(scl + (am + 32 * i) * 16) >> (8 * fh));
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            nb4[j] = static_cast<int>(*reinterpret_cast<const uint32_t*>(scl + (bn + 32 * j) * 16) >> (8 * fh));
    };
    auto take_scales = [&]() {
#pragma unroll
        for (int i = 0; i < T::TM; ++i)
            sa[i] = na[i];
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            sb[j] = nb4[j];
    };
    if (k0 < k1) {
#pragma unroll
        for (int c = 0; c < kScaleRows; ++c)
            sheld[c] = load16(srow[c] + 4 * static_cast<int64_t>(k0), nb - 4 * static_cast<int64_t>(k0));
        if constexpr (DIRECT) {
#pragma unroll
            for (int x = 0; x < 3; ++x)
                fetch(2 * k0 + x, x, 0, kChunks);
            put_scales(kScales);
            arrive();
            fetch(2 * k0 + 3, 3, 0, kChunks * D / T::TM);
        } else {
            fetch(2 * k0, 0, 0, 0);
            put_scales(kScales);
            put(0);
            arrive();
            fetch(2 * k0 + 1, 1, 0, 0);
        }
        read_scales(0);
        take_scales();
#pragma unroll
        for (int j = 0; j < T::TN; ++j)
            fb[0][j] = frag(base_b, j, 0);
#pragma unroll
        for (int g = 0; g < D; ++g)
            fa[g] = frag(base_a, g % T::TM, g / T::TM);
        for (int kt = k0; kt < k1; ++kt) {
            const unsigned at = static_cast<unsigned>(kt - k0);
            const int pair = static_cast<int>(at & 1) * 2;   /* places pair, pair + 1 of the ring */
            int here_a = base_a + pair * kSlice, here_b = base_b + pair * kSlice;
            /* not to be kept for both halves of the ring in registers that the sums need */
            asm volatile("" : "+v"(here_a), "+v"(here_b));
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int slice = g / T::TM;
                if (g % T::TM == T::TM - D) {
                    put(slice == 0 ? pair + 1 : pair ^ 2);
                    arrive();
                    if constexpr (!DIRECT)
                        fetch(2 * kt + 2 + slice, 0, 0, 0);
                    if (slice == 1) {
                        /* four stages' scales are fetched in the second of the four before and put down in the third */
                        if ((at & 3) == 1)
                            fetch_scales(4 * static_cast<int64_t>(kt + 3));
                        if ((at & 3) == 2)
                            put_scales(kScales + ((at >> 2 & 1) ^ 1) * kScaleStage);
                        read_scales(at + 1);
                        here_a = base_a + (pair ^ 2) * kSlice;
                        here_b = base_b + (pair ^ 2) * kSlice;
                        asm volatile("" : "+v"(here_a), "+v"(here_b));
                    }
                }
                const int h = (g + D) % G, s = h / T::TM;
                if constexpr (DIRECT) {
                    /* a group's share of the loads: all at once they would keep every wavefront from its products
                     * until the last is taken.  Before slice 0's barrier they are still those of the stage before. */
                    const int q = h % T::TM;
                    const int first = q * kChunks / T::TM, last = (q + 1) * kChunks / T::TM, freed = (g + D - T::TM) / T::TM;
                    if (g < T::TM - D)
                        fetch(2 * kt + 3, pair ^ 3, first, last);
                    else
                        fetch(2 * kt + 4 + freed, pair + freed, first, last);
                }
                if (h % T::TM == 0) {
#pragma unroll
                    for (int j = 0; j < T::TN; ++j)
                        fb[s][j] = frag(here_b, j, s);
                }
                fa[(g + D) % S] = frag(here_a, h % T::TM, s);
                __builtin_amdgcn_sched_barrier(0);
                const int i = g % T::TM;
#pragma unroll
                for (int j = 0; j < T::TN; ++j) {
                    if (slice == 0)
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[0][j], fa[g % S], acc[i][j], 0, 0, 0,
                                                                                    sb[j], 0, sa[i]);
                    else
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[1][j], fa[g % S], acc[i][j], 0, 0, 2,
                                                                                    sb[j], 2, sa[i]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            take_scales();
        }
    }
    land();
    epilogue<T, false>(p, w, lds, acc);
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
    const int64_t depth = kind == kLinear ? 128 : kStepK, steps = (k + depth - 1) / depth;
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

template <typename T>
hipError_t linear_tile(const ProductArgs& p, bool direct, uint32_t grid, hipStream_t stream)
{
    return direct ? launch(k_mx8_linear<T, true>, dim3(grid), T::kThreads, stream, p)
                  : launch(k_mx8_linear<T, false>, dim3(grid), T::kThreads, stream, p);
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
    Cut c = cut_of(kind, p.batch, p.m, p.n, p.k);
    const bool direct = is_direct(kind, p, c.tile);
    if (!direct && c.tile == 256) {   /* the stages pass through registers, and beside 128 sums there are none */
        c.tile = 128;
        c.tiles_m = (p.m + 127) / 128;
        c.tiles_n = (p.n + 127) / 128;
    }
    const int64_t grid = p.batch * c.tiles_m * c.tiles_n * c.splits;
    if (grid > INT32_MAX)
        return hipErrorInvalidConfiguration;
    p.tiles_m = static_cast<int32_t>(c.tiles_m);
    p.tiles_n = static_cast<int32_t>(c.tiles_n);
    p.splits = c.splits;
    const uint32_t g = static_cast<uint32_t>(grid);
    hipError_t e = kind != kLinear ? launch_mx8_grad(kind == kWgrad, p, c.tile, direct, g, stream)
                   : c.tile == 256 ? launch(k_mx8_linear<Tile256, true>, dim3(g), Tile256::kThreads, stream, p)
                   : c.tile == 128 ? linear_tile<Tile128>(p, direct, g, stream)
                                   : linear_tile<Tile64>(p, direct, g, stream);
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
