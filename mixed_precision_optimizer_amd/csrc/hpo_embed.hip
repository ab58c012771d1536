/*
 * hpo_embed.hip -- gfx950 kernels of the embedding table: rows by token
 * (hpo_embedding) and their gradient added to the main grad
 * (hpo_embedding_grad).
 *
 * Both are bound by HBM.  The lookup moves one table row and one output row per token; a group of
 * lanes takes a row, eight elements a lane: 8192 tokens of 4096 bf16 take 24 to 26 us, 19 where table and results stay in
 * the 256 MB cache from call to call (the rows of repeated tokens come from L2).
 *
 * The gradient adds rows of dY that belong to one token.  Atomics on the main grad would leave
 * the order of the sums to chance and pass over G once per token, so the tokens are sorted
 * first (stable: equal tokens stay in order of position) and the sorted list is cut into
 * slabs of equal length, one per group of lanes and column piece: the work is even however often a
 * token comes.  A run of equal tokens inside a slab goes straight into its row of G, each row read and
 * written once; a run that crosses a slab's border leaves its parts in the workspace, and a last
 * launch adds these in order.  Up to 128 tokens one launch does without the sort: the first
 * token of its kind adds up the others.  8192 tokens of 4096 into an fp32 main grad take 69 to 71 us: sort 13, sums 53 (196 MB
 * from and to HBM at 3.7 TB/s), join 6, no gaps between the launches; 51 us, 34 of them the sums, where one call's
 * operands are in the 256 MB cache from the call before.
 */
#include <hip/hip_runtime.h>

#include "hpo_model_device.h"

namespace hpo {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ int64_t id_at(const void* ids, int id64, int64_t t)
{
    return id64 ? static_cast<const int64_t*>(ids)[t] : static_cast<int64_t>(static_cast<const int32_t*>(ids)[t]);
}

/* Row of the table, or -1. */
__device__ __forceinline__ int64_t row_of(const void* ids, int id64, int64_t t, int64_t first, int64_t rows)
{
    const uint64_t d = static_cast<uint64_t>(id_at(ids, id64, t)) - static_cast<uint64_t>(first);
    return d < static_cast<uint64_t>(rows) ? static_cast<int64_t>(d) : -1;
}

/* Eight weights of a row in fp32. */
template <int WT>
__device__ __forceinline__ void weight8(const EmbedArgs& a, int64_t row, int64_t col, int n, float (&x)[8])
{
    if constexpr (WT == HPO_WEIGHT_MX8) {
        const uint8_t* p = static_cast<const uint8_t*>(a.w) + row * a.w_rs + col;
        const int64_t nb = (a.cols + kMxBlock - 1) / kMxBlock;
        const uint32_t byte = a.scales[row * nb + col / kMxBlock];
        uint32_t v[2] = {0, 0};
        if (n >= 8) {
            const u32x2_t t = *reinterpret_cast<const u32x2_any*>(p);
            v[0] = t.x;
            v[1] = t.y;
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n)
                    v[e >> 2] |= static_cast<uint32_t>(p[e]) << (8 * (e & 3));
        }
        /* 2^(byte - 127): the exponent field, but 2^-127 is subnormal; exact products of four bits */
        const float f = __uint_as_float(byte == 255u ? 0x7fc00000u : (byte > 0u ? byte << 23 : 1u << 22));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v[h]), false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(v[h]), true);
            x[4 * h] = lo[0] * f;
            x[4 * h + 1] = lo[1] * f;
            x[4 * h + 2] = hi[0] * f;
            x[4 * h + 3] = hi[1] * f;
        }
    } else {
        load8<WT>(a.w, row * a.w_rs + col, n, x);
    }
}

/* LANES lanes take a row, in steps of eight elements each. */
template <int WT, int OT, int LANES>
__global__ __launch_bounds__(kRowThreads) void k_embedding(EmbedArgs a)
{
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / LANES) + threadIdx.x / LANES;
    if (t >= a.n)
        return;
    const int64_t row = row_of(a.ids, a.id64, t, a.first, a.rows);
#pragma unroll 2
    for (int64_t c = 8 * (threadIdx.x % LANES); c < a.cols; c += 8 * LANES) {
        const int n = a.cols - c > 8 ? 8 : static_cast<int>(a.cols - c);
        float x[8] = {};
        if (row >= 0) {
            weight8<WT>(a, row, c, n, x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] *= a.scale;
        }
        store8<OT>(a.out, t * a.out_rs + c, n, x);
    }
}

/* ---------------------------------------------------------------------- */
/* the sorted tokens                                                       */
/* ---------------------------------------------------------------------- */
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kDigitBits = 11;                 /* of a pass, at most; keys have 22 at most */
constexpr int kBins = 1 << kDigitBits;
constexpr int kBlockItems = 4;                 /* where many do */
constexpr int kBlockTokens = kSortThreads * kBlockItems;

/* Where the sorted list lies: row of the table (or `rows`, behind all others, for an id without one) and
 * position of each token. */
struct Sorted {
    int32_t *key, *tok;          /* the result */
    int32_t *key_mid, *tok_mid;  /* between two passes */
    int32_t* hist;               /* [block][bin] */
};

/* The tokens' counts by digit of one workgroup, and the offsets they turn into. */
struct DigitLds {
    uint16_t count[kSortWaves][kBins];   /* per wavefront; then: tokens of earlier wavefronts in the bin */
    uint32_t base[kBins];                /* position of the bin's first token of this workgroup */
    uint32_t wave_sum[kSortWaves];
};

/* Exclusive sums of lds.base over the bins. */
__device__ __forceinline__ void scan_bins(DigitLds& lds, int bins)
{
    constexpr int kPer = kBins / kSortThreads;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    uint32_t v[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        v[j] = tid * kPer + j < bins ? lds.base[tid * kPer + j] : 0;
        mine += v[j];
    }
    uint32_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(sum, d, 64);
        if (lane >= d)
            sum += o;
    }
    if (lane == 63)
        lds.wave_sum[wave] = sum;
    __syncthreads();
    uint32_t before = sum - mine;
    for (int w = 0; w < wave; ++w)
        before += lds.wave_sum[w];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (tid * kPer + j < bins) {
            lds.base[tid * kPer + j] = before;
            before += v[j];
        }
    __syncthreads();
}

/* Ranks the workgroup's tokens (ITEMS a lane; a wavefront holds 64 * ITEMS in a row, item i of its lanes being 64 of
 * them in a row) by one digit: rank[i] = tokens of the same digit before it in its wavefront, and
 * lds.count the tokens of earlier wavefronts.  n[bin] of the workgroup goes to lds.base. */
template <int ITEMS>
__device__ __forceinline__ void rank_digits(DigitLds& lds, const int32_t (&key)[ITEMS], uint32_t valid, int shift, int bits,
                                            uint32_t (&rank)[ITEMS])
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, bins = 1 << bits;
    for (int i = tid; i < kSortWaves * bins; i += kSortThreads)
        lds.count[i / bins][i % bins] = 0;
    __syncthreads();
    volatile uint16_t* mine = lds.count[wave];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const bool in = (valid >> i) & 1u;
        const uint32_t d = (static_cast<uint32_t>(key[i]) >> shift) & (bins - 1);
        uint64_t same = __ballot(in);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((d >> b) & 1u);
            same &= (d >> b) & 1u ? set : ~set;
        }
        /* a wavefront's LDS accesses keep their order: every lane reads before a first one writes */
        const uint32_t before = in ? mine[d] : 0;
        const uint32_t below = __builtin_popcountll(same & ((uint64_t{1} << lane) - 1));
        rank[i] = before + below;
        __builtin_amdgcn_wave_barrier();
        if (in && below == 0)
            mine[d] = static_cast<uint16_t>(before + __builtin_popcountll(same));
        __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();
    for (int d = tid; d < bins; d += kSortThreads) {
        uint32_t sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = lds.count[w][d];
            lds.count[w][d] = static_cast<uint16_t>(sum);
            sum += c;
        }
        lds.base[d] = sum;
    }
    __syncthreads();
}

__device__ __forceinline__ int32_t key_of(const EmbedGradArgs& a, int64_t t)
{
    const int64_t row = row_of(a.ids, a.id64, t, a.first, a.rows);
    return static_cast<int32_t>(row < 0 ? a.rows : row);
}

/* One launch for up to kBucketMax tokens, as every workgroup looks through all of them; counting passes (two or four
 * launches) behind that.  Whole calls, in microseconds, by buckets and by counting: 4096 tokens of 1024 into 32000 rows 22
 * and 34, 16384 43 and 54, 32768 65 and 65, 65536 108 and 84, 131072 227 and 153; into 1000 rows 16384 39 and 40, 32768 57
 * and 47; of 64 into 128256 rows 32768 39 and 46, 65536 68 and 53.  So the two meet between 16384 and 65536 tokens, and up
 * to the limit the worst is 1.6 times the better.
 *
 * Workgroup b looks through all of them for the rows with row mod
 * gridDim.x = b, which are its part of the list (behind those of the buckets before it), collects them in
 * order of position, and sorts them by the rest of the row.  So equal rows come together, though not in
 * their order; ids without a row come last. */
constexpr int kBucketThreads = 1024;
constexpr int kBucketWaves = kBucketThreads / 64;
constexpr int kBucketMax = 65536;
constexpr int kBucketBins = 2048;   /* rests of a row */
constexpr int kBucketHold = 16;     /* tokens of a lane that are kept between the two looks */

__global__ __launch_bounds__(kBucketThreads) void k_sort_bucket(EmbedGradArgs a, Sorted s, int shift)
{
    __shared__ uint32_t count[kBucketWaves][kBucketBins];
    __shared__ uint32_t wave_in[kBucketWaves], wave_below[kBucketWaves], wave_rows[kBucketWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = static_cast<int>(a.n);
    const uint32_t bucket = blockIdx.x, mask = (1u << shift) - 1u;
    const int bins = static_cast<int>((a.rows - 1) >> shift) + 1;
    const int chunks = (n + 64 * kBucketWaves - 1) / (64 * kBucketWaves), first = wave * chunks * 64 + lane;
    const int32_t none = static_cast<int32_t>(a.rows);
    int32_t held[kBucketHold];
    uint32_t in = 0, below = 0, listed = 0;
    auto look = [&](int32_t key) {
        const uint32_t r = static_cast<uint32_t>(key) & mask;
        in += __builtin_popcountll(__ballot(key < none && r == bucket));
        below += __builtin_popcountll(__ballot(key < none && r < bucket));
        listed += __builtin_popcountll(__ballot(key < none));
    };
#pragma unroll
    for (int c = 0; c < kBucketHold; ++c) {
        const int t = first + 64 * c;
        held[c] = c < chunks && t < n ? key_of(a, t) : none;
    }
#pragma unroll
    for (int c = 0; c < kBucketHold; ++c)
        look(held[c]);
    for (int c = kBucketHold; c < chunks; ++c) {
        const int t = first + 64 * c;
        look(t < n ? key_of(a, t) : none);
    }
    if (lane == 0) {
        wave_in[wave] = in;
        wave_below[wave] = below;
        wave_rows[wave] = listed;
    }
    for (int d = tid; d < bins; d += kBucketThreads)
#pragma unroll
        for (int w = 0; w < kBucketWaves; ++w)
            count[w][d] = 0;
    __syncthreads();
    uint32_t start = 0, mine = 0, all = 0, rows = 0;
#pragma unroll
    for (int w = 0; w < kBucketWaves; ++w) {
        start += wave_below[w];
        mine += w < wave ? wave_in[w] : 0;
        all += wave_in[w];
        rows += wave_rows[w];
    }
    for (uint32_t p = rows + bucket * kBucketThreads + tid; p < a.n; p += gridDim.x * kBucketThreads)
        s.key[p] = none;   /* its token is not looked at */
    if (all == 0)
        return;
    /* the bucket's tokens in order of position, to their part of the list */
    uint32_t at = start + mine;
    auto collect = [&](int t, int32_t key) {
        const uint64_t got = __ballot(key < none && (static_cast<uint32_t>(key) & mask) == bucket);
        if ((got >> lane) & 1u) {
            const uint32_t p = at + __builtin_popcountll(got & ((uint64_t{1} << lane) - 1));
            s.key_mid[p] = key;
            s.tok_mid[p] = t;
        }
        at += __builtin_popcountll(got);
    };
#pragma unroll
    for (int c = 0; c < kBucketHold; ++c)
        collect(first + 64 * c, held[c]);
    for (int c = kBucketHold; c < chunks; ++c) {
        const int t = first + 64 * c;
        collect(t, t < n ? key_of(a, t) : none);
    }
    __threadfence_block();
    __syncthreads();
    /* how many each wavefront has of every row, then where they go */
    const int parts = (static_cast<int>(all) + 64 * kBucketWaves - 1) / (64 * kBucketWaves);
    const uint32_t end = start + all;
    auto each = [&](auto&& fn) {
        for (int c = 0; c < parts; ++c) {
            const uint32_t p = start + (wave * parts + c) * 64 + lane;
            const bool there = p < end;
            const int32_t key = there ? s.key_mid[p] : -1;
            uint64_t same = __ballot(there);   /* lanes with this lane's row */
            for (int d = 0; (bins - 1) >> d != 0; ++d) {
                const uint64_t set = __ballot((key >> (shift + d)) & 1);
                same &= (key >> (shift + d)) & 1 ? set : ~set;
            }
            if (there)
                fn(p, key, same);
        }
    };
    volatile uint32_t* own = count[wave];
    each([&](uint32_t, int32_t key, uint64_t same) {
        if ((same & ((uint64_t{1} << lane) - 1)) == 0)
            own[key >> shift] += __builtin_popcountll(same);
    });
    __syncthreads();
    /* exclusive sums over the rows, and over the wavefronts within one */
    constexpr int kPer = (kBucketBins + kBucketThreads - 1) / kBucketThreads;
    uint32_t sums[kPer], total = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = tid * kPer + j;
        sums[j] = 0;
        if (d < bins)
#pragma unroll
            for (int w = 0; w < kBucketWaves; ++w)
                sums[j] += count[w][d];
        total += sums[j];
    }
    uint32_t incl = total;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(incl, d, 64);
        if (lane >= d)
            incl += o;
    }
    if (lane == 63)
        wave_in[wave] = incl;
    __syncthreads();
    uint32_t before = start + incl - total;
    for (int w = 0; w < wave; ++w)
        before += wave_in[w];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = tid * kPer + j;
        if (d < bins)
#pragma unroll
            for (int w = 0; w < kBucketWaves; ++w) {
                const uint32_t c = count[w][d];
                count[w][d] = before;
                before += c;
            }
    }
    __syncthreads();
    each([&](uint32_t p, int32_t key, uint64_t same) {
        const uint32_t rank = __builtin_popcountll(same & ((uint64_t{1} << lane) - 1)), to = own[key >> shift] + rank;
        s.key[to] = key;
        s.tok[to] = s.tok_mid[p];
        __builtin_amdgcn_wave_barrier();
        if (rank == 0)
            own[key >> shift] += __builtin_popcountll(same);
        __builtin_amdgcn_wave_barrier();
    });
}

/* FIRST: the keys come from the ids, else from the first pass. */
template <bool FIRST>
__device__ __forceinline__ uint32_t load_block(const EmbedGradArgs& a, const Sorted& s, int32_t (&key)[kBlockItems],
                                               int32_t (&tok)[kBlockItems])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t valid = 0;
#pragma unroll
    for (int i = 0; i < kBlockItems; ++i) {
        const int64_t t = static_cast<int64_t>(blockIdx.x) * kBlockTokens + wave * 64 * kBlockItems + 64 * i + lane;
        const bool in = t < a.n;
        valid |= static_cast<uint32_t>(in) << i;
        key[i] = 0;
        tok[i] = 0;
        if (in) {
            key[i] = FIRST ? key_of(a, t) : s.key_mid[t];
            tok[i] = FIRST ? static_cast<int32_t>(t) : s.tok_mid[t];
        }
    }
    return valid;
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void k_sort_count(EmbedGradArgs a, Sorted s, int shift, int bits)
{
    __shared__ uint32_t count[kBins];
    const int bins = 1 << bits;
    for (int d = threadIdx.x; d < bins; d += kSortThreads)
        count[d] = 0;
    __syncthreads();
    int32_t key[kBlockItems], tok[kBlockItems];
    const uint32_t valid = load_block<FIRST>(a, s, key, tok);
#pragma unroll
    for (int i = 0; i < kBlockItems; ++i)
        if ((valid >> i) & 1u)
            atomicAdd(&count[(static_cast<uint32_t>(key[i]) >> shift) & (bins - 1)], 1u);
    __syncthreads();
    for (int d = threadIdx.x; d < bins; d += kSortThreads)
        s.hist[static_cast<int64_t>(blockIdx.x) * bins + d] = static_cast<int32_t>(count[d]);
}

/* LAST: to the result, else between the passes. */
template <bool FIRST, bool LAST>
__global__ __launch_bounds__(kSortThreads) void k_sort_move(EmbedGradArgs a, Sorted s, int shift, int bits)
{
    __shared__ DigitLds lds;
    const int bins = 1 << bits, wave = threadIdx.x >> 6;
    int32_t key[kBlockItems], tok[kBlockItems];
    const uint32_t valid = load_block<FIRST>(a, s, key, tok);
    uint32_t rank[kBlockItems];
    rank_digits<kBlockItems>(lds, key, valid, shift, bits, rank);
    /* a bin's tokens in all workgroups, and in those before this one */
    constexpr int kPer = kBins / kSortThreads;
    uint32_t before[kPer] = {};
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = threadIdx.x + j * kSortThreads;
        if (d < bins) {
            uint32_t all = 0;
#pragma unroll 4
            for (uint32_t b = 0; b < gridDim.x; ++b) {
                const uint32_t c = static_cast<uint32_t>(s.hist[static_cast<int64_t>(b) * bins + d]);
                before[j] += b < blockIdx.x ? c : 0;
                all += c;
            }
            lds.base[d] = all;
        }
    }
    __syncthreads();
    scan_bins(lds, bins);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int d = threadIdx.x + j * kSortThreads;
        if (d < bins)
            lds.base[d] += before[j];
    }
    __syncthreads();
    int32_t* out_key = LAST ? s.key : s.key_mid;
    int32_t* out_tok = LAST ? s.tok : s.tok_mid;
#pragma unroll
    for (int i = 0; i < kBlockItems; ++i)
        if ((valid >> i) & 1u) {
            const uint32_t d = (static_cast<uint32_t>(key[i]) >> shift) & (bins - 1);
            const uint32_t p = lds.base[d] + lds.count[wave][d] + rank[i];
            out_key[p] = key[i];
            out_tok[p] = tok[i];
        }
}

/* ---------------------------------------------------------------------- */
/* sums over the sorted tokens                                             */
/* ---------------------------------------------------------------------- */
struct Slabs {
    const int32_t *key, *tok;
    float* part;       /* [slab][head, tail][width] */
    int64_t width;     /* cols, rounded up to eight */
    int64_t count;
    int32_t length;    /* tokens of a slab */
};

/* G[row] = G[row] + scale * sum, eight elements. */
template <int GT>
__device__ __forceinline__ void add8(const EmbedGradArgs& a, int64_t row, int64_t col, int n, const float (&g)[8],
                                     const float (&sum)[8])
{
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float d = a.scale * sum[e];
        x[e] = g[e] + d;
    }
    store8<GT>(a.g, row * a.g_rs + col, n, x);
}

constexpr int kFlight = 4;   /* rows of dY in flight */

/* LANES lanes take a slab's column piece of 8 * LANES elements. */
template <int YT, int GT, int LANES>
__global__ __launch_bounds__(kRowThreads) void k_grad_slabs(EmbedGradArgs a, Slabs s)
{
    const int64_t slab = static_cast<int64_t>(blockIdx.x) * (kRowThreads / LANES) + threadIdx.x / LANES;
    const int64_t col = (static_cast<int64_t>(blockIdx.y) * LANES + threadIdx.x % LANES) * 8;
    if (slab >= s.count)
        return;
    const int n = a.cols - col > 8 ? 8 : static_cast<int>(a.cols - col);   /* <= 0: no columns */
    const int64_t p0 = slab * s.length;
    const int len = a.n - p0 < s.length ? static_cast<int>(a.n - p0) : s.length;
    const int32_t none = static_cast<int32_t>(a.rows);
    /* the slab's list: a whole wavefront has it in a register, an entry per lane, and its branches are scalar */
    int32_t keys = -1, toks = 0;
    if constexpr (LANES == 64) {
        const int lane = threadIdx.x & 63, at = lane < len ? lane : len - 1;
        keys = s.key[p0 + at];
        toks = s.tok[p0 + at];
    }
    const int32_t prev = p0 > 0 ? s.key[p0 - 1] : -1, behind = p0 + len < a.n ? s.key[p0 + len] : -1;
    auto key_at = [&](int i) {
        if constexpr (LANES == 64)
            return i < len ? __builtin_amdgcn_readlane(keys, i) : __builtin_amdgcn_readfirstlane(behind);
        else
            return i < len ? s.key[p0 + i] : behind;
    };
    auto tok_at = [&](int i) {
        if constexpr (LANES == 64)
            return __builtin_amdgcn_readlane(toks, i);
        else
            return s.tok[p0 + i];
    };
    bool head = prev == key_at(0);     /* the current run began in an earlier slab */
    float sum[8] = {};
    for (int p = 0; p < len; p += kFlight) {
        int32_t key[kFlight + 1];
        Raw8<YT> y[kFlight];
        Raw8<GT> g[kFlight];
#pragma unroll
        for (int u = 0; u <= kFlight; ++u)
            key[u] = p + u <= len ? key_at(p + u) : none;
        if (key[0] >= none)
            return;               /* ids without a row: all that is left */
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            /* behind the slab or the rows: the first once more, which costs nothing */
            const int i = p + u < len && key[u] < none ? p + u : p;
            y[u] = load_raw8<YT>(a.dy, static_cast<int64_t>(tok_at(i)) * a.dy_rs + col, n);
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u)
            if (p + u < len && key[u] < none && key[u] != key[u + 1])
                g[u] = load_raw8<GT>(a.g, static_cast<int64_t>(key[u]) * a.g_rs + col, n);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (p + u >= len || key[u] >= none)
                break;
            float x[8];
            unpack8<YT>(y[u], x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] += x[e];
            const bool ends = key[u] != key[u + 1];
            if (ends && !head) {
                unpack8<GT>(g[u], x);
                add8<GT>(a, key[u], col, n, x, sum);
            } else if ((ends || p + u + 1 == len) && n > 0) {
                store8<HPO_PARAM_FP32>(s.part, (2 * slab + (head ? 0 : 1)) * s.width + col, 8, sum);
            }
            if (ends) {
                head = false;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] = 0.0f;
            }
        }
    }
}

constexpr int kJoinWaves = 8;
constexpr int kJoinAlone = 8;   /* slabs whose parts one wavefront adds up */

/* Sum of the runs' first parts of slabs from .. to - 1, every `step`-th, in order. */
__device__ __forceinline__ void sum_parts(const Slabs& s, int64_t from, int64_t to, int step, int64_t col, bool any, float (&sum)[8])
{
    for (int64_t j = from; j < to; j += step * kFlight) {
        Raw8<HPO_PARAM_FP32> x[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int64_t k = j + u * step;
            x[u] = load_raw8<HPO_PARAM_FP32>(s.part, 2 * (k < to ? k : j) * s.width + col, any && k < to ? 8 : 0);
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            float y[8];
            unpack8<HPO_PARAM_FP32>(x[u], y);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] += y[e];
        }
    }
}

/* The runs that cross borders: a wavefront looks whether one begins in its slab, and adds up the run's parts in
 * order.  Where these are many, the workgroup's wavefronts take every eighth each, and the sums of the eight
 * are added in order. */
template <int GT>
__global__ __launch_bounds__(64 * kJoinWaves) void k_grad_join(EmbedGradArgs a, Slabs s)
{
    __shared__ float other[kJoinWaves][64][8];
    __shared__ int64_t behind[kJoinWaves];   /* of a long run that begins in the wavefront's slab, its end; else 0 */
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t col = (static_cast<int64_t>(blockIdx.y) * 64 + lane) * 8;
    const int n = a.cols - col > 8 ? 8 : static_cast<int>(a.cols - col);   /* <= 0: no columns */
    const int32_t none = static_cast<int32_t>(a.rows);
    const int64_t slab = static_cast<int64_t>(blockIdx.x) * kJoinWaves + wave;
    int64_t last = 0;
    int32_t key = none;
    if (slab + 1 < s.count) {
        const int64_t p0 = slab * s.length, p1 = p0 + s.length;
        const int32_t next = s.key[p1], first = s.key[p0], prev = s.key[p0 > 0 ? p0 - 1 : 0];
        key = s.key[p1 - 1];
        if (key < none && next == key && !(first == key && p0 > 0 && prev == key)) {
            last = slab + 1;
            for (;;) {
                const int64_t j = last + lane;
                const uint64_t on = __ballot(j < s.count && s.key[(j < s.count ? j : s.count - 1) * s.length] == key);
                const int more = on == ~uint64_t{0} ? 64 : __builtin_ctzll(~on);
                last += more;
                if (more < 64)
                    break;
            }
        }
    }
    auto finish = [&](const float (&sum)[8]) {
        if (n <= 0)
            return;
        float x[8], g[8];
        load8<HPO_PARAM_FP32>(s.part, (2 * slab + 1) * s.width + col, 8, x);
        load8<GT>(a.g, static_cast<int64_t>(key) * a.g_rs + col, n, g);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            x[e] += sum[e];
        add8<GT>(a, key, col, n, g, x);
    };
    const bool far = last - slab > kJoinAlone;
    if (lane == 0)
        behind[wave] = far ? last : 0;
    __syncthreads();
    if (last > 0 && !far) {
        float sum[8] = {};
        sum_parts(s, slab + 1, last, 1, col, n > 0, sum);
        finish(sum);
    }
    for (int w = 0; w < kJoinWaves; ++w) {
        const int64_t end = behind[w];
        if (end == 0)
            continue;
        float sum[8] = {};
        sum_parts(s, static_cast<int64_t>(blockIdx.x) * kJoinWaves + w + 1 + wave, end, kJoinWaves, col, n > 0, sum);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            other[wave][lane][e] = sum[e];
        __syncthreads();
        if (wave == w) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum[e] = 0.0f;
#pragma unroll
            for (int v = 0; v < kJoinWaves; ++v)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] += other[v][lane][e];
            finish(sum);
        }
        __syncthreads();
    }
}

/* Tokens up to which no sort is needed: every token looks through all of them.  Without a sort and with it, in
 * microseconds, rows of 4096 elements into 32000 rows, tokens as in text: 16 tokens 4 and 15, 64 8 and 15, 128 14 and 17, 192
 * 21 and 17; rows of 64 elements (eight lanes each): 64 11 and 15, 128 24 and 17.  One token all along is one lane group's
 * work without the sort: 16 7 and 15, 64 20 and 16, 128 39 and 16. */
constexpr int kFewMax = 128;

/* LANES lanes take a token's row: the first token of its kind adds up all of them. */
template <int YT, int GT, int LANES>
__global__ __launch_bounds__(kRowThreads) void k_grad_few(EmbedGradArgs a)
{
    __shared__ int32_t keys[kFewMax];
    const int n_tok = static_cast<int>(a.n);
    if (threadIdx.x < n_tok)
        keys[threadIdx.x] = key_of(a, threadIdx.x);
    __syncthreads();
    const int t = static_cast<int>(blockIdx.x) * (kRowThreads / LANES) + threadIdx.x / LANES;
    const int64_t col = (static_cast<int64_t>(blockIdx.y) * LANES + threadIdx.x % LANES) * 8;
    if (t >= n_tok || col >= a.cols)
        return;
    const int n = a.cols - col > 8 ? 8 : static_cast<int>(a.cols - col);
    const int32_t key = keys[t];
    if (key >= static_cast<int32_t>(a.rows))
        return;
    for (int u = 0; u < t; ++u)
        if (keys[u] == key)
            return;
    float sum[8] = {}, g[8];
    load8<GT>(a.g, static_cast<int64_t>(key) * a.g_rs + col, n, g);
    int u = t;
    while (u < n_tok) {
        float y[kFlight][8];
        int got = 0;
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            while (u < n_tok && keys[u] != key)
                ++u;
            if (u < n_tok) {
                load8<YT>(a.dy, static_cast<int64_t>(u) * a.dy_rs + col, n, y[j]);
                got = j + 1;
                ++u;
            }
        }
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
            if (j < got)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum[e] += y[j][e];
    }
    add8<GT>(a, key, col, n, g, sum);
}

/* ---------------------------------------------------------------------- */
/* launches                                                                */
/* ---------------------------------------------------------------------- */
/* Lanes of a row of `cols`: a power of two up to `most`. */
int lanes_of(int64_t cols, int most)
{
    int l = 8;
    while (l < most && l * 8 < cols)
        l *= 2;
    return l;
}

template <int WT, int OT>
hipError_t embedding(const EmbedArgs& a, hipStream_t stream)
{
    const int lanes = lanes_of(a.cols, 256);
    const dim3 grid(static_cast<uint32_t>((a.n + kRowThreads / lanes - 1) / (kRowThreads / lanes)));
    switch (lanes) {
    case 8: return launch(k_embedding<WT, OT, 8>, grid, kRowThreads, stream, a);
    case 16: return launch(k_embedding<WT, OT, 16>, grid, kRowThreads, stream, a);
    case 32: return launch(k_embedding<WT, OT, 32>, grid, kRowThreads, stream, a);
    case 64: return launch(k_embedding<WT, OT, 64>, grid, kRowThreads, stream, a);
    case 128: return launch(k_embedding<WT, OT, 128>, grid, kRowThreads, stream, a);
    default: return launch(k_embedding<WT, OT, 256>, grid, kRowThreads, stream, a);
    }
}

template <int WT>
hipError_t embedding_out(const EmbedArgs& a, hipStream_t stream)
{
    if (a.out_dtype == HPO_PARAM_BF16)
        return embedding<WT, HPO_PARAM_BF16>(a, stream);
    if (a.out_dtype == HPO_PARAM_FP16)
        return embedding<WT, HPO_PARAM_FP16>(a, stream);
    return embedding<WT, HPO_PARAM_FP32>(a, stream);
}

/* Tokens of a slab: the more the fewer runs cross borders, as long as there are some 6144 wavefronts (6 a
 * SIMD).  The sums and the join of bf16 rows, with operands in the 256 MB cache: 20000 of 1001 take 27 us with slabs of
 * 8 and 34 with 16; 8192 of 4096 44 and 39. */
int32_t slab_length(int64_t n, int64_t cols)
{
    const int64_t pieces = (cols + 511) / 512;
    int32_t l = 8;
    while (l < 64 && (n + l - 1) / l * pieces > 6144)
        l *= 2;
    return l;
}

int64_t pad256(int64_t bytes) { return (bytes + 255) / 256 * 256; }

/* The workspace's parts; returns its size. */
int64_t carve(int64_t n, int64_t cols, void* ws, Sorted* s, Slabs* b)
{
    if (n <= kFewMax)
        return 0;
    const int64_t list = pad256(4 * n), blocks = (n + kBlockTokens - 1) / kBlockTokens;
    const int64_t mid = 2 * list + (n > kBucketMax ? pad256(4 * blocks * kBins) : 0);
    const int32_t length = slab_length(n, cols);
    const int64_t count = (n + length - 1) / length, width = (cols + 7) / 8 * 8;
    const int64_t part = pad256(8 * count * width);
    if (ws) {
        char* p = static_cast<char*>(ws);
        s->key = reinterpret_cast<int32_t*>(p);
        s->tok = reinterpret_cast<int32_t*>(p + list);
        b->part = reinterpret_cast<float*>(p + 2 * list);
        p += 2 * list + part;
        s->key_mid = reinterpret_cast<int32_t*>(p);
        s->tok_mid = reinterpret_cast<int32_t*>(p + list);
        s->hist = reinterpret_cast<int32_t*>(p + 2 * list);
        b->key = s->key;
        b->tok = s->tok;
        b->width = width;
        b->count = count;
        b->length = length;
    }
    return 2 * list + part + mid;
}

/* Sorts the tokens by row of the table. */
hipError_t sort_tokens(const EmbedGradArgs& a, const Sorted& s, hipStream_t stream)
{
    if (a.n <= kBucketMax) {
        int shift = 8;   /* 256 buckets: one workgroup a CU */
        while (((a.rows - 1) >> shift) + 1 > kBucketBins)
            ++shift;
        return launch(k_sort_bucket, dim3(1u << shift), kBucketThreads, stream, a, s, shift);
    }
    int bits = 1;
    while ((a.rows >> bits) != 0)   /* keys are 0 .. rows */
        ++bits;
    const int bits0 = bits <= kDigitBits ? bits : (bits + 1) / 2, bits1 = bits - bits0;
    const dim3 grid(static_cast<uint32_t>((a.n + kBlockTokens - 1) / kBlockTokens));
    hipError_t e = launch(k_sort_count<true>, grid, kSortThreads, stream, a, s, 0, bits0);
    if (e != hipSuccess)
        return e;
    if (bits1 == 0)
        return launch(k_sort_move<true, true>, grid, kSortThreads, stream, a, s, 0, bits0);
    e = launch(k_sort_move<true, false>, grid, kSortThreads, stream, a, s, 0, bits0);
    if (e == hipSuccess)
        e = launch(k_sort_count<false>, grid, kSortThreads, stream, a, s, bits0, bits1);
    if (e == hipSuccess)
        e = launch(k_sort_move<false, true>, grid, kSortThreads, stream, a, s, bits0, bits1);
    return e;
}

template <int YT, int GT, int LANES>
hipError_t embedding_grad(const EmbedGradArgs& a, const Slabs& b, hipStream_t stream)
{
    const uint32_t pieces = static_cast<uint32_t>((a.cols + 8 * LANES - 1) / (8 * LANES));
    constexpr int kPer = kRowThreads / LANES;
    if (a.n <= kFewMax)
        return launch(k_grad_few<YT, GT, LANES>, dim3(static_cast<uint32_t>((a.n + kPer - 1) / kPer), pieces), kRowThreads,
                      stream, a);
    hipError_t e = launch(k_grad_slabs<YT, GT, LANES>, dim3(static_cast<uint32_t>((b.count + kPer - 1) / kPer), pieces),
                          kRowThreads, stream, a, b);
    if (e != hipSuccess || b.count == 1)
        return e;
    return launch(k_grad_join<GT>, dim3(static_cast<uint32_t>((b.count + kJoinWaves - 2) / kJoinWaves),
                                        static_cast<uint32_t>((a.cols + 511) / 512)),
                  64 * kJoinWaves, stream, a, b);
}

template <int YT, int GT>
hipError_t embedding_grad_lanes(const EmbedGradArgs& a, const Slabs& b, hipStream_t stream)
{
    switch (lanes_of(a.cols, 64)) {
    case 8: return embedding_grad<YT, GT, 8>(a, b, stream);
    case 16: return embedding_grad<YT, GT, 16>(a, b, stream);
    case 32: return embedding_grad<YT, GT, 32>(a, b, stream);
    default: return embedding_grad<YT, GT, 64>(a, b, stream);
    }
}

template <int YT>
hipError_t embedding_grad_out(const EmbedGradArgs& a, const Slabs& b, hipStream_t stream)
{
    return a.g_dtype == HPO_PARAM_BF16 ? embedding_grad_lanes<YT, HPO_PARAM_BF16>(a, b, stream)
                                       : embedding_grad_lanes<YT, HPO_PARAM_FP32>(a, b, stream);
}

}  // namespace

hipError_t launch_embedding(const EmbedArgs& a, hipStream_t stream)
{
    switch (a.w_dtype) {
    case HPO_PARAM_BF16: return embedding_out<HPO_PARAM_BF16>(a, stream);
    case HPO_PARAM_FP16: return embedding_out<HPO_PARAM_FP16>(a, stream);
    case HPO_PARAM_FP32: return embedding_out<HPO_PARAM_FP32>(a, stream);
    default: return embedding_out<HPO_WEIGHT_MX8>(a, stream);
    }
}

int64_t embed_grad_workspace(int64_t n, int64_t cols) { return carve(n, cols, nullptr, nullptr, nullptr); }

hipError_t launch_embedding_grad(const EmbedGradArgs& a, hipStream_t stream)
{
    Sorted s{};
    Slabs b{};
    if (carve(a.n, a.cols, a.ws, &s, &b) > 0) {
        const hipError_t e = sort_tokens(a, s, stream);
        if (e != hipSuccess)
            return e;
    }
    switch (a.dy_dtype) {
    case HPO_PARAM_BF16: return embedding_grad_out<HPO_PARAM_BF16>(a, b, stream);
    case HPO_PARAM_FP16: return embedding_grad_out<HPO_PARAM_FP16>(a, b, stream);
    default: return embedding_grad_out<HPO_PARAM_FP32>(a, b, stream);
    }
}

}  // namespace hpo
