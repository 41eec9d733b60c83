// embedding_lookup.cu -- embedding lookup with scaling, and the table's
// gradient by sorted tokens.
//
// Forward: y_i = scale * E[tok_i], one 16-byte vector of y at a time; bound by memory.
//
// Backward: dE[w] = scale * sum over the tokens i with id w of dy_i.
//  1. The (id, position) pairs are sorted by id, stably: a least-significant-
//     digit radix sort, 8 bits a pass, as many passes as the vocabulary needs.
//     Tokens that add nothing (padding, ids outside the table) get the key
//     `vocab` and end up last.  Up to kClusterTokens tokens are sorted by one
//     cluster of CTAs in one launch; more by three launches a pass.  The
//     launches' other CTAs write the zeros of a dE that is not accumulated
//     into; what is more than fits beside a one-launch sort is left to step 2.
//  2. One warp per window of sorted positions and 256 columns walks its
//     positions in order and keeps the running sum of the current id in FP32
//     registers.  An id whose positions all lie in the window is written at
//     once; the sums of ids that cross a window's border go to the workspace.
//  3. For each id that crosses a border, one CTA adds those sums in window order.
// The order of every addition is fixed by the ids, so results repeat bit for
// bit; dy is read once, and the table is written once (the rows of the
// tokens' ids twice: zeros first).
#include <math.h>

#include <algorithm>

#include "vec.cuh"
#include "vocab_internal.h"

namespace ls {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlockCols = 32 * kVec;  // columns of one warp

// --- forward ------------------------------------------------------------------
constexpr int kLookupUnroll = 4;  // vectors of a thread

template <typename I> struct LookupArgs {
    I nvec;       // n * hidden / 8
    int vecs;     // hidden / 8
    FastDiv div;  // by vecs
    int vocab;
    float scale;
};

// Vector i of y belongs to token i / vecs.
template <typename T, typename I>
__global__ void __launch_bounds__(kThreads)
lookup_fwd_kernel(T* __restrict__ y, const int32_t* __restrict__ tokens, const T* __restrict__ table,
                  const __grid_constant__ LookupArgs<I> a) {
    pdl_enter();
    const I i0 = static_cast<I>(blockIdx.x) * (kThreads * kLookupUnroll) + threadIdx.x;
    Raw8<T> r[kLookupUnroll];
    int32_t w[kLookupUnroll];
    uint32_t v[kLookupUnroll];
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
        const I i = i0 + u * kThreads;
        w[u] = -1;
        if (i >= a.nvec) continue;
        I t;
        if constexpr (sizeof(I) == 4)
            t = fdiv(i, a.div);
        else
            t = i / a.vecs;
        v[u] = static_cast<uint32_t>(i - t * a.vecs);
        w[u] = tokens[t];
    }
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u)
        r[u] = w[u] >= 0 && w[u] < a.vocab
                   ? load8<T>(table + (static_cast<int64_t>(w[u]) * a.vecs + v[u]) * kVec)
                   : zero8<T>();
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
        const I i = i0 + u * kThreads;
        if (i >= a.nvec) break;
        float f[kVec];
        unpack(r[u], f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) f[j] *= a.scale;
        store8f<T>(y + static_cast<int64_t>(i) * kVec, f);
    }
}

// --- radix sort ---------------------------------------------------------------
// Sorted pairs: x = id, y = position.
constexpr int kDigits = 256;
constexpr int kItems = 4;                        // keys per thread
constexpr int kSortTile = kThreads * kItems;     // keys per CTA; a warp owns 128 consecutive ones

struct SortArgs {
    int64_t n;
    int shift;
    int blocks;
    int vocab;
    int padding_id;
    bool first;  // pairs come from the tokens, positions are 0..n-1
    // The CTAs behind the tiles write zeros over these 16-byte vectors.
    float* zero;
    int64_t zero_from, zero_to;
};

__device__ __forceinline__ void write_zeros(const SortArgs& a) {
    const int64_t step = static_cast<int64_t>(gridDim.x - a.blocks) * kThreads;
    for (int64_t v = a.zero_from + static_cast<int64_t>(blockIdx.x - a.blocks) * kThreads + threadIdx.x;
         v < a.zero_to; v += step)
        st16(a.zero + v * 4, make_uint4(0, 0, 0, 0));
}

__device__ __forceinline__ int2 sort_pair(const int32_t* tokens, const int2* src, int64_t i, bool first,
                                          int vocab, int padding_id) {
    if (!first) return __ldcg(src + i);  // written by other SMs, maybe in this launch
    const int32_t w = tokens[i];
    return make_int2(w >= 0 && w < vocab && w != padding_id ? w : vocab, static_cast<int>(i));
}

// The lanes that hold this lane's digit (d < 0: none), by a ballot for each
// bit: 8 of them cost a fraction of one match.any.
__device__ __forceinline__ unsigned same_digit(int d) {
    unsigned same = __ballot_sync(0xffffffffu, d >= 0);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const bool bit = (d >> b) & 1;
        const unsigned set = __ballot_sync(0xffffffffu, bit);
        same &= bit ? set : ~set;
    }
    return same;
}
// Places for a warp's 32 digits, in lane order, from its row of next places,
// which move on (-1 takes no place).
__device__ __forceinline__ int place_digit(int* next, int d) {
    const unsigned same = same_digit(d);
    const unsigned lower = same & ((1u << (threadIdx.x & 31)) - 1u);
    int to = 0;
    if (d >= 0) to = next[d];
    __syncwarp();
    if (d >= 0 && lower == 0) next[d] = to + __popc(same);
    __syncwarp();
    return to + __popc(lower);
}

// The whole sort by one cluster (the grid's first), and zeros over d_table by
// the other CTAs of the launch.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxCluster = 8;
// Rounds of 32 keys for a warp.  A round costs a pass about 1 us, whatever the
// CTAs: more than 32768 tokens go to more SMs faster (131072 tokens of 30522
// ids: one cluster 59 us, a launch for each step 44 us).
constexpr int kRounds = 4;
constexpr int64_t kClusterTokens = kMaxCluster * kSortThreads * kRounds;

struct ClusterSortArgs {
    int64_t zero_vecs;  // 16-byte vectors of d_table to write zeros to, from its first row on
    uint32_t* present;  // if given, bit w: some token has the id w
    int n;
    int passes, cluster, rounds;
    int vocab, padding_id;
};

// Shared memory: the CTA's pairs in digit order [rounds * 1024], and counts.
// Pairs leave in that order, so that a warp's stores run along a digit's
// places instead of going to 32 of them.
constexpr int kCountRow = kDigits + 1;  // rows of counts start in different banks
__host__ __device__ constexpr size_t sort_smem(int rounds) {
    return static_cast<size_t>(rounds) * kSortThreads * 8 + kSortWarps * kCountRow * 4;
}

__global__ void __launch_bounds__(kSortThreads)
cluster_sort_kernel(int2* buf0, int2* buf1, const int32_t* __restrict__ tokens, float* d_table,
                    const __grid_constant__ ClusterSortArgs a) {
    extern __shared__ __align__(16) unsigned char sort_mem[];
    int2* stage = reinterpret_cast<int2*>(sort_mem);
    int(*hist)[kCountRow] = reinterpret_cast<int(*)[kCountRow]>(stage + a.rounds * kSortThreads);
    __shared__ int cta_hist[kDigits];
    __shared__ int shift_of[kDigits];  // a digit's places in memory, less those in `stage`
    __shared__ int2 warp_sums[kSortWarps];
    pdl_enter();
    if (blockIdx.x >= a.cluster) {
        const int64_t step = static_cast<int64_t>(gridDim.x - a.cluster) * kSortThreads;
        for (int64_t v = static_cast<int64_t>(blockIdx.x - a.cluster) * kSortThreads + threadIdx.x;
             v < a.zero_vecs; v += step)
            st16(d_table + v * 4, make_uint4(0, 0, 0, 0));
        return;
    }
    const int rank = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile = a.rounds * kSortThreads;
    const int mine = max(0, min(tile, a.n - rank * tile));               // pairs of this CTA
    const int base = rank * tile + warp * a.rounds * 32 + lane;          // a warp's are consecutive
    // Four threads for each digit, each with eight warps' counts.
    const int digit = threadIdx.x >> 2, part = threadIdx.x & 3;
    if (a.present)  // a barrier of every CTA of the cluster follows before the first bit is set
        for (int i = rank * kSortThreads + threadIdx.x; i <= a.vocab / 32; i += a.cluster * kSortThreads)
            a.present[i] = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int2* src = pass & 1 ? buf0 : buf1;
        int2* dst = pass & 1 ? buf1 : buf0;
        const int shift = 8 * pass;
        // One CTA alone finds the last pass's pairs in `stage`.
        const bool staged = a.cluster == 1 && pass > 0;
        auto pair_at = [&](int i) {
            return staged ? stage[i] : sort_pair(tokens, src, i, pass == 0, a.vocab, a.padding_id);
        };
        for (int d = threadIdx.x; d < kSortWarps * kCountRow; d += kSortThreads) (&hist[0][0])[d] = 0;
        __syncthreads();
        // A pair's place among the warp's pairs of the same digit, and the digit (-1: no pair).
        int place[kRounds];
        int2 keep[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = base + r * 32;
            keep[r] = make_int2(-1, 0);
            if (r < a.rounds && i < a.n) keep[r] = pair_at(i);
            place[r] = keep[r].x < 0 ? -1 : (keep[r].x >> shift) & (kDigits - 1);
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (r < a.rounds) {
                const int d = place[r];
                const int to = place_digit(hist[warp], d);
                if (d >= 0) place[r] = to << 8 | d;
            }
        __syncthreads();
        // Exclusive sums over the warps of the CTA ...
        int sum = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += hist[part * 8 + w][digit];
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, inc, o, 4);
            if (part >= o) inc += t;
        }
        const int own = __shfl_sync(0xffffffffu, inc, 3, 4);  // the CTA's count
        int at = inc - sum;
        int lower = 0, total = own;
        if (a.cluster > 1) {
            // ... over the CTAs of the cluster ...
            if (part == 3) cta_hist[digit] = own;
            cluster_sync();
            total = 0;
            for (int c = part; c < a.cluster; c += 4) {
                const int t = __float_as_int(ld_cluster(map_rank(cta_hist + digit, c)));
                if (c < rank) lower += t;
                total += t;
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                lower += __shfl_xor_sync(0xffffffffu, lower, o);
                total += __shfl_xor_sync(0xffffffffu, total, o);
            }
        }
        // ... and over the digits, of the CTA's pairs (x) and of all (y): eight digits in a warp.
        int2 up = make_int2(own, total);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            const int tx = __shfl_up_sync(0xffffffffu, up.x, o), ty = __shfl_up_sync(0xffffffffu, up.y, o);
            if (lane >= o) {
                up.x += tx;
                up.y += ty;
            }
        }
        if (lane == 31) warp_sums[warp] = up;
        __syncthreads();
        int2 before = lane < warp ? warp_sums[lane] : make_int2(0, 0);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            before.x += __shfl_xor_sync(0xffffffffu, before.x, o);
            before.y += __shfl_xor_sync(0xffffffffu, before.y, o);
        }
        const int first = before.x + up.x - own;  // the digit's first place in `stage`
        if (part == 0) shift_of[digit] = before.y + up.y - total + lower - first;
        at += first;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const int c = hist[part * 8 + w][digit];
            hist[part * 8 + w][digit] = at;
            at += c;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (place[r] >= 0) stage[hist[warp][place[r] & 255] + (place[r] >> 8)] = keep[r];
        __syncthreads();
        if (a.cluster > 1 || pass == a.passes - 1)
            for (int j = threadIdx.x; j < mine; j += kSortThreads) {
                const int2 p = stage[j];
                dst[shift_of[(p.x >> shift) & (kDigits - 1)] + j] = p;
                if (a.present && pass == a.passes - 1 && p.x < a.vocab && (j == 0 || stage[j - 1].x != p.x))
                    atomicOr(a.present + p.x / 32, 1u << (p.x & 31));
            }
        if (a.cluster > 1)
            cluster_sync();  // the pairs are there; cta_hist, hist and stage have been read
        else
            __syncthreads();
    }
}

// Per-warp digit counts of the CTA's tile in sm[warp][digit].
__device__ __forceinline__ void count_digits(int (*sm)[kDigits], const int32_t* tokens, const int2* src,
                                             const SortArgs& a) {
    for (int d = threadIdx.x; d < kWarps * kDigits; d += kThreads) (&sm[0][0])[d] = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortTile + warp * (32 * kItems);
    int d[kItems];
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int64_t i = base + r * 32 + lane;
        d[r] = i < a.n ? (sort_pair(tokens, src, i, a.first, a.vocab, a.padding_id).x >> a.shift) & (kDigits - 1) : -1;
    }
#pragma unroll
    for (int r = 0; r < kItems; ++r) place_digit(sm[warp], d[r]);
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads)
sort_count_kernel(int* __restrict__ counts, const int32_t* __restrict__ tokens, const int2* src,
                  const __grid_constant__ SortArgs a) {
    __shared__ int sm[kWarps][kDigits];
    pdl_enter();
    if (blockIdx.x >= a.blocks) return write_zeros(a);
    count_digits(sm, tokens, src, a);
    int t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += sm[w][threadIdx.x];
    counts[static_cast<int64_t>(threadIdx.x) * a.blocks + blockIdx.x] = t;
}

// CTA d: exclusive prefix sums of digit d's counts over the tiles, and their
// total behind the last digit's counts.
__global__ void __launch_bounds__(kThreads) sort_scan_kernel(int* counts, int64_t blocks) {
    __shared__ int sm[kWarps];
    pdl_enter();
    int* row = counts + blockIdx.x * blocks;
    int carry = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t base = 0; base < blocks; base += kThreads) {
        const int64_t i = base + threadIdx.x;
        const int v = i < blocks ? row[i] : 0;
        int inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) sm[warp] = inc;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sm[w];
            all += sm[w];
        }
        if (i < blocks) row[i] = carry + before + inc - v;
        carry += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) counts[kDigits * blocks + blockIdx.x] = carry;
}

__global__ void __launch_bounds__(kThreads)
sort_scatter_kernel(int2* __restrict__ dst, const int* __restrict__ counts,
                    const int32_t* __restrict__ tokens, const int2* src,
                    const __grid_constant__ SortArgs a) {
    __shared__ int sm[kWarps][kDigits];
    __shared__ int warp_sums[kWarps];
    pdl_enter();
    if (blockIdx.x >= a.blocks) return write_zeros(a);
    count_digits(sm, tokens, src, a);
    // The digit's first place: the totals of the smaller digits, and its keys in earlier tiles.
    const int total = counts[static_cast<int64_t>(kDigits) * a.blocks + threadIdx.x];
    int at = counts[static_cast<int64_t>(threadIdx.x) * a.blocks + blockIdx.x];
    int inc = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if ((threadIdx.x & 31) >= o) inc += u;
    }
    if ((threadIdx.x & 31) == 31) warp_sums[threadIdx.x >> 5] = inc;
    __syncthreads();
    at += inc - total;
    for (int w = 0; w < threadIdx.x >> 5; ++w) at += warp_sums[w];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int c = sm[w][threadIdx.x];
        sm[w][threadIdx.x] = at;
        at += c;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortTile + warp * (32 * kItems);
    int2 p[kItems];
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int64_t i = base + r * 32 + lane;
        p[r] = make_int2(-1, 0);
        if (i < a.n) p[r] = sort_pair(tokens, src, i, a.first, a.vocab, a.padding_id);
    }
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int to = place_digit(sm[warp], p[r].x < 0 ? -1 : (p[r].x >> a.shift) & (kDigits - 1));
        if (p[r].x >= 0) dst[to] = p[r];
    }
}

// --- sums ---------------------------------------------------------------------
struct SumArgs {
    int64_t n;
    int64_t windows;
    int window;      // sorted positions of one warp, 8 to 32
    int hidden;
    int vocab;
    int col_blocks;
    float scale;
    bool accumulate;
    // window_sum_kernel: the CTAs behind the first `sum_blocks` write zeros to the rows from zero_row
    // on that no token has.
    int64_t sum_blocks;
    int zero_row;
    const uint32_t* present;
};

__device__ __forceinline__ void put_row(float* d_table, int32_t w, int c, const float (&acc)[kVec],
                                        const SumArgs& a) {
    float* p = d_table + static_cast<int64_t>(w) * a.hidden + c;
    float o[kVec];
    if (a.accumulate) {
        load8f<float>(p, o);
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] = fmaf(acc[j], a.scale, o[j]);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] = acc[j] * a.scale;
    }
    store8f<float>(p, o);
}

// partial: [2][windows][hidden] FP32; row 0 of a window: the sum of its first
// id where that began before the window; row 1: the sum of its last id where
// that begins in the window and goes on behind it.
template <typename T>
__global__ void __launch_bounds__(kThreads)
window_sum_kernel(float* d_table, float* __restrict__ partial, const T* __restrict__ dy,
                  const int2* __restrict__ pairs, const __grid_constant__ SumArgs a) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    if (blockIdx.x >= a.sum_blocks) {
        const int step = static_cast<int>(gridDim.x - a.sum_blocks) * kWarps;
        for (int row = a.zero_row + static_cast<int>(blockIdx.x - a.sum_blocks) * kWarps + (threadIdx.x >> 5);
             row < a.vocab; row += step) {
            if (a.present[row / 32] >> (row & 31) & 1) continue;
            float* p = d_table + static_cast<int64_t>(row) * a.hidden;
            for (int c = lane * 4; c < a.hidden; c += 128) st16(p + c, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t w = item / a.col_blocks;
    if (w >= a.windows) return;
    const int c = static_cast<int>(item - w * a.col_blocks) * kBlockCols + lane * kVec;
    const int64_t base = w * a.window;
    const int count = static_cast<int>(min(static_cast<int64_t>(a.window), a.n - base));
    const int2 pair = lane < count ? pairs[base + lane] : make_int2(a.vocab, 0);
    const int my_key = pair.x, my_pos = pair.y;
    const int before = base > 0 ? pairs[base - 1].x : -1;
    const int behind = base + a.window < a.n ? pairs[base + a.window].x : -1;
    // The valid positions come first.  Bit i of `starts`: position i has another id than i - 1.
    const int valid = __popc(__ballot_sync(0xffffffffu, my_key < a.vocab));
    const int key_before = __shfl_up_sync(0xffffffffu, my_key, 1);
    const unsigned starts = __ballot_sync(0xffffffffu, lane > 0 && my_key != key_before);
    if (valid == 0) return;
    const bool in = c < a.hidden;
    const T* col = dy + c;
    float acc[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) acc[j] = 0.f;
    bool began_before = __shfl_sync(0xffffffffu, my_key, 0) == before;
    // The run that ends before position `end` leaves the registers.
    auto flush = [&](int end, bool goes_on) {
        const int id = __shfl_sync(0xffffffffu, my_key, end - 1);
        if (in) {
            if (began_before)
                store8f<float>(partial + w * a.hidden + c, acc);
            else if (goes_on)
                store8f<float>(partial + (a.windows + w) * a.hidden + c, acc);
            else
                put_row(d_table, id, c, acc, a);
        }
        began_before = false;
#pragma unroll
        for (int j = 0; j < kVec; ++j) acc[j] = 0.f;
    };
    constexpr int U = 8;
    for (int i0 = 0; i0 < valid; i0 += U) {
        Raw8<T> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = __shfl_sync(0xffffffffu, my_pos, i0 + u);
            if (in && i0 + u < valid) r[u] = load8<T>(col + static_cast<int64_t>(p) * a.hidden);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= valid) break;
            if (starts >> (i0 + u) & 1) flush(i0 + u, false);
            float f[kVec];
            unpack(r[u], f);
#pragma unroll
            for (int j = 0; j < kVec; ++j) acc[j] += f[j];
        }
    }
    flush(valid, __shfl_sync(0xffffffffu, my_key, valid - 1) == behind);
}

// acc += the partial sums of windows lo, lo + 1, ... below hi, in order.
__device__ __forceinline__ void add_partials(float (&acc)[kVec], const float* partial, int64_t lo, int64_t hi,
                                             int c, const SumArgs& a) {
    constexpr int U = 4;
    for (int64_t v0 = lo; v0 < hi; v0 += U) {
        Raw8<float> r[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (v0 + u < hi) r[u] = load8<float>(partial + (v0 + u) * a.hidden + c);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (v0 + u >= hi) break;
            float f[kVec];
            unpack(r[u], f);
#pragma unroll
            for (int j = 0; j < kVec; ++j) acc[j] += f[j];
        }
    }
}

// One warp per window and 256 columns: if an id begins in the window and goes
// on behind it, its sum over the windows that hold it.  A warp adds up to
// kAlone windows in order by itself; more are shared out among the CTA's
// warps, equal runs of windows in order, and the runs' sums added in order.
// A CTA's items are neighbouring windows of one column block (blockIdx.y), so
// that it hardly ever has two ids of many windows.
constexpr int kAlone = 16;

__global__ void __launch_bounds__(kThreads, 4)
join_windows_kernel(float* d_table, const float* __restrict__ partial,
                    const int2* __restrict__ pairs, const __grid_constant__ SumArgs a) {
    __shared__ float sm[kWarps][kBlockCols];
    __shared__ int64_t long_more[kWarps];  // 0: this warp's window has nothing left to do
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kWarps;
    const int64_t w = first + warp;
    const int64_t begin = w * a.window, end = begin + a.window;
    const int c0 = blockIdx.y * kBlockCols, c = c0 + lane * kVec;
    int64_t more = 0;  // windows behind w whose first position still has the id: the keys are sorted
    if (end < a.n) {
        const int id = pairs[end - 1].x;
        if (id < a.vocab && pairs[end].x == id && !(w > 0 && pairs[begin - 1].x == id)) {
            for (;;) {
                bool has[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int64_t p = (w + 1 + more + u * 32 + lane) * a.window;
                    has[u] = p < a.n && pairs[p].x == id;
                }
                int here = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) here += __popc(__ballot_sync(0xffffffffu, has[u]));
                more += here;
                if (here < 128) break;
            }
            if (more <= kAlone && c < a.hidden) {
                float acc[kVec];
                load8f<float>(partial + (a.windows + w) * a.hidden + c, acc);
                add_partials(acc, partial, w + 1, w + 1 + more, c, a);
                put_row(d_table, id, c, acc, a);
            }
        }
    }
    if (lane == 0) long_more[warp] = more > kAlone ? more : 0;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) {
        const int64_t n = long_more[i];
        if (n == 0) continue;
        const int64_t wi = first + i;
        const int id = pairs[wi * a.window + a.window - 1].x;
        const int64_t share = (n + kWarps - 1) / kWarps;
        const int64_t lo = min(n, warp * share), hi = min(n, lo + share);
        float acc[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) acc[j] = 0.f;
        if (c < a.hidden) {
            if (warp == 0) load8f<float>(partial + (a.windows + wi) * a.hidden + c, acc);
            add_partials(acc, partial, wi + 1 + lo, wi + 1 + hi, c, a);
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) sm[warp][lane * kVec + j] = acc[j];
        __syncthreads();
        const int col = c0 + threadIdx.x;
        if (col < a.hidden) {
            float s = sm[0][threadIdx.x];
#pragma unroll
            for (int v = 1; v < kWarps; ++v) s += sm[v][threadIdx.x];
            float* p = d_table + static_cast<int64_t>(id) * a.hidden + col;
            *p = a.accumulate ? fmaf(s, a.scale, *p) : s * a.scale;
        }
        __syncthreads();
    }
}

// --- workspace ----------------------------------------------------------------
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

constexpr int64_t kMostPresent = 1 << 20;  // ids with a presence bit: one cluster clears them in no time

struct LookupPlan {
    int64_t n, windows, blocks;
    int passes, window, cluster;          // cluster: CTAs of the one-launch sort, 0 for the other
    int64_t early_rows;                   // rows whose zeros are written beside the sort (the rest: the sums)
    size_t pairs[2], counts, present, partial, bytes;  // byte offsets
    LookupPlan(int64_t tokens, int64_t hidden, int64_t vocab) {
        n = tokens;
        // Short windows where there are few: a window's rows are read one batch after the other.
        window = n <= 8192 ? 8 : n <= 32768 ? 16 : 32;
        windows = (n + window - 1) / window;
        blocks = (n + kSortTile - 1) / kSortTile;
        cluster = 0;
        if (n <= kClusterTokens) {
            cluster = 1;
            while (cluster < kMaxCluster && n > cluster * kRounds * kSortThreads) cluster *= 2;
        }
        passes = 1;
        while (passes < 4 && (vocab >> (8 * passes)) > 0) ++passes;  // keys 0..vocab
        size_t at = 0;
        for (int i = 0; i < 2; ++i) {
            pairs[i] = at;
            at += round16(static_cast<size_t>(n) * 8);
        }
        counts = at;
        if (!cluster) at += round16(static_cast<size_t>(blocks + 1) * kDigits * 4);
        present = at;
        early_rows = vocab;
        // The one-launch sort takes 6 to 16 us; that many bytes of zeros cost nothing beside it.  Where
        // there are more, the rest is left to the launch of the sums, which then has to know the rows
        // that it must not touch (4096 x 1280 of 50257 FP16, the gradient alone: 52.6 us with all of them
        // beside the sort, 47.7).
        const int64_t early =
            ((int64_t{40} << 20) + std::min<int64_t>(n, 8192) * 8192) / (hidden * 4);
        if (cluster && vocab <= kMostPresent && vocab > early + early / 4) {
            early_rows = early;
            at += round16(static_cast<size_t>(vocab / 32 + 1) * 4);
        }
        partial = at;
        at += static_cast<size_t>(2 * windows * hidden) * 4;
        bytes = at;
    }
};

template <typename T>
cudaError_t fwd(void* y, const int32_t* tokens, const void* table, int64_t n, int64_t hidden,
                int64_t vocab, float scale, cudaStream_t s) {
    const int64_t nvec = n * hidden / kVec;
    const int64_t per = kThreads * kLookupUnroll;
    const dim3 grid(static_cast<unsigned>((nvec + per - 1) / per));
    const int vecs = static_cast<int>(hidden / kVec);
    // Indexes of 31 bits (and room to step past the end) divide by a multiplication.
    if (nvec <= (int64_t{1} << 31) - 2 * per) {
        LookupArgs<uint32_t> a{static_cast<uint32_t>(nvec), vecs, make_fastdiv(vecs),
                               static_cast<int>(vocab), scale};
        return launch_pdl(lookup_fwd_kernel<T, uint32_t>, grid, dim3(kThreads), 0, s,
                          static_cast<T*>(y), tokens, static_cast<const T*>(table), a);
    }
    LookupArgs<int64_t> a{nvec, vecs, make_fastdiv(vecs), static_cast<int>(vocab), scale};
    return launch_pdl(lookup_fwd_kernel<T, int64_t>, grid, dim3(kThreads), 0, s,
                      static_cast<T*>(y), tokens, static_cast<const T*>(table), a);
}

template <typename T>
cudaError_t sums(float* d_table, float* partial, const void* dy, const int2* pairs,
                 const SumArgs& a, cudaStream_t s) {
    const int64_t zeros = a.zero_row < a.vocab ? std::min((a.vocab - a.zero_row + kWarps - 1) / kWarps, 2432) : 0;
    return launch_pdl(window_sum_kernel<T>, dim3(static_cast<unsigned>(a.sum_blocks + zeros)), dim3(kThreads),
                      0, s, d_table, partial, static_cast<const T*>(dy), pairs, a);
}

// Pairs sorted by id, by a launch for each step of each pass; each writes its
// share of the table's zeros beside its own work.
cudaError_t sort_in_steps(int2* const (&pairs)[2], int* counts, const int32_t* tokens, float* d_table,
                          int64_t zero_vecs, const LookupPlan& p, int64_t vocab, int32_t padding_id,
                          cudaStream_t s) {
    const int64_t share = (zero_vecs + 2 * p.passes - 1) / (2 * p.passes);
    const int64_t zeros = std::min<int64_t>(608, (share + kThreads - 1) / kThreads);
    const dim3 grid(static_cast<unsigned>(p.blocks + zeros));
    SortArgs a;
    a.n = p.n;
    a.blocks = static_cast<int>(p.blocks);
    a.vocab = static_cast<int>(vocab);
    a.padding_id = padding_id;
    a.zero = d_table;
    a.zero_to = 0;
    auto next_share = [&] {
        a.zero_from = a.zero_to;
        a.zero_to = std::min(zero_vecs, a.zero_from + share);
    };
    for (int pass = 0; pass < p.passes; ++pass) {
        a.shift = 8 * pass;
        a.first = pass == 0;
        const int2* src = pairs[(pass + 1) & 1];
        next_share();
        cudaError_t e = launch_pdl(sort_count_kernel, grid, dim3(kThreads), 0, s, counts, tokens, src, a);
        if (e == cudaSuccess)
            e = launch_pdl(sort_scan_kernel, dim3(kDigits), dim3(kThreads), 0, s, counts, p.blocks);
        next_share();
        if (e == cudaSuccess)
            e = launch_pdl(sort_scatter_kernel, grid, dim3(kThreads), 0, s, pairs[pass & 1], counts,
                           tokens, src, a);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_embedding_lookup_fwd(ls_dtype dt, void* y, const int32_t* tokens,
                                        const void* table, int64_t n, int64_t hidden,
                                        int64_t vocab, float scale, cudaStream_t s) {
    if (dt == LS_F16) return fwd<__half>(y, tokens, table, n, hidden, vocab, scale, s);
    if (dt == LS_BF16) return fwd<bf16>(y, tokens, table, n, hidden, vocab, scale, s);
    return fwd<float>(y, tokens, table, n, hidden, vocab, scale, s);
}

size_t embedding_lookup_workspace_bytes(int64_t tokens, int64_t hidden, int64_t vocab) {
    return LookupPlan(tokens, hidden, vocab).bytes;
}

cudaError_t launch_embedding_lookup_bwd(ls_dtype dt, float* d_table, const void* dy,
                                        const int32_t* tokens, int64_t n, int64_t hidden,
                                        int64_t vocab, float scale, int32_t padding_id,
                                        bool accumulate, void* workspace, cudaStream_t s) {
    const LookupPlan p(n, hidden, vocab);
    char* ws = static_cast<char*>(workspace);
    int2* const pairs[2] = {reinterpret_cast<int2*>(ws + p.pairs[0]),
                            reinterpret_cast<int2*>(ws + p.pairs[1])};
    float* partial = reinterpret_cast<float*>(ws + p.partial);
    const int64_t zero_vecs = accumulate ? 0 : vocab * hidden / 4;
    uint32_t* present = reinterpret_cast<uint32_t*>(ws + p.present);
    cudaError_t e = cudaSuccess;
    if (p.cluster) {
        ClusterSortArgs a;
        a.n = static_cast<int>(n);
        a.rounds = static_cast<int>((n + p.cluster * kSortThreads - 1) / (p.cluster * kSortThreads));
        a.zero_vecs = accumulate ? 0 : p.early_rows * hidden / 4;
        a.present = accumulate || p.early_rows == vocab ? nullptr : present;
        a.passes = p.passes;
        a.cluster = p.cluster;
        a.vocab = static_cast<int>(vocab);
        a.padding_id = padding_id;
        static int done[kMaxDevices];
        e = allow_max_dynamic_smem(cluster_sort_kernel, done);
        if (e != cudaSuccess) return e;
        const int64_t want = (a.zero_vecs + kSortThreads * 4 - 1) / (kSortThreads * 4);
        const int64_t zeros = want < 296 ? want : 296;
        const int64_t grid = p.cluster + (zeros + p.cluster - 1) / p.cluster * p.cluster;
        e = launch_cluster(cluster_sort_kernel, dim3(static_cast<unsigned>(grid)), p.cluster,
                           dim3(kSortThreads), sort_smem(a.rounds), s, pairs[0], pairs[1], tokens, d_table, a);
    } else {
        e = sort_in_steps(pairs, reinterpret_cast<int*>(ws + p.counts), tokens, d_table, zero_vecs, p,
                          vocab, padding_id, s);
    }
    if (e != cudaSuccess) return e;
    const int2* sorted = pairs[(p.passes - 1) & 1];
    SumArgs a;
    a.n = n;
    a.windows = p.windows;
    a.window = p.window;
    a.hidden = static_cast<int>(hidden);
    a.vocab = static_cast<int>(vocab);
    a.col_blocks = static_cast<int>((hidden + kBlockCols - 1) / kBlockCols);
    a.scale = scale;
    a.accumulate = accumulate;
    a.sum_blocks = (a.windows * a.col_blocks + kWarps - 1) / kWarps;
    a.zero_row = static_cast<int>(accumulate ? vocab : p.early_rows);
    a.present = present;
    if (dt == LS_F16) e = sums<__half>(d_table, partial, dy, sorted, a, s);
    else if (dt == LS_BF16) e = sums<bf16>(d_table, partial, dy, sorted, a, s);
    else e = sums<float>(d_table, partial, dy, sorted, a, s);
    if (e != cudaSuccess || p.windows == 1) return e;
    return launch_pdl(join_windows_kernel,
                      dim3(static_cast<unsigned>((p.windows + kWarps - 1) / kWarps),
                           static_cast<unsigned>(a.col_blocks)),
                      dim3(kThreads), 0, s, d_table, partial, sorted, a);
}

}  // namespace ls
