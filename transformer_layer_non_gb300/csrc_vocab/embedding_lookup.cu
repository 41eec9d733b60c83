// embedding_lookup.cu -- embedding lookup with scaling, and the table's
// gradient by sorted tokens.
//
// Forward: y_i = scale * E[tok_i], one warp per token and 256 columns; bound by memory.
//
// Backward: dE[w] = scale * sum over the tokens i with id w of dy_i.
//  1. The (id, position) pairs are sorted by id, stably: a least-significant-
//     digit radix sort, 8 bits a pass, as many passes as the vocabulary needs.
//     Tokens that add nothing (padding, ids outside the table) get the key
//     `vocab` and end up last.
//  2. One warp per window of 32 sorted positions and 256 columns walks its
//     positions in order and keeps the running sum of the current id in FP32
//     registers.  An id whose positions all lie in the window is written at
//     once; the sums of ids that cross a window's border go to the workspace.
//  3. For each id that crosses a border, one CTA adds those sums in window order.
// The order of every addition is fixed by the ids, so results repeat bit for
// bit; the gradient rows dy are read once, and the table is written once.
#include <math.h>

#include "vec.cuh"
#include "vocab_internal.h"

namespace ls {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlockCols = 32 * kVec;  // columns of one warp
constexpr int kWindow = 32;            // sorted positions of one warp

// --- forward ------------------------------------------------------------------
struct LookupArgs {
    int64_t n;
    int hidden;
    int vocab;
    int col_blocks;
    float scale;
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
lookup_fwd_kernel(T* __restrict__ y, const int32_t* __restrict__ tokens, const T* __restrict__ table,
                  const __grid_constant__ LookupArgs a) {
    pdl_enter();
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t i = item / a.col_blocks;
    const int c = static_cast<int>(item - i * a.col_blocks) * kBlockCols + (threadIdx.x & 31) * kVec;
    if (i >= a.n || c >= a.hidden) return;
    const int32_t w = tokens[i];
    float f[kVec];
    if (w >= 0 && w < a.vocab) {
        load8f<T>(table + static_cast<int64_t>(w) * a.hidden + c, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) f[j] *= a.scale;
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) f[j] = 0.f;
    }
    store8f<T>(y + i * a.hidden + c, f);
}

// --- radix sort ---------------------------------------------------------------
constexpr int kDigits = 256;
constexpr int kItems = 8;                        // keys per thread
constexpr int kSortTile = kThreads * kItems;     // keys per CTA; a warp owns 256 consecutive ones

struct SortArgs {
    int64_t n;
    int shift;
    int blocks;
    int vocab;
    int padding_id;
    bool first;  // keys come from the tokens, positions are 0..n-1
};

__device__ __forceinline__ int sort_key(const int32_t* src, int64_t i, const SortArgs& a) {
    const int32_t w = src[i];
    if (!a.first) return w;
    return (w >= 0 && w < a.vocab && w != a.padding_id) ? w : a.vocab;
}

// Per-warp digit counts of the CTA's tile in sm[warp][digit].
__device__ __forceinline__ void count_digits(int (*sm)[kDigits], const int32_t* src,
                                             const SortArgs& a) {
    for (int d = threadIdx.x; d < kWarps * kDigits; d += kThreads) (&sm[0][0])[d] = 0;
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortTile + warp * (32 * kItems);
#pragma unroll
    for (int r = 0; r < kItems; ++r) {
        const int64_t i = base + r * 32 + lane;
        const int d = i < a.n ? (sort_key(src, i, a) >> a.shift) & (kDigits - 1) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, d);
        if (d >= 0 && lane == __ffs(same) - 1) sm[warp][d] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads)
sort_count_kernel(int* __restrict__ counts, const int32_t* __restrict__ src,
                  const __grid_constant__ SortArgs a) {
    __shared__ int sm[kWarps][kDigits];
    pdl_enter();
    count_digits(sm, src, a);
    int t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += sm[w][threadIdx.x];
    counts[static_cast<int64_t>(threadIdx.x) * a.blocks + blockIdx.x] = t;
}

// Exclusive prefix sum of the counts, digit-major, by one CTA.
__global__ void __launch_bounds__(1024) sort_scan_kernel(int* counts, int64_t total) {
    __shared__ int sm[32];
    pdl_enter();
    int carry = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t base = 0; base < total; base += 1024) {
        const int64_t i = base + threadIdx.x;
        const int v = i < total ? counts[i] : 0;
        int inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
        if (lane == 31) sm[warp] = inc;
        __syncthreads();
        int before = 0, all = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < warp) before += sm[w];
            all += sm[w];
        }
        if (i < total) counts[i] = carry + before + inc - v;
        carry += all;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads)
sort_scatter_kernel(int32_t* __restrict__ dst_key, int32_t* __restrict__ dst_pos,
                    const int* __restrict__ counts, const int32_t* __restrict__ src_key,
                    const int32_t* __restrict__ src_pos, const __grid_constant__ SortArgs a) {
    __shared__ int sm[kWarps][kDigits];
    pdl_enter();
    count_digits(sm, src_key, a);
    int at = counts[static_cast<int64_t>(threadIdx.x) * a.blocks + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int c = sm[w][threadIdx.x];
        sm[w][threadIdx.x] = at;
        at += c;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortTile + warp * (32 * kItems);
    for (int r = 0; r < kItems; ++r) {
        const int64_t i = base + r * 32 + lane;
        const int key = i < a.n ? sort_key(src_key, i, a) : 0;
        const int d = i < a.n ? (key >> a.shift) & (kDigits - 1) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, d);
        const int leader = __ffs(same) - 1;
        int to = 0;
        if (d >= 0 && lane == leader) {
            to = sm[warp][d];
            sm[warp][d] = to + __popc(same);
        }
        to = __shfl_sync(0xffffffffu, to, leader) + __popc(same & ((1u << lane) - 1u));
        if (d >= 0) {
            dst_key[to] = key;
            dst_pos[to] = a.first ? static_cast<int32_t>(i) : src_pos[i];
        }
        __syncwarp();
    }
}

// --- sums ---------------------------------------------------------------------
struct SumArgs {
    int64_t n;
    int64_t windows;
    int hidden;
    int vocab;
    int col_blocks;
    float scale;
    bool accumulate;
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
                  const int32_t* __restrict__ key, const int32_t* __restrict__ pos,
                  const __grid_constant__ SumArgs a) {
    pdl_enter();
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t w = item / a.col_blocks;
    if (w >= a.windows) return;
    const int lane = threadIdx.x & 31;
    const int c = static_cast<int>(item - w * a.col_blocks) * kBlockCols + lane * kVec;
    const int64_t base = w * kWindow;
    const int count = static_cast<int>(min(static_cast<int64_t>(kWindow), a.n - base));
    const int my_key = lane < count ? key[base + lane] : a.vocab;
    const int my_pos = lane < count ? pos[base + lane] : 0;
    const int before = base > 0 ? key[base - 1] : -1;
    const int behind = base + kWindow < a.n ? key[base + kWindow] : -1;
    float acc[kVec];
    int cur = -1;
    bool began_before = false;
    for (int i0 = 0; i0 < count; i0 += 8) {
        Raw8<T> r[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int k = __shfl_sync(0xffffffffu, my_key, i0 + u);
            const int p = __shfl_sync(0xffffffffu, my_pos, i0 + u);
            if (k < a.vocab && c < a.hidden)
                r[u] = load8<T>(dy + static_cast<int64_t>(p) * a.hidden + c);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int k = __shfl_sync(0xffffffffu, my_key, i0 + u);
            if (k >= a.vocab) break;  // the rest adds nothing
            if (k != cur) {
                if (cur >= 0 && c < a.hidden) {
                    if (began_before)
                        store8f<float>(partial + w * a.hidden + c, acc);
                    else
                        put_row(d_table, cur, c, acc, a);
                }
                began_before = cur < 0 && k == before;
                cur = k;
#pragma unroll
                for (int j = 0; j < kVec; ++j) acc[j] = 0.f;
            }
            if (c < a.hidden) {
                float f[kVec];
                unpack(r[u], f);
#pragma unroll
                for (int j = 0; j < kVec; ++j) acc[j] += f[j];
            }
        }
    }
    if (cur < 0 || c >= a.hidden) return;
    if (began_before)
        store8f<float>(partial + w * a.hidden + c, acc);
    else if (cur == behind)
        store8f<float>(partial + (a.windows + w) * a.hidden + c, acc);
    else
        put_row(d_table, cur, c, acc, a);
}

// CTA (window, column block): if an id begins in the window and goes on behind
// it, its sum: warp v adds the v-th of kWarps equal shares of the windows that
// hold it, in order, then the shares are added in order.
__global__ void __launch_bounds__(kThreads)
join_windows_kernel(float* d_table, const float* __restrict__ partial,
                    const int32_t* __restrict__ key, const __grid_constant__ SumArgs a) {
    __shared__ float sm[kWarps][kBlockCols];
    pdl_enter();
    const int64_t w = blockIdx.x;
    const int64_t last = w * kWindow + kWindow - 1;
    if (last + 1 >= a.n) return;
    const int id = key[last];
    if (id >= a.vocab || key[last + 1] != id) return;
    // began in this window?
    if (w > 0 && key[w * kWindow] == id && key[w * kWindow - 1] == id) return;
    // The windows behind it whose first position still has the id: the keys are sorted.
    int64_t more = 0;
    for (;;) {
        const int64_t p = (w + 1 + more + threadIdx.x) * kWindow;
        const int here = __syncthreads_count(p < a.n && key[p] == id);
        more += here;
        if (here < kThreads) break;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t share = (more + kWarps - 1) / kWarps;
    const int64_t lo = min(more, warp * share), hi = min(more, lo + share);
    for (int cb = blockIdx.y; cb < a.col_blocks; cb += gridDim.y) {
        const int c = cb * kBlockCols + lane * kVec;
        float acc[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) acc[j] = 0.f;
        if (c < a.hidden) {
            if (warp == 0) load8f<float>(partial + (a.windows + w) * a.hidden + c, acc);
#pragma unroll 4
            for (int64_t v = lo; v < hi; ++v) {
                float f[kVec];
                load8f<float>(partial + (w + 1 + v) * a.hidden + c, f);
#pragma unroll
                for (int j = 0; j < kVec; ++j) acc[j] += f[j];
            }
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) sm[warp][lane * kVec + j] = acc[j];
        __syncthreads();
        const int t = threadIdx.x;
        const int col = cb * kBlockCols + t;
        if (col < a.hidden) {
            float s = sm[0][t];
#pragma unroll
            for (int v = 1; v < kWarps; ++v) s += sm[v][t];
            float* p = d_table + static_cast<int64_t>(id) * a.hidden + col;
            *p = a.accumulate ? fmaf(s, a.scale, *p) : s * a.scale;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kThreads) zero_kernel(float* p, int64_t nvec) {
    pdl_enter();
    for (int64_t v = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; v < nvec;
         v += static_cast<int64_t>(gridDim.x) * kThreads)
        st16(p + v * 4, make_uint4(0, 0, 0, 0));
}

// --- workspace ----------------------------------------------------------------
size_t round16(size_t n) { return (n + 15) / 16 * 16; }

struct LookupPlan {
    int64_t n, windows, blocks;
    int passes;
    size_t key[2], pos[2], counts, partial, bytes;  // byte offsets
    LookupPlan(int64_t tokens, int64_t hidden, int64_t vocab) {
        n = tokens;
        windows = (n + kWindow - 1) / kWindow;
        blocks = (n + kSortTile - 1) / kSortTile;
        passes = 1;
        while (passes < 4 && (vocab >> (8 * passes)) > 0) ++passes;  // keys 0..vocab
        size_t at = 0;
        for (int i = 0; i < 2; ++i) {
            key[i] = at;
            at += round16(static_cast<size_t>(n) * 4);
            pos[i] = at;
            at += round16(static_cast<size_t>(n) * 4);
        }
        counts = at;
        at += round16(static_cast<size_t>(blocks) * kDigits * 4);
        partial = at;
        at += static_cast<size_t>(2 * windows * hidden) * 4;
        bytes = at;
    }
};

template <typename T>
cudaError_t fwd(void* y, const int32_t* tokens, const void* table, int64_t n, int64_t hidden,
                int64_t vocab, float scale, cudaStream_t s) {
    LookupArgs a;
    a.n = n;
    a.hidden = static_cast<int>(hidden);
    a.vocab = static_cast<int>(vocab);
    a.col_blocks = static_cast<int>((hidden + kBlockCols - 1) / kBlockCols);
    a.scale = scale;
    const int64_t items = n * a.col_blocks;
    return launch_pdl(lookup_fwd_kernel<T>, dim3(static_cast<unsigned>((items + kWarps - 1) / kWarps)),
                      dim3(kThreads), 0, s, static_cast<T*>(y), tokens,
                      static_cast<const T*>(table), a);
}

template <typename T>
cudaError_t sums(float* d_table, float* partial, const void* dy, const int32_t* key,
                 const int32_t* pos, const SumArgs& a, cudaStream_t s) {
    const int64_t items = a.windows * a.col_blocks;
    return launch_pdl(window_sum_kernel<T>,
                      dim3(static_cast<unsigned>((items + kWarps - 1) / kWarps)), dim3(kThreads), 0,
                      s, d_table, partial, static_cast<const T*>(dy), key, pos, a);
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
    int32_t* key[2] = {reinterpret_cast<int32_t*>(ws + p.key[0]),
                       reinterpret_cast<int32_t*>(ws + p.key[1])};
    int32_t* pos[2] = {reinterpret_cast<int32_t*>(ws + p.pos[0]),
                       reinterpret_cast<int32_t*>(ws + p.pos[1])};
    int* counts = reinterpret_cast<int*>(ws + p.counts);
    float* partial = reinterpret_cast<float*>(ws + p.partial);
    cudaError_t e = cudaSuccess;
    if (!accumulate) {
        const int64_t nvec = vocab * hidden / 4;
        const int64_t blocks = (nvec + kThreads - 1) / kThreads;
        e = launch_pdl(zero_kernel, dim3(static_cast<unsigned>(blocks < 152 * 8 ? blocks : 152 * 8)),
                       dim3(kThreads), 0, s, d_table, nvec);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(static_cast<unsigned>(p.blocks));
    for (int pass = 0; pass < p.passes; ++pass) {
        SortArgs a;
        a.n = n;
        a.shift = 8 * pass;
        a.blocks = static_cast<int>(p.blocks);
        a.vocab = static_cast<int>(vocab);
        a.padding_id = padding_id;
        a.first = pass == 0;
        const int32_t* src_key = pass == 0 ? tokens : key[(pass + 1) & 1];
        const int32_t* src_pos = pos[(pass + 1) & 1];
        e = launch_pdl(sort_count_kernel, grid, dim3(kThreads), 0, s, counts, src_key, a);
        if (e != cudaSuccess) return e;
        e = launch_pdl(sort_scan_kernel, dim3(1), dim3(1024), 0, s, counts, p.blocks * kDigits);
        if (e != cudaSuccess) return e;
        e = launch_pdl(sort_scatter_kernel, grid, dim3(kThreads), 0, s, key[pass & 1],
                       pos[pass & 1], counts, src_key, src_pos, a);
        if (e != cudaSuccess) return e;
    }
    const int32_t* skey = key[(p.passes - 1) & 1];
    const int32_t* spos = pos[(p.passes - 1) & 1];
    SumArgs a;
    a.n = n;
    a.windows = p.windows;
    a.hidden = static_cast<int>(hidden);
    a.vocab = static_cast<int>(vocab);
    a.col_blocks = static_cast<int>((hidden + kBlockCols - 1) / kBlockCols);
    a.scale = scale;
    a.accumulate = accumulate;
    if (dt == LS_F16) e = sums<__half>(d_table, partial, dy, skey, spos, a, s);
    else if (dt == LS_BF16) e = sums<bf16>(d_table, partial, dy, skey, spos, a, s);
    else e = sums<float>(d_table, partial, dy, skey, spos, a, s);
    if (e != cudaSuccess || p.windows == 1) return e;
    return launch_pdl(join_windows_kernel,
                      dim3(static_cast<unsigned>(p.windows), static_cast<unsigned>(a.col_blocks)),
                      dim3(kThreads), 0, s, d_table, partial, skey, a);
}

}  // namespace ls
