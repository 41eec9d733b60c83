// linear_ce.cu -- the output projection fused with its softmax cross entropy,
// in pieces of the vocabulary, without keeping the logits.
//
// Forward: tiles of z = x W^T are computed and reduced at once to a maximum, a
// sum of exponentials and a plain sum per row and tile; a second kernel merges
// a row's tiles (the online softmax rule) into lse and loss.
// Backward, one piece of the vocabulary after the other: the piece's z again,
// g = dloss (exp(z - lse) - (1 - eps) [j == y] - eps / V) rounded to the
// storage type in the workspace, then dx += g W_piece and dW_piece = g^T x.
//
// All three products run in one kernel (head_kernel) on tcgen05: persistent
// pairs of CTAs, each pair a tile of 256 x 256 (z also narrower) with FP32 accumulators in tensor
// memory (two of them, so that one is read while the other is filled), operands
// brought by TMA through a ring of 64-wide K blocks.  Warp 0 issues the copies,
// warp 1 of the pair's first CTA the products, the other warps take the accumulators
// to the statistics, to g or to the outputs.  A pair, because a CTA on its own
// needs 48 KB of operands for the 128 x 256 x 64 products that take it 512
// cycles, more than the L2 gives an SM; each of a pair needs 32 KB.
//
// Operands of which M or N is the contiguous axis (W in g W; g and x in g^T x)
// are read as they lie in memory: the matrix descriptors take either order.
//
// g is stored divided by D = max|dloss| (1 - eps), and the FP32 sums are
// multiplied by D again.  The entries at the targets, which carry most of a
// row's gradient, are then near -1, which both formats hold exactly; dloss
// itself (1/rows, say) would be off by the same half step in every row, and
// with it the whole gradient.  FP16, which has no exponent range for 1/rows
// times 1/vocab, also gets a factor of 2^14.
#include <cuda.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "tc.cuh"
#include "vocab_internal.h"

namespace ls {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// exp(z - m) = 2^(z log2(e) - m log2(e)) by one FMA as long as the rounding of m log2(e), at most 2^-24 of it,
// is harmless: below 2^17 it is at most 2^-8, less than the rounding of the row's FP32 lse.  At 1e10 it is
// hundreds, and the exponential of the maximum itself, which is 1, would be infinite or 0.
constexpr float kMostFma = 131072.f;

constexpr int kTileM = 256;   // of a pair; 128 rows for each CTA
constexpr int kTileN = 256;
constexpr int kBlockK = 64;   // 128 bytes: the swizzle's row
constexpr int kStages = 5;
constexpr int kEpilogueWarps = 8;  // two for each quarter of the tensor memory's lanes, half the columns each
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kWarpBoxes = 2;      // a warp's store boxes: one is filled while the other is on its way
constexpr uint32_t kOperandBytes = 128 * kBlockK * 2;          // one operand of one CTA and stage
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr uint32_t kStoreBytes = 32 * 128;                     // one warp's store box
constexpr uint32_t kTmemColumns = 512;
constexpr uint32_t kSmemBytes = 1024 + kStages * kStageBytes + kEpilogueWarps * kWarpBoxes * kStoreBytes;
constexpr int kGroupM = 16;   // row tiles that share a sweep over the vocabulary
constexpr int kPairs = 76;    // pairs of SMs; a constant, so that plans depend on the shapes alone

enum Mode { kStats = 0, kGrad = 1, kOut = 2 };

struct HeadArgs {
    int rows, vocab, hidden;
    int col0, cols;        // this piece of the vocabulary
    int m_tiles, n_tiles;  // kStats, kGrad: rows x piece
    int tile_n;            // kStats, kGrad: columns of a tile, a multiple of 32 (kStats), 128 or 256 (kGrad)
    int warp_columns;      // and of the first of its two warps in a quarter of the lanes, a multiple of 32
    int row_box;           // rows of the copies of x and g with rows as M: 128, or all where there are fewer
    int k_blocks;
    float eps;
    int32_t ignore_index;
    // kOut
    int slices;            // of the piece's columns (K of dx, M of dweight)
    int x_units, w_units;  // units of dx and of dweight in a slice
    int units;             // in all
    int x_m_tiles, h_tiles;
    int x_k_blocks, slice_blocks;
    int w_kb0, w_k_blocks;  // the rows that dweight's sums run over in this launch
    int w_row;              // row of `out2` that the piece's first entry has
    bool by_slice, w_first, x_partial, x_add, w_f32;
    bool w_partial, w_add;  // dweight's sums go to FP32 scratch, without the scale; they are added to what is there
    // kStats
    int parts;             // partial statistics of a row: two for each tile, or one for each CTA
    float2* part;          // [rows][parts]: maximum, sum of exponentials
    float* part_sum;       // [rows][parts]: sum
    float* zy;             // [rows]
    const int32_t* target;
    const float* lse;
    const float* dloss;
    float* scale;          // [2] in the workspace: g's factor and its inverse, if dloss is given
    float2 fixed_scale;    // the same if not
    bool find_scale;       // kGrad: from dloss, by every CTA (and left in `scale`), while the first tile's products run
    const void* x;         // kGrad: copied to used_x, if that is given, with zeros for the rows that are
    void* used_x;          //        not used: what they hold (a NaN, say) stays out of g^T x
};

// g's factor and its inverse for the largest finite |dloss| of the rows that are used.
template <typename T> __host__ __device__ __forceinline__ float2 scale_for(float largest, float eps) {
    const float up = std::is_same<T, __half>::value ? 16384.f : 1.f;
    // 1 - eps is left out where p / (1 - eps) would leave FP16's range.
    float d = largest * (eps <= 0.5f ? 1.f - eps : 1.f);
    if (!(d > 0x1p-100f)) d = largest > 0.f ? 0x1p-100f : 1.f;
    return make_float2(up / d, d / up);
}
__device__ __forceinline__ float2 scale_of(const HeadArgs& a) {
    return a.dloss ? make_float2(a.scale[0], a.scale[1]) : a.fixed_scale;
}

struct HeadMaps {
    CUtensorMap a, b;    // kStats, kGrad: x, W;  kOut: g, W for dx
    CUtensorMap a2, b2;  // kOut: g, x for dweight
    CUtensorMap out, out2;
};

__device__ __forceinline__ bool used_target(int32_t y, const HeadArgs& a) {
    return y != a.ignore_index && y >= 0 && y < a.vocab;
}

// One unit of work of a pair.
struct Unit {
    int m0, n0;        // first row and column of the tile
    int kb0, kbs;      // K blocks
    int slice;
    bool weight;       // kOut: a tile of dweight
};

template <int MODE> __device__ __forceinline__ Unit unit_of(int u, const HeadArgs& a) {
    Unit t;
    t.weight = false;
    t.slice = 0;
    t.kb0 = 0;
    if constexpr (MODE != kOut) {
        const int g = u / (kGroupM * a.n_tiles);
        const int first = g * kGroupM;
        const int gm = min(kGroupM, a.m_tiles - first);
        const int r = u - first * a.n_tiles;
        t.n0 = (r / gm) * a.tile_n;
        t.m0 = (first + r % gm) * kTileM;
        t.kbs = a.k_blocks;
    } else {
        int r = u;
        if (!a.by_slice) {  // all of one, then all of the other
            const int x_all = a.slices * a.x_units, first = a.w_first ? a.units - x_all : x_all;
            t.weight = (r >= first) != a.w_first;
            if (r >= first) r -= first;
            if (!t.weight) {
                t.slice = r / a.x_units;
                r -= t.slice * a.x_units;
            }
        } else {
            // One slice of g after the other, for dx and then for dweight, so that the second reading
            // finds it in L2; the last slice, which may be narrower, first: it was written last.
            const int first = a.units - (a.slices - 1) * (a.x_units + a.w_units);
            int q = 0;
            if (u >= first) {
                q = (u - first) / (a.x_units + a.w_units);
                r = u - first - q * (a.x_units + a.w_units);
                ++q;
            }
            t.slice = a.slices - 1 - q;
            t.weight = r >= a.x_units;
            if (t.weight) r -= a.x_units;
        }
        t.kb0 = t.slice * a.slice_blocks;
        t.n0 = (r % a.h_tiles) * kTileN;
        t.m0 = (r / a.h_tiles) * kTileM;
        if (t.weight) {
            t.m0 += t.kb0 * kBlockK;
            t.kb0 = a.w_kb0;
            t.kbs = a.w_k_blocks;
        } else {
            t.kbs = min(a.slice_blocks, a.x_k_blocks - t.kb0);
        }
    }
    return t;
}
template <int MODE> __device__ __forceinline__ int units_of(const HeadArgs& a) {
    return MODE == kOut ? a.units : a.m_tiles * a.n_tiles;
}

// Bounded wait of a converged warp; false (and the failure flagged for the CTA
// and the host) when it runs out.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead,
                                         uint32_t polls = kWaitPolls) {
    for (uint32_t i = 0; i < polls; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 63) == 63 && __any_sync(0xffffffffu, *dead)) return false;
    }
    flag_device_error(kDevErrWaitTimeout);
    *dead = 1;
    return false;
}

// 16 bytes `c` of a lane's 128-byte row in a swizzled store box.
__device__ __forceinline__ void put16(unsigned char* box, int lane, int c, uint4 v) {
    st16(box + lane * 128 + ((c ^ (lane & 7)) << 4), v);
}

// Statistics of 32 logits of one row: n of them exist (n >= 1).
template <bool EDGE, bool SUM>
__device__ __forceinline__ void add_stats(float (&z)[32], int n, float& m, float2& l, float2& s) {
    if constexpr (SUM) {
#pragma unroll
        for (int j = 0; j < 32; j += 2)
            s = add2(s, make_float2(EDGE && j >= n ? 0.f : z[j], EDGE && j + 1 >= n ? 0.f : z[j + 1]));
    }
    if constexpr (EDGE) {
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = j < n ? z[j] : -INFINITY;
    }
    float c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = fmaxf(fmaxf(z[j], z[j + 8]), fmaxf(z[j + 16], z[j + 24]));
    const float cm = fmaxf(fmaxf(fmaxf(c[0], c[1]), fmaxf(c[2], c[3])),
                           fmaxf(fmaxf(c[4], c[5]), fmaxf(c[6], c[7])));
    if (cm > m) {
        const float f = exp2_approx((m - cm) * kLog2e);
        l = mul2(l, make_float2(f, f));
        m = cm;
    }
    float mc = m == -INFINITY ? 0.f : -m * kLog2e;  // nothing but -inf (or NaN) so far
    if (fabsf(mc) > kMostFma) {  // the difference first
        mc = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] -= m;
    }
    const float2 cc = make_float2(kLog2e, kLog2e), mm = make_float2(mc, mc);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 t = fma2(make_float2(z[j], z[j + 1]), cc, mm);
        l = add2(l, make_float2(exp2_approx(t.x), exp2_approx(t.y)));
    }
}

// 32 values of a row of g: d (exp(z - lse) - q0 - [j == at] (1 - eps)).  FAR: some row of the warp has an lse
// too far from zero for one FMA (ml = -lse log2(e)).
template <bool HIT, bool FAR>
__device__ __forceinline__ void grads_of(float (&z)[32], float d, float lse, float ml, float q0, float qy, int at) {
    if constexpr (FAR) {
        if (fabsf(ml) > kMostFma) {  // the difference first; it is at most 0 but for the rounding of z and lse
            ml = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = z[j] > lse ? 0.f : z[j] - lse;
        }
    }
    const float2 cc = make_float2(kLog2e, kLog2e), mm = make_float2(ml, ml);
    const float2 dd = make_float2(d, d), dq = make_float2(-d * q0, -d * q0);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        const float2 t = fma2(make_float2(z[j], z[j + 1]), cc, mm);
        float2 p = make_float2(exp2_approx(t.x), exp2_approx(t.y));
        if constexpr (HIT) {  // subtracted before the product with d: p is near 1 there
            if (at == j) p.x -= qy;
            if (at == j + 1) p.y -= qy;
        }
        p = fma2(p, dd, dq);
        z[j] = p.x;
        z[j + 1] = p.y;
    }
}

template <typename T> __device__ __forceinline__ uint4 pack8(const float (&z)[32], int j, float sc) {
    return make_uint4(pack2<T>(z[j] * sc, z[j + 1] * sc), pack2<T>(z[j + 2] * sc, z[j + 3] * sc),
                      pack2<T>(z[j + 4] * sc, z[j + 5] * sc), pack2<T>(z[j + 6] * sc, z[j + 7] * sc));
}

// f(c, z) for the warp's four groups of 32 accumulator columns, the next group
// on its way while f works; release() once all of them are in registers.
template <typename R, typename F>
__device__ __forceinline__ void sweep(uint32_t cols, R&& release, F&& f) {
    float za[32], zb[32];
    tmem_ld32(za, cols);
    tmem_ld_wait(za);
    tmem_ld32(zb, cols + 32);
    f(0, za);
    tmem_ld_wait(zb);
    tmem_ld32(za, cols + 64);
    f(1, zb);
    tmem_ld_wait(za);
    tmem_ld32(zb, cols + 96);
    f(2, za);
    tmem_ld_wait(zb);
    release();
    f(3, zb);
}

// kGrad has two more warps, which write used_x.
template <int MODE> constexpr int threads_of() { return MODE == kGrad ? kThreads + 64 : kThreads; }

template <typename T, int MODE, bool SUM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of<MODE>(), 1)
head_kernel(const __grid_constant__ HeadMaps maps, const __grid_constant__ HeadArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    __shared__ float largest[kEpilogueWarps];
    // The swizzle's pattern repeats every 1024 bytes of the address.
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int units = units_of<MODE>(a);
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        dead = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(&drained, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + s, 1);
            mbar_init(acc_empty + s, 2 * kEpilogueWarps);
        }
        mbar_init_fence();
        prefetch_map(&maps.a);
        prefetch_map(&maps.b);
    }
    if (warp == 1) tmem_alloc(&tmem_at, kTmemColumns);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    pdl_enter();

    // The copying and the multiplying warp stay converged: all lanes wait, one elected lane issues.
    if (warp == 0) {
        uint32_t it = 0;
        for (int u = pair; u < units; u += pairs) {
            const Unit t = unit_of<MODE>(u, a);
            const int b_rows = MODE == kOut ? 128 : a.tile_n / 2;
            const int m = t.m0 + static_cast<int>(rank) * 128, n = t.n0 + static_cast<int>(rank) * b_rows;
            // Rows behind the last one are not copied (filling them with zeros costs a copy of 1 row
            // 10 us in 40): what the shared memory holds there reaches rows of the accumulator that
            // nothing reads.
            auto a_bytes = [&](int first) -> uint32_t {
                return t.weight ? kOperandBytes : first < a.rows ? static_cast<uint32_t>(a.row_box) * 128 : 0;
            };
            const uint32_t bytes = 2 * b_rows * 128 + a_bytes(t.m0) + a_bytes(t.m0 + 128);  // of both CTAs
            const bool has_a = a_bytes(m) > 0;
            for (int kb = 0; kb < t.kbs; ++kb, ++it) {
                const uint32_t s = it % kStages;
                if (!wait_bar(empty + s, ((it / kStages) & 1) ^ 1, &dead)) break;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(full + s, bytes);
                    const uint32_t bar = map_rank(full + s, 0);
                    unsigned char* pa = smem + s * kStageBytes;
                    unsigned char* pb = pa + kOperandBytes;
                    const int k = (t.kb0 + kb) * kBlockK;
                    if constexpr (MODE != kOut) {
                        if (has_a) tma_load_2d(pa, &maps.a, k, m, bar);
                        tma_load_2d(pb, &maps.b, k, a.col0 + n, bar);
                    } else if (!t.weight) {
                        if (has_a) tma_load_2d(pa, &maps.a, k, m, bar);
                        tma_load_2d(pb, &maps.b, n, a.col0 + k, bar);
                        tma_load_2d(pb + kOperandBytes / 2, &maps.b, n + 64, a.col0 + k, bar);
                    } else {
                        tma_load_2d(pa, &maps.a2, m, k, bar);
                        tma_load_2d(pa + kOperandBytes / 2, &maps.a2, m + 64, k, bar);
                        tma_load_2d(pb, &maps.b2, n, k, bar);
                        tma_load_2d(pb + kOperandBytes / 2, &maps.b2, n + 64, k, bar);
                    }
                }
                __syncwarp();
            }
            if (dead) break;
        }
        // After a failed wait: the copies in flight land before the CTA ends.
        if (dead && rank == 0)
            for (uint32_t s = 0; s < kStages && s < it; ++s) {
                const uint32_t uses = (it - 1 - s) / kStages;  // its last use, counted from 0
                for (uint32_t i = 0; i < kWaitPolls; ++i)
                    if (mbar_try_wait(full + s, uses & 1)) break;
            }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr bool kBf16 = std::is_same<T, bf16>::value;
            const uint64_t kmajor = desc_base(16), mnmajor = desc_base(kOperandBytes / 2);
            uint32_t it = 0, tile = 0;
            for (int u = pair; u < units; u += pairs, ++tile) {
                const Unit t = unit_of<MODE>(u, a);
                const uint32_t acc = tile & 1;
                if (!wait_bar(acc_empty + acc, ((tile >> 1) & 1) ^ 1, &dead)) break;
                tc_fence_after();
                // Which operands have M or N as their contiguous axis.
                const bool a_mn = MODE == kOut && t.weight, b_mn = MODE == kOut;
                const uint32_t idesc = instr_desc(kBf16, a_mn, b_mn, kTileM, MODE == kOut ? kTileN : a.tile_n);
                const uint64_t da = desc_at(a_mn ? mnmajor : kmajor, smem_u32(smem));
                const uint64_t db = desc_at(b_mn ? mnmajor : kmajor, smem_u32(smem) + kOperandBytes);
                // 16 values of K further on, in the descriptors' units of 16 bytes
                const uint32_t step_a = a_mn ? 128 : 2, step_b = b_mn ? 128 : 2;
                const uint32_t d = tmem + acc * kTileN;
                for (int kb = 0; kb < t.kbs; ++kb, ++it) {
                    const uint32_t s = it % kStages;
                    if (!wait_bar(full + s, (it / kStages) & 1, &dead)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = s * (kStageBytes >> 4);
#pragma unroll
                        for (int k = 0; k < kBlockK / 16; ++k)
                            tc_mma(d, da + (at + k * step_a), db + (at + k * step_b), idesc, kb + k > 0);
                        tc_commit(empty + s);
                    }
                    __syncwarp();
                }
                if (dead) break;
                if (elect_one()) tc_commit(acc_full + acc);
                __syncwarp();
            }
            if (dead) {  // the products in flight end before their operands' memory is given back
                if (elect_one()) tc_commit(&drained);
                __syncwarp();
                for (uint32_t i = 0; i < kWaitPolls; ++i)
                    if (mbar_try_wait(&drained, 0)) break;
            }
        }
        __syncwarp();
    } else if (MODE == kGrad && warp >= kThreads / 32) {
        const T* x = static_cast<const T*>(a.x);
        T* used_x = static_cast<T*>(a.used_x);
        if (used_x)
            for (int row = blockIdx.x * 2 + warp - kThreads / 32; row < a.rows; row += 2 * gridDim.x) {
                const bool used = used_target(a.target[row], a);
                const int64_t first = static_cast<int64_t>(row) * a.hidden;
                for (int c = lane * kVec; c < a.hidden; c += 32 * kVec)
                    store8<T>(used_x + first + c, used ? load8<T>(x + first + c) : zero8<T>());
            }
    } else {
        const int quad = warp & 3;          // the TMEM lanes this warp may read
        const int part = (warp - 2) >> 2;   // its part of the tile's columns
        unsigned char* const boxes = smem + kStages * kStageBytes + (warp - 2) * kWarpBoxes * kStoreBytes;
        unsigned char* box = boxes;
        uint32_t opened = 0;
        const int warp_n0 = part * (MODE == kOut ? kTileN / 2 : a.warp_columns);  // this warp's first column
        const int warp_n = MODE == kOut ? kTileN / 2 : part ? a.tile_n - a.warp_columns : a.warp_columns;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + warp_n0;
        uint32_t tile = 0;
        float2 scale = make_float2(1.f, 1.f);
        if constexpr (MODE == kGrad) {
            if (a.find_scale) {  // while the first tile's products run
                const int id = threadIdx.x - 64;
                float m = 0.f;
                for (int i = id; i < a.rows; i += 32 * kEpilogueWarps) {
                    const float d = fabsf(a.dloss[i]);
                    if (d < INFINITY && used_target(a.target[i], a)) m = fmaxf(m, d);
                }
                m = group_max<32>(m);
                if (lane == 0) largest[warp - 2] = m;
                asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpilogueWarps) : "memory");
                m = largest[0];
#pragma unroll
                for (int w = 1; w < kEpilogueWarps; ++w) m = fmaxf(m, largest[w]);
                scale = scale_for<T>(m, a.eps);
                if (blockIdx.x == 0 && id == 0) {
                    a.scale[0] = scale.x;
                    a.scale[1] = scale.y;
                }
            } else {
                scale = scale_of(a);
            }
        }
        if constexpr (MODE == kOut) scale = scale_of(a);
        for (int u = pair; u < units; u += pairs, ++tile) {
            const Unit t = unit_of<MODE>(u, a);
            const uint32_t acc = tile & 1;
            const int row0 = t.m0 + static_cast<int>(rank) * 128 + quad * 32;  // this warp's first row
            const int row = row0 + lane;
            const int n0 = t.n0 + warp_n0;                                     // and column
            // The row's values, on their way while the products end.
            const bool there = row < a.rows;
            int32_t y = -1;
            float row_lse = 0.f, row_dloss = 1.f;
            if (MODE != kOut && there) {
                y = a.target[row];
                if constexpr (MODE == kGrad) {
                    row_lse = a.lse[row];
                    if (a.dloss) row_dloss = a.dloss[row];
                }
            }
            if (!wait_bar(acc_full + acc, (tile >> 1) & 1, &dead)) break;
            tc_fence_after();
            const uint32_t cols = lanes + acc * kTileN;
            auto release = [&]() {  // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_rank(acc_empty + acc, 0));
            };
            // The next store box, free to be written; and on its way to memory.
            auto open_box = [&]() {
                box = boxes + (opened++ % kWarpBoxes) * kStoreBytes;
                if (lane == 0) bulk_wait_read<kWarpBoxes - 1>();
                __syncwarp();
            };
            auto close_box = [&](auto&& store) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    store();
                    bulk_commit();
                }
            };
            if constexpr (MODE == kStats) {
                const int n = min(a.cols - n0, warp_n);  // columns that exist
                const int at = used_target(y, a) && y - n0 < n ? y - n0 : -1;
                float m = -INFINITY;
                float2 l = make_float2(0.f, 0.f), s = make_float2(0.f, 0.f);
                sweep(cols, release, [&](int c, float (&z)[32]) {
                    const int rel = at - c * 32;
                    if (__any_sync(0xffffffffu, rel >= 0 && rel < 32)) {
                        float zy = 0.f;
#pragma unroll
                        for (int j = 0; j < 32; ++j) zy = rel == j ? z[j] : zy;
                        if (rel >= 0 && rel < 32) a.zy[row] = zy;
                    }
                    if (c * 32 + 32 <= n)
                        add_stats<false, SUM>(z, 32, m, l, s);
                    else if (c * 32 < n)
                        add_stats<true, SUM>(z, n - c * 32, m, l, s);
                });
                if (row < a.rows) {
                    const int64_t o = static_cast<int64_t>(row) * a.parts + t.n0 / a.tile_n * 2 + part;
                    a.part[o] = make_float2(m, l.x + l.y);
                    if constexpr (SUM) a.part_sum[o] = s.x + s.y;
                }
            } else if constexpr (MODE == kGrad) {
                const int n = min(a.cols - n0, warp_n);
                const bool used = there && used_target(y, a);
                const int at = used ? y - a.col0 - n0 : -1;
                const float d = used ? row_dloss * scale.x : 0.f;
                const float ml = -row_lse * kLog2e;
                const float q0 = a.eps / static_cast<float>(a.vocab), qy = 1.f - a.eps;
                auto columns = [&](int c, float (&z)[32], auto far) {
                    constexpr bool kFar = decltype(far)::value;
                    if (c * 32 >= n) return;
                    if ((c & 1) == 0) open_box();
                    const int rel = at - c * 32;
                    if (kFar || __any_sync(0xffffffffu, rel >= 0 && rel < 32))
                        grads_of<true, kFar>(z, d, row_lse, ml, q0, qy, rel);
                    else
                        grads_of<false, kFar>(z, d, row_lse, ml, q0, qy, rel);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 v = pack8<T>(z, 8 * j, 1.f);
                        put16(box, lane, (c & 1) * 4 + j, used ? v : make_uint4(0, 0, 0, 0));
                    }
                    if ((c & 1) == 1 || c * 32 + 32 >= n)
                        close_box([&] {
                            if (row0 < a.rows) tma_store_2d(&maps.out, n0 + (c & ~1) * 32, row0, box);
                        });
                };
                // Code of its own for rows far from zero, so that it is not fetched with the others'.
                if (__any_sync(0xffffffffu, fabsf(ml) > kMostFma))
                    sweep(cols, release, [&](int c, float (&z)[32]) { columns(c, z, std::true_type{}); });
                else
                    sweep(cols, release, [&](int c, float (&z)[32]) { columns(c, z, std::false_type{}); });
            } else {
                const bool f32 = t.weight ? a.w_f32 || a.w_partial : a.x_partial;
                const float sc = (t.weight ? a.w_partial : a.x_partial) ? 1.f : scale.y;
                const int n = a.hidden - n0;
                const bool stores = row0 < (t.weight ? a.cols : a.rows);
                if (f32)
                    sweep(cols, release, [&](int c, float (&z)[32]) {
                        if (c * 32 >= n) return;
                        open_box();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            put16(box, lane, j,
                                  f2u4(make_float4(z[4 * j] * sc, z[4 * j + 1] * sc, z[4 * j + 2] * sc,
                                                   z[4 * j + 3] * sc)));
                        close_box([&] {
                            if (stores && t.weight && a.w_add)
                                tma_add_2d(&maps.out2, n0 + c * 32, a.w_row + row0, box);
                            else if (stores && t.weight)
                                tma_store_2d(&maps.out2, n0 + c * 32, a.w_row + row0, box);
                            else if (stores && a.x_add)
                                tma_add_3d(&maps.out, n0 + c * 32, row0, t.slice, box);
                            else if (stores)
                                tma_store_3d(&maps.out, n0 + c * 32, row0, t.slice, box);
                        });
                    });
                else
                    sweep(cols, release, [&](int c, float (&z)[32]) {
                        if (c * 32 >= n) return;
                        if ((c & 1) == 0) open_box();
#pragma unroll
                        for (int j = 0; j < 4; ++j) put16(box, lane, (c & 1) * 4 + j, pack8<T>(z, 8 * j, sc));
                        if ((c & 1) == 1 || c * 32 + 32 >= n)
                            close_box([&] {
                                if (stores && t.weight)
                                    tma_store_2d(&maps.out2, n0 + (c & ~1) * 32, a.w_row + row0, box);
                                else if (stores)
                                    tma_store_2d(&maps.out, n0 + (c & ~1) * 32, row0, box);
                            });
                    });
            }
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    if (warp == 1) tmem_free(tmem, kTmemColumns);
}

// Self-test of the waits' failure path: two warps wait, as those of head_kernel do, on a barrier that expects
// an arrival nobody makes; the first whose polls run out flags the failure, the other one sees it.
__global__ void __launch_bounds__(64) wait_selftest_kernel(uint32_t polls) {
    __shared__ uint64_t bar;
    __shared__ volatile int dead;
    if (threadIdx.x == 0) {
        dead = 0;
        mbar_init(&bar, 1);
        mbar_init_fence();
    }
    __syncthreads();
    wait_bar(&bar, 0, &dead, polls);
}

// (m, l) <- the maximum and the sum of exponentials of two sets of logits.
__device__ __forceinline__ void merge_stats(float& m, float& l, float m2, float l2) {
    const float mm = fmaxf(m, m2);
    if (mm == -INFINITY) {  // both empty (or NaN)
        l += l2;
        return;
    }
    l = l * exp2_approx((m - mm) * kLog2e) + l2 * exp2_approx((m2 - mm) * kLog2e);
    m = mm;
}

// Statistics of a single row (scoring one token): bound by reading W once.
// Each warp goes through an equal run of W's rows, two at a time, 16 bytes a
// lane, against x in shared memory; FP32 products and sums.  The loads run
// ahead over the rows' ends, so that they never wait for a row's reduction.
// Measured with the merging at 50257 x 1280 BF16: 24 us (a 256-row tile 28),
// at 128000 x 4096 150 (172; 7.0 TB/s), at 30522 x 768 12.8; four rows and two
// columns in flight are as fast, 12 or 16 vectors in flight slower.  Two rows
// of x are no faster this way than in a tile.
constexpr int kOneThreads = 256;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kOneCtas = 456;               // three on each SM
constexpr int kOneRows = 2, kOneSlots = 4;  // a lane's loads in flight: vectors of so many rows of W, so often
constexpr int64_t kOneHidden = (48 << 9) - 256;  // x in the 48 KB that every launch may have, less the warps' sums

template <typename T>
__global__ void __launch_bounds__(kOneThreads, 3)
one_row_kernel(const T* __restrict__ x, const T* __restrict__ w, const __grid_constant__ HeadArgs a) {
    extern __shared__ __align__(16) unsigned char one_mem[];
    T* xs = reinterpret_cast<T*>(one_mem);
    __shared__ float sm_m[kOneWarps], sm_l[kOneWarps], sm_s[kOneWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int vecs = a.hidden / kVec;
    pdl_enter();
    const int64_t all = gridDim.x * kOneWarps, id = blockIdx.x * kOneWarps + warp;
    const int end = static_cast<int>((id + 1) * a.vocab / all);
    int j0 = static_cast<int>(id * a.vocab / all);
    const int columns = (vecs + 31) / 32;  // vectors of a row for a lane
    // The columns of the groups of rows, one after the other: each is loaded into the place of the one that
    // has just been used, kOneSlots columns ahead, the next group's too.
    Raw8<T> r[kOneSlots][kOneRows];
    int load_j = j0, load_v = lane;
    auto load = [&](int slot) {
#pragma unroll
        for (int q = 0; q < kOneRows; ++q)
            r[slot][q] = load_j < end && load_v < vecs
                             ? load8<T>(w + static_cast<int64_t>(min(load_j + q, end - 1)) * a.hidden + load_v * kVec)
                             : zero8<T>();
        load_v += 32;
        if (load_v - lane >= columns * 32) {
            load_v = lane;
            load_j += kOneRows;
        }
    };
#pragma unroll
    for (int u = 0; u < kOneSlots; ++u) load(u);
    for (int v = threadIdx.x; v < vecs; v += kOneThreads) store8<T>(xs + v * kVec, load8<T>(x + v * kVec));
    for (int v = vecs + threadIdx.x; v < columns * 32; v += kOneThreads) store8<T>(xs + v * kVec, zero8<T>());
    __syncthreads();
    const int32_t y = a.target[0];
    const bool used = used_target(y, a);
    float m = -INFINITY, l = 0.f, s = 0.f;
    float z[kOneRows] = {};
    for (int v = 0; j0 < end;) {
#pragma unroll
        for (int u = 0; u < kOneSlots; ++u) {
            float h[kVec];
            unpack(load8<T>(xs + (v * 32 + lane) * kVec), h);
#pragma unroll
            for (int q = 0; q < kOneRows; ++q) {
                float g[kVec];
                unpack(r[u][q], g);
#pragma unroll
                for (int j = 0; j < kVec; ++j) z[q] = fmaf(g[j], h[j], z[q]);
            }
            load(u);
            if (++v < columns) continue;
            v = 0;
#pragma unroll
            for (int q = 0; q < kOneRows; ++q) z[q] = group_sum<32>(z[q]);
#pragma unroll
            for (int q = 0; q < kOneRows; ++q) {
                if (j0 + q >= end) break;
                if (used && y == j0 + q && lane == 0) a.zy[0] = z[q];
                merge_stats(m, l, z[q], 1.f);
                if (z[q] != z[q]) l = z[q];  // a NaN, which no maximum shows
                s += z[q];
            }
            j0 += kOneRows;
#pragma unroll
            for (int q = 0; q < kOneRows; ++q) z[q] = 0.f;
        }
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
        sm_s[warp] = s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int v = 1; v < kOneWarps; ++v) {
            merge_stats(m, l, sm_m[v], sm_l[v]);
            s += sm_s[v];
        }
        a.part[blockIdx.x] = make_float2(m, l);
        a.part_sum[blockIdx.x] = s;
    }
}

// One warp per row: the row's partial statistics merged.
__global__ void __launch_bounds__(256)
merge_stats_kernel(float* __restrict__ loss, float* __restrict__ lse_out, const __grid_constant__ HeadArgs a) {
    pdl_enter();
    const int row = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (row >= a.rows) return;
    const float2* part = a.part + static_cast<int64_t>(row) * a.parts;
    const float* part_sum = a.part_sum + static_cast<int64_t>(row) * a.parts;
    float m = -INFINITY, l = 0.f, s = 0.f;
    constexpr int U = 16;  // loads in flight
    for (int t0 = lane; t0 < a.parts; t0 += 32 * U) {
        float2 p[U];
        float q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool there = t0 + 32 * u < a.parts;
            p[u] = there ? part[t0 + 32 * u] : make_float2(-INFINITY, 0.f);
            q[u] = there && a.eps > 0.f ? part_sum[t0 + 32 * u] : 0.f;
        }
        float mm = m;
#pragma unroll
        for (int u = 0; u < U; ++u) mm = fmaxf(mm, p[u].x);
        const float mc = mm == -INFINITY ? 0.f : mm;  // nothing but -inf (or NaN sums) so far
        l *= exp2_approx((m - mc) * kLog2e);
        m = mm;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            l += p[u].y * exp2_approx((p[u].x - mc) * kLog2e);
            s += q[u];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
        merge_stats(m, l, m2, l2);
        s += __shfl_xor_sync(0xffffffffu, s, o);
    }
    if (lane != 0) return;
    const float lse = m + logf(l);
    if (lse_out) lse_out[row] = lse;
    float v = 0.f;
    if (used_target(a.target[row], a)) {
        v = (1.f - a.eps) * (lse - a.zy[row]);
        if (a.eps > 0.f) v += a.eps * (lse - s / static_cast<float>(a.vocab));
    }
    loss[row] = v;
}

// scale_for the largest finite |dloss| of many rows.
template <typename T>
__global__ void __launch_bounds__(1024) grad_scale_kernel(const __grid_constant__ HeadArgs a) {
    __shared__ float sm[32];
    pdl_enter();
    float m = 0.f;
    for (int i = threadIdx.x; i < a.rows; i += 1024) {
        const float d = fabsf(a.dloss[i]);
        if (d < INFINITY && used_target(a.target[i], a)) m = fmaxf(m, d);
    }
    m = group_max<32>(m);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = group_max<32>(sm[threadIdx.x]);
        if (threadIdx.x == 0) {
            const float2 f = scale_for<T>(m, a.eps);
            a.scale[0] = f.x;
            a.scale[1] = f.y;
        }
    }
}

// dx (or a piece of dweight) = scale * sum over the slices' partial sums, in slice order.
template <typename T>
__global__ void __launch_bounds__(256)
join_slices_kernel(T* __restrict__ dx, const float* __restrict__ part, int slices, int64_t nvec,
                   const __grid_constant__ HeadArgs a) {
    pdl_enter();
    const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (v >= nvec) return;
    const float sc = scale_of(a).y;
    float acc[kVec];
    load8f<float>(part + v * kVec, acc);
    for (int s = 1; s < slices; ++s) {
        float f[kVec];
        load8f<float>(part + (s * nvec + v) * kVec, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) acc[j] += f[j];
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) acc[j] *= sc;
    store8f<T>(dx + v * kVec, acc);
}

// --- host ----------------------------------------------------------------------
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Pieces: g for `cols` vocabulary entries at a time, at most about 128 MB of it
// (never fewer than 2048 entries).
constexpr int64_t kPieceBytes = int64_t{128} << 20;
constexpr int64_t kMaxSlices = 16;
constexpr int64_t kSliceBytes = int64_t{64} << 20;
// Tensor cores drop low bits as they accumulate: a sum of terms of one sign loses about 5.6e-9 of itself for
// each of them (measured: 2^17 rows 5.7e-4, 2^20 6.5e-3, 2^24 0.10).  No accumulator adds up more than these;
// what it has then is added, rounded, in FP32.  16384 rows lose 9e-5, 32768 columns 1.8e-4, an FP16 half step
// being 4.9e-4.
constexpr int64_t kMostRows = 16384;
constexpr int64_t kMostColumns = 32768;
// The plan below counts time in K blocks of a pair's tile (256 x 256 x 64
// products, about 0.25 us).  A launch costs about kLaunchBlocks of them until
// its tiles run and until the last is written, a unit about one.
constexpr int64_t kLaunchBlocks = 24;

// Columns of the forward's tiles.  One or two tiles of rows get fewer than 256 where the busiest pair has
// less to do that way: a K block's time goes with the columns down to 128, and a unit costs about one K block
// more (8 x 1280 of 50257: three rounds of 256 columns 27.5 us, of 224 26.7; 130 x 264 of 4099: 17 tiles 7.9,
// 65 of 64 columns 7.4).  More rows lose more by reading x for each tile (1024 x 768 of 30522: 30 -> 34).
int stats_columns(int64_t rows, int64_t hidden, int64_t vocab) {
    if (rows > 2 * kTileM) return kTileN;
    const int64_t m_tiles = ceil_div(rows, kTileM), k_blocks = ceil_div(hidden, kBlockK);
    int best_n = kTileN;
    int64_t best = INT64_MAX;
    for (int n = kTileN; n >= 64; n -= 32) {
        const int64_t t = ceil_div(m_tiles * ceil_div(vocab, n), kPairs) * ((std::max(n, 128) + 8) * k_blocks + n + 256);
        if (t < best) {
            best = t;
            best_n = n;
        }
    }
    return best_n;
}
// Columns of the tiles of g: 128 where that takes no pair a second one (130 x 264 of 4099, both gradients:
// 17.5 -> 16.1 us; 333 x 512 of 32000, seven rounds for four: 46 -> 50).
int grad_columns(int64_t rows, int64_t cols) {
    return ceil_div(rows, kTileM) * ceil_div(cols, kTileN / 2) <= kPairs ? kTileN / 2 : kTileN;
}

// Sizes and workspace layout; they depend on the shapes alone.
struct HeadPlan {
    int stats_n;                           // columns of the forward's tiles
    int64_t cols, pieces;                  // columns of a piece (the last may have fewer)
    int64_t slices, slice_blocks;          // dx: K blocks of a piece per slice
    size_t part, part_sum, zy, scale, g, used_x, partial, w_partial, fwd_bytes, bytes;
    bool partial_dx;
    bool by_slice, w_first;                // the order of kOut's units
    HeadPlan(int64_t rows, int64_t hidden, int64_t vocab) {
        stats_n = stats_columns(rows, hidden, vocab);
        const int64_t n_tiles = ceil_div(vocab, stats_n);
        const size_t parts = static_cast<size_t>(rows == 1 ? std::max<int64_t>(2 * n_tiles, kOneCtas) : rows * 2 * n_tiles);
        part = 0;
        part_sum = round256(parts * 8);
        zy = part_sum + round256(parts * 4);
        fwd_bytes = zy + static_cast<size_t>(rows) * 4;

        // The number of pieces, and of slices that cut dx's long K (the vocabulary) into units about
        // as long as dweight's (K is the rows): those whose tiles deal out evenly to the pairs.
        const int64_t most =
            std::min(kMaxSlices * kMostColumns, std::max<int64_t>(2048, kPieceBytes / 2 / rows / kTileN * kTileN));
        const int64_t fewest = ceil_div(vocab, most);
        const int64_t m_tiles = ceil_div(rows, kTileM), h_tiles = ceil_div(hidden, kTileN);
        const int64_t row_blocks = ceil_div(rows, kBlockK), h_blocks = ceil_div(hidden, kBlockK);
        int64_t best = INT64_MAX;
        for (int64_t n = fewest; n <= fewest + (fewest > 1 ? 4 : 0); ++n) {
            const int64_t c = ceil_div(ceil_div(vocab, n), kTileN) * kTileN;
            const int64_t np = ceil_div(vocab, c), kb = ceil_div(std::min(c, vocab), kBlockK);
            const int64_t grad = ceil_div(m_tiles * (c / kTileN), kPairs) * (h_blocks + 1);
            // Where g has left L2 before it is read again, at about 1.1 TB/s of what the products hide.
            const int64_t g_bytes = rows * std::min(c, vocab) * 2;
            const int64_t reread = g_bytes > kSliceBytes ? g_bytes >> 22 : 0;
            for (int64_t s = 1; s <= std::min(kb, kMaxSlices); ++s) {
                const int64_t len = ceil_div(ceil_div(kb, s), kTileM / kBlockK) * (kTileM / kBlockK);
                if (ceil_div(kb, len) != s || len * kBlockK > kMostColumns) continue;
                // Units of dx (a slice's K blocks long) and of dweight (the rows'), dealt to the pairs in turn.
                const int64_t x_units = s * m_tiles * h_tiles, w_units = (c / kTileM) * h_tiles;
                const int64_t x_len = std::min(len, kb) + 1 + (s > 1 || np > 1), w_len = row_blocks + 1;
                const int64_t units = x_units + w_units;
                // The longer ones first: what the pair with the most of it gets.
                const bool longer_w = w_len > x_len;
                const int64_t n_first = longer_w ? w_units : x_units;
                int64_t out = 0;
                for (const int64_t p : {int64_t{0}, n_first % kPairs, units % kPairs}) {
                    const int64_t n = n_first / kPairs + (p < n_first % kPairs);
                    const int64_t rest = units / kPairs + (p < units % kPairs) - n;
                    out = std::max(out, n * std::max(x_len, w_len) + rest * std::min(x_len, w_len));
                }
                out += reread;
                // Or slice by slice: no more than this.
                const int64_t sliced = ceil_div(units, kPairs) * std::max(x_len, w_len);
                const bool interleaved = s > 1 && reread > 0 && sliced < out;
                if (interleaved) out = sliced;
                // joining the slices: their bytes at about 1.7 MB for a K block's time
                const int64_t join = s > 1 || np > 1 ? 12 + s * rows * hidden * 4 / 1700000 : 0;
                const int64_t t = np * (grad + out + 2 * kLaunchBlocks) + join;
                if (t < best) {
                    best = t;
                    cols = c;
                    pieces = np;
                    slices = s;
                    slice_blocks = len;
                    by_slice = interleaved;
                    w_first = longer_w;
                }
            }
        }
        partial_dx = slices > 1 || pieces > 1;
        scale = 0;
        g = 256;
        used_x = g + round256(static_cast<size_t>(rows * cols) * 2);
        partial = used_x + round256(static_cast<size_t>(rows * hidden) * 2);
        w_partial = partial + (partial_dx ? static_cast<size_t>(slices * rows * hidden) * 4 : 0);
        const size_t bwd = w_partial + (rows > kMostRows ? static_cast<size_t>(cols * hidden) * 4 : 0);
        bytes = std::max(fwd_bytes, bwd);
    }
};

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                               cudaEnableDefault, &r);
        return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(p) : nullptr;
    }();
    return fn;
}

// A row-major [depth][outer][inner] tensor in boxes of [1][box_outer][128 bytes].
template <typename E>
cudaError_t make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld, int box_outer,
                     int64_t depth = 0) {
    const EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const CUtensorMapDataType type = std::is_same<E, float>::value  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : std::is_same<E, bf16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t size = sizeof(E);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer),
                                static_cast<cuuint64_t>(depth)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * size,
                                   static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(outer) * size};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(box_outer), 1};
    const cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = fn(map, type, depth ? 3 : 2, const_cast<void*>(base), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <typename T, int MODE, bool SUM>
cudaError_t launch_head(const HeadMaps& maps, const HeadArgs& a, int64_t units, cudaStream_t s) {
    static int done[kMaxDevices];
    cudaError_t e = allow_max_dynamic_smem(head_kernel<T, MODE, SUM>, done);
    if (e != cudaSuccess) return e;
    const int64_t pairs = std::min<int64_t>(units, kPairs);
    return launch_pdl(head_kernel<T, MODE, SUM>, dim3(static_cast<unsigned>(2 * pairs)), dim3(threads_of<MODE>()), kSmemBytes,
                      s, maps, a);
}

HeadArgs make_args(const HeadShape& sh, const int32_t* target) {
    HeadArgs a = {};
    a.rows = static_cast<int>(sh.rows);
    a.vocab = static_cast<int>(sh.vocab);
    a.hidden = static_cast<int>(sh.hidden);
    a.cols = a.vocab;
    a.m_tiles = static_cast<int>(ceil_div(sh.rows, kTileM));
    a.k_blocks = static_cast<int>(ceil_div(sh.hidden, kBlockK));
    a.row_box = static_cast<int>(std::min<int64_t>(sh.rows, 128));
    a.eps = sh.eps;
    a.ignore_index = sh.ignore_index;
    a.target = target;
    return a;
}

// Tiles of z with n columns, over the piece.
void set_tiles(HeadArgs& a, int n) {
    a.tile_n = n;
    a.warp_columns = (n / 2 + 31) / 32 * 32;
    a.n_tiles = static_cast<int>(ceil_div(a.cols, n));
}

#define LS_CUDA(expr)                        \
    do {                                     \
        const cudaError_t _e = (expr);       \
        if (_e != cudaSuccess) return _e;    \
    } while (0)

template <typename T>
cudaError_t fwd(float* loss, float* lse, const void* x, const void* w, const int32_t* target, const HeadShape& sh,
                void* workspace, cudaStream_t s) {
    const HeadPlan p(sh.rows, sh.hidden, sh.vocab);
    char* ws = static_cast<char*>(workspace);
    HeadArgs a = make_args(sh, target);
    a.part = reinterpret_cast<float2*>(ws + p.part);
    a.part_sum = reinterpret_cast<float*>(ws + p.part_sum);
    a.zy = reinterpret_cast<float*>(ws + p.zy);
    if (sh.rows == 1 && sh.hidden <= kOneHidden) {
        a.parts = static_cast<int>(std::min<int64_t>(kOneCtas, ceil_div(sh.vocab, kOneWarps)));
        LS_CUDA(launch_pdl(one_row_kernel<T>, dim3(static_cast<unsigned>(a.parts)), dim3(kOneThreads),
                           static_cast<size_t>(ceil_div(sh.hidden, 32 * kVec)) * 32 * kVec * 2, s, static_cast<const T*>(x),
                           static_cast<const T*>(w), a));
        return launch_pdl(merge_stats_kernel, dim3(1), dim3(256), 0, s, loss, lse, a);
    }
    set_tiles(a, p.stats_n);
    a.parts = 2 * a.n_tiles;
    HeadMaps maps = {};
    LS_CUDA(make_map<T>(&maps.a, x, sh.hidden, sh.rows, sh.hidden, a.row_box));
    LS_CUDA(make_map<T>(&maps.b, w, sh.hidden, sh.vocab, sh.hidden, a.tile_n / 2));
    const int64_t units = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
    if (sh.eps > 0.f)
        LS_CUDA((launch_head<T, kStats, true>(maps, a, units, s)));
    else
        LS_CUDA((launch_head<T, kStats, false>(maps, a, units, s)));
    return launch_pdl(merge_stats_kernel, dim3(static_cast<unsigned>(ceil_div(sh.rows, 8))), dim3(256), 0, s, loss,
                      lse, a);
}

template <typename T>
cudaError_t bwd(void* dx, void* dweight, bool f32_dweight, const void* x, const void* w, const int32_t* target,
                const float* lse, const float* dloss, const HeadShape& sh, void* workspace, cudaStream_t s) {
    const HeadPlan p(sh.rows, sh.hidden, sh.vocab);
    char* ws = static_cast<char*>(workspace);
    T* g = reinterpret_cast<T*>(ws + p.g);
    float* partial = reinterpret_cast<float*>(ws + p.partial);
    HeadArgs a = make_args(sh, target);
    a.lse = lse;
    a.dloss = dloss;
    a.scale = reinterpret_cast<float*>(ws + p.scale);
    a.fixed_scale = scale_for<T>(1.f, sh.eps);
    // Up to this many rows each CTA of the first piece looks for the scale itself, before it reads its first
    // accumulator (16384 rows: 6 us, a launch for it 4 to 6; 4096: 1); the other pieces find it in `scale`.
    const bool find_scale = dloss && sh.rows <= 16384;
    if (dloss && !find_scale)
        LS_CUDA(launch_pdl(grad_scale_kernel<T>, dim3(1), dim3(1024), 0, s, a));
    a.x_m_tiles = a.m_tiles;
    a.h_tiles = static_cast<int>(ceil_div(sh.hidden, kTileN));
    a.slice_blocks = static_cast<int>(p.slice_blocks);
    a.x_partial = p.partial_dx;
    a.w_f32 = f32_dweight;
    a.w_first = p.w_first;
    HeadMaps mz = {}, mo = {};
    LS_CUDA(make_map<T>(&mz.a, x, sh.hidden, sh.rows, sh.hidden, a.row_box));
    const int grad_n = grad_columns(sh.rows, std::min(p.cols, sh.vocab));
    LS_CUDA(make_map<T>(&mz.b, w, sh.hidden, sh.vocab, sh.hidden, grad_n / 2));
    LS_CUDA(make_map<T>(&mo.b, w, sh.hidden, sh.vocab, sh.hidden, 64));
    LS_CUDA(make_map<T>(&mo.b2, ws + p.used_x, sh.hidden, sh.rows, sh.hidden, 64));
    if (dx && p.partial_dx)
        LS_CUDA(make_map<float>(&mo.out, partial, sh.hidden, sh.rows, sh.hidden, 32, p.slices));
    else if (dx)
        LS_CUDA(make_map<T>(&mo.out, dx, sh.hidden, sh.rows, sh.hidden, 32));
    // dweight's sums over the rows, kMostRows of them at a time: added to an FP32 dweight, or to scratch.
    const int64_t row_blocks = ceil_div(sh.rows, kBlockK);
    a.w_partial = dweight && !f32_dweight && sh.rows > kMostRows;
    float* w_partial = reinterpret_cast<float*>(ws + p.w_partial);
    if (a.w_partial)
        LS_CUDA(make_map<float>(&mo.out2, w_partial, sh.hidden, p.cols, sh.hidden, 32));
    else if (dweight && f32_dweight)
        LS_CUDA(make_map<float>(&mo.out2, dweight, sh.hidden, sh.vocab, sh.hidden, 32));
    else if (dweight)
        LS_CUDA(make_map<T>(&mo.out2, dweight, sh.hidden, sh.vocab, sh.hidden, 32));
    for (int64_t c = 0; c < sh.vocab; c += p.cols) {
        const int64_t cols = std::min(p.cols, sh.vocab - c);
        a.col0 = static_cast<int>(c);
        a.cols = static_cast<int>(cols);
        set_tiles(a, grad_n);
        a.find_scale = find_scale && c == 0;
        a.x = x;
        a.used_x = dweight && c == 0 ? ws + p.used_x : nullptr;
        LS_CUDA(make_map<T>(&mz.out, g, cols, sh.rows, p.cols, 32));
        LS_CUDA((launch_head<T, kGrad, false>(mz, a, static_cast<int64_t>(a.m_tiles) * a.n_tiles, s)));
        LS_CUDA(make_map<T>(&mo.a, g, cols, sh.rows, p.cols, a.row_box));
        LS_CUDA(make_map<T>(&mo.a2, g, cols, sh.rows, p.cols, 64));
        a.x_k_blocks = static_cast<int>(ceil_div(cols, kBlockK));
        a.x_add = c > 0;
        a.slices = static_cast<int>(ceil_div(a.x_k_blocks, a.slice_blocks));
        a.x_units = dx ? a.x_m_tiles * a.h_tiles : 0;
        a.w_units = dweight ? a.slice_blocks / (kTileM / kBlockK) * a.h_tiles : 0;
        const int all_w_units = dweight ? static_cast<int>(ceil_div(cols, kTileM)) * a.h_tiles : 0;
        a.units = a.slices * a.x_units + all_w_units;
        a.by_slice = p.by_slice;
        a.w_row = a.w_partial ? 0 : a.col0;
        a.w_add = f32_dweight;
        for (int64_t kb = 0; kb < (dweight ? row_blocks : 1); kb += kMostRows / kBlockK) {
            a.w_kb0 = static_cast<int>(kb);
            a.w_k_blocks = static_cast<int>(std::min(kMostRows / kBlockK, row_blocks - kb));
            LS_CUDA((launch_head<T, kOut, false>(mo, a, a.units, s)));
            a.x_units = 0;
            a.units = all_w_units;
            a.by_slice = false;
            a.w_add = true;
        }
        if (a.w_partial) {
            const int64_t nvec = cols * sh.hidden / kVec;
            LS_CUDA(launch_pdl(join_slices_kernel<T>, dim3(static_cast<unsigned>(ceil_div(nvec, 256))), dim3(256), 0, s,
                               static_cast<T*>(dweight) + c * sh.hidden, static_cast<const float*>(w_partial), 1, nvec, a));
        }
    }
    if (!dx || !p.partial_dx) return cudaSuccess;
    const int64_t nvec = sh.rows * sh.hidden / kVec;
    return launch_pdl(join_slices_kernel<T>, dim3(static_cast<unsigned>(ceil_div(nvec, 256))), dim3(256), 0, s,
                      static_cast<T*>(dx), partial, static_cast<int>(p.slices), nvec, a);
}

}  // namespace

size_t linear_ce_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab) {
    return HeadPlan(rows, hidden, vocab).bytes;
}

size_t linear_ce_fwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab) {
    return HeadPlan(rows, hidden, vocab).fwd_bytes;
}

cudaError_t launch_linear_ce_fwd(ls_dtype dt, float* loss, float* lse, const void* x,
                                 const void* weight, const int32_t* target, const HeadShape& sh,
                                 void* workspace, cudaStream_t s) {
    if (dt == LS_F16) return fwd<__half>(loss, lse, x, weight, target, sh, workspace, s);
    return fwd<bf16>(loss, lse, x, weight, target, sh, workspace, s);
}

cudaError_t launch_linear_ce_bwd(ls_dtype dt, void* dx, void* dweight, bool f32_dweight,
                                 const void* x, const void* weight, const int32_t* target,
                                 const float* lse, const float* dloss, const HeadShape& sh,
                                 void* workspace, cudaStream_t s) {
    if (dt == LS_F16)
        return bwd<__half>(dx, dweight, f32_dweight, x, weight, target, lse, dloss, sh, workspace,
                           s);
    return bwd<bf16>(dx, dweight, f32_dweight, x, weight, target, lse, dloss, sh, workspace, s);
}

cudaError_t launch_vocab_wait_selftest(uint32_t polls, cudaStream_t s) {
    wait_selftest_kernel<<<1, 64, 0, s>>>(polls);
    return cudaGetLastError();
}

cudaError_t linear_ce_take_device_error(unsigned int* flags) {
    return take_device_error_word(flags);
}

}  // namespace ls
