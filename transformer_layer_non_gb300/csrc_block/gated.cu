// gated.cu -- the gated feed-forward block: h = act(x Wg^T) * (x Wu^T), and its
// gradients, on tcgen05.
//
// Forward: a tile has 256 rows and the same `half` columns of both projections.
// They are one product whose second operand is Wg's rows in the pair's first CTA
// and Wu's in its second, so that the accumulator has gate and up side by side
// and one warp reads both of an element: the activation and the product never
// leave registers.
// Backward: the same tiles again, with dh; dg and du are rounded to the storage
// type in the workspace.  Then dx = [dg du] [Wg; Wu] and dW = [dg du]^T x, in one
// launch.  Computing g and u again costs 2 of 6 products; keeping them in 16 bits
// instead would cost two more roundings in dg and du and 4 bytes for each element
// of the block, in FP32 8.
//
// Persistent pairs of CTAs, each pair a tile of up to 256 x 256 with FP32
// accumulators in tensor memory (two of them, so that one is read while the
// other is filled), operands brought by TMA through a ring of 64-wide K blocks.
// Warp 0 issues the copies, warp 1 of the pair's first CTA the products, the
// other warps take the accumulators to the outputs.  Operands of which M or N is
// the contiguous axis (the weights in dx; dg, du and x in dW) are read as they
// lie in memory.
//
// Step 4096 x 1280 x 5120 BF16: forward 59 us (1.8 PFLOP/s), dg and du 73, gradients
// 113 (1.9); tensor pipes 83, 67 and 90 % of their cycles.  What keeps the second one
// from the first's rate are its stores, next to the 64 bytes a cycle that each SM
// takes from L2 for operands.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "../csrc_vocab/tc_tile.cuh"
#include "block_internal.h"
#include "gated_act.cuh"

namespace ls {
namespace {

constexpr int kTileM = 256;   // of a pair; 128 rows for each CTA
constexpr int kTileN = 256;
constexpr int kBlockK = 64;   // 128 bytes: the swizzle's row
constexpr int kStages = 5;
constexpr int kEpilogueWarps = 8;  // two for each quarter of the tensor memory's lanes, half the columns each
constexpr int kThreads = 64 + 32 * kEpilogueWarps;
constexpr int kWarpBoxes = 2;      // a warp's store boxes
constexpr uint32_t kOperandBytes = 128 * kBlockK * 2;  // one operand of one CTA and stage
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
// Tiles of which a CTA holds no more than 64 rows of B take two K blocks to a stage, in fewer stages: the two waits for
// each stage, one in the copying and one in the multiplying warp, cost about 0.2 us, more than such a K block's products.
constexpr int kPairStages = 3;
constexpr uint32_t kPairStageBytes = 3 * kOperandBytes;
static_assert(kPairStages * kPairStageBytes <= kStages * kStageBytes, "the stages' memory");
constexpr uint32_t kStoreBytes = 32 * 128;             // one warp's store box
constexpr uint32_t kTmemColumns = 512;
constexpr uint32_t kSmemBytes = 1024 + kStages * kStageBytes + kEpilogueWarps * kWarpBoxes * kStoreBytes;
constexpr int kGroupM = 16;   // row tiles that share a sweep over the columns
constexpr int kPairs = 76;    // pairs of SMs; a constant, so that plans depend on the shapes alone
constexpr int kMostHalf = 128;
// dg and du are rounded to 16 bits before they are summed up to gradients, which adds as much error again as the
// gradients' own rounding: sqrt(2) times that as a whole, at any size (4096 x 1280 x 5120 BF16: 0.00235 and 0.00166).  How
// far single tensors are from that depends on how many roundings there are, rows x ffn of each: of few of them some are
// well above it (3 x 376 x 240: 1.52 times), so these are kept as two 16-bit numbers each.  Up to kPairRows rows, whose
// K block of dW has room for the second ones; dx takes twice the K blocks (1 x 344 x 480, step: 10.1 -> 10.7 us).
constexpr int kPairRows = 32;
constexpr int64_t kPairElements = 16384;

enum Mode { kFwd = 0, kGrad = 1, kOut = 2 };

struct GatedArgs {
    int rows, ffn, hidden;
    int act;
    int m_tiles, n_tiles;  // kFwd, kGrad: rows x ffn
    int half;              // columns of h in a tile: 32, 64, 96 or 128
    int whole_tiles;       // the tiles behind these are halved, a unit each
    int row_box;           // rows of the copies with rows as M: 128, or all where there are fewer
    int k_blocks;
    int part_blocks;       // of two accumulators for a tile: the K blocks that the first one takes
    const void* dh;        // kGrad
    void *out, *out2;      // tiles of fewer than 128 columns: h; dg and du
    // kOut
    int slices, slice_blocks;  // of dx's K, dg's columns and then du's
    int x_units, w_units;      // units of dx in a slice; units of both dW
    int w_tiles;               // of one dW, in a slice
    int width;                 // columns of a tile: 128 or 256
    int w_slice_blocks;        // of the rows
    int h_tiles, f_blocks, x_blocks;  // x_blocks: K blocks of dx
    bool pairs;                // dg and du as sums of two 16-bit numbers, of which the second ones are apart
    int w_kb0, w_k_blocks;     // the rows that dW's sums run over in this launch
    bool w_first, x_partial, w_partial, w_f32, w_add;  // partial: FP32 sums of slices go to scratch
    int pairs1, first_short1;  // how the shorter units are dealt, see Deal
};

struct GatedMaps {
    CUtensorMap a, b, b2;      // kFwd, kGrad: x, Wg, Wu;  kOut: dg for dx, Wg, Wu
    CUtensorMap a2;            // kOut: du for dx
    CUtensorMap a_low, a2_low, wa_low, wa2_low;  // kOut: the second numbers of dg and du
    CUtensorMap wa, wa2, wb;   // kOut: dg, du, x for dW;  kFwd, kGrad: Wg, Wu for halved tiles
    CUtensorMap out, out2, out3;  // h; dg, du; dx, dWg, dWu
};

// One unit of work of a pair.
struct Unit {
    int m0, n0;   // first row and column of the tile
    int kb0, kbs;  // K blocks
    int slice;
    int weight;   // kOut: 0 a tile of dx, 1 of dWg, 2 of dWu
    int half;     // kFwd, kGrad: columns of h
};

template <int MODE> __device__ __forceinline__ Unit unit_of(int u, const GatedArgs& a) {
    Unit t;
    t.weight = 0;
    t.slice = 0;
    t.kb0 = 0;
    if constexpr (MODE != kOut) {
        const bool halved = u >= a.whole_tiles;
        const int tile = halved ? a.whole_tiles + (u - a.whole_tiles) / 2 : u;
        const int g = tile / (kGroupM * a.n_tiles);
        const int first = g * kGroupM;
        const int gm = min(kGroupM, a.m_tiles - first);
        const int r = tile - first * a.n_tiles;
        t.half = halved ? a.half / 2 : a.half;
        t.n0 = (r / gm) * a.half + (halved ? (u - a.whole_tiles) % 2 * t.half : 0);
        t.m0 = (first + r % gm) * kTileM;
        t.kbs = a.k_blocks;
    } else {  // all of one kind, then all of the other
        const int first = a.w_first ? a.w_units : a.slices * a.x_units;
        int r = u;
        const bool weight = (r >= first) != a.w_first;
        if (r >= first) r -= first;
        if (weight) {
            t.slice = r / (2 * a.w_tiles);
            r -= t.slice * 2 * a.w_tiles;
            t.weight = 1 + r / a.w_tiles;
            r -= (t.weight - 1) * a.w_tiles;
            t.kb0 = a.w_kb0 + t.slice * a.w_slice_blocks;
            t.kbs = min(a.w_slice_blocks, a.w_k_blocks - t.slice * a.w_slice_blocks);
        } else {
            t.slice = r / a.x_units;
            r -= t.slice * a.x_units;
            t.kb0 = t.slice * a.slice_blocks;
            t.kbs = min(a.slice_blocks, a.x_blocks - t.kb0);
        }
        t.half = 0;
        t.n0 = (r % a.h_tiles) * a.width;
        t.m0 = (r / a.h_tiles) * kTileM;
    }
    return t;
}

// The units of a pair, one after the other: its number'th in turn of the tiles.  kOut: the longer units in turn,
// then the shorter ones, of which the pairs that got one more of the longer (the first `pairs1`) have those from
// number `first_short1` on among themselves, and the others those before it.
template <int MODE> struct PairUnits {
    int u, step, end;
    int next, next_step, next_end;  // the shorter ones
    __device__ __forceinline__ PairUnits(int pair, int pairs, const GatedArgs& a) {
        u = pair;
        step = pairs;
        end = MODE == kOut ? (a.w_first ? a.w_units : a.slices * a.x_units) : 2 * a.m_tiles * a.n_tiles - a.whole_tiles;
        if constexpr (MODE == kOut) {
            const int all = a.slices * a.x_units + a.w_units;
            const bool more = pair < a.pairs1;
            next = end + (more ? a.first_short1 + pair : pair - a.pairs1);
            next_step = more ? a.pairs1 : pairs - a.pairs1;
            next_end = more ? all : end + a.first_short1;
            settle();
        }
    }
    __device__ __forceinline__ void settle() {
        if (MODE == kOut && u >= end) {
            u = next;
            step = next_step;
            end = next_end;
            next = next_end;  // none behind these
        }
    }
    __device__ __forceinline__ bool there() const { return u < end; }
    __device__ __forceinline__ void advance() {
        u += step;
        settle();
    }
};

// 32 values each of g and u to act(g) u, or with dh to dg and du in their places.
template <int MODE, int ACT, typename T>
__device__ __forceinline__ void combine(float (&g)[32], float (&u)[32], const uint4 (&dh)[4]) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        float d[kVec];
        if constexpr (MODE == kGrad) unpack(Raw8<T>{dh[v]}, d);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int i = v * kVec + j;
            const ActValue a = act_of<ACT>(g[i]);
            if constexpr (MODE == kFwd) {
                g[i] = a.a * u[i];
            } else {
                g[i] = d[j] * u[i] * a.slope;
                u[i] = d[j] * a.a;
            }
        }
    }
}
template <int MODE, typename T>
__device__ __forceinline__ void combine_act(int act, float (&g)[32], float (&u)[32], const uint4 (&dh)[4]) {
    if (act == LS_ACT_SILU) combine<MODE, LS_ACT_SILU, T>(g, u, dh);
    else if (act == LS_ACT_GELU) combine<MODE, LS_ACT_GELU, T>(g, u, dh);
    else if (act == LS_ACT_GELU_TANH) combine<MODE, LS_ACT_GELU_TANH, T>(g, u, dh);
    else combine<MODE, LS_ACT_RELU, T>(g, u, dh);
}

// z += 32 more columns of accumulators.
__device__ __forceinline__ void add_columns(float (&z)[32], uint32_t cols) {
    float more[32];
    tmem_ld32(more, cols);
    tmem_ld_wait(more);
#pragma unroll
    for (int i = 0; i < 32; ++i) z[i] += more[i];
}

// BLOCKS: K blocks of a stage.  PARTS: accumulators of a tile, 2 where one would add up too much (a parameter, since what
// it adds to the multiplying warp's loop cost chains of K blocks 6 %).
template <typename T, int MODE, int BLOCKS, int PARTS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
gated_kernel(const __grid_constant__ GatedMaps maps, const __grid_constant__ GatedArgs a) {
    // A stage has its blocks of A, and behind them those of B.
    constexpr uint32_t kCount = BLOCKS == 1 ? kStages : kPairStages, kBytes = BLOCKS == 1 ? kStageBytes : kPairStageBytes;
    constexpr uint32_t kStepB = kOperandBytes / BLOCKS;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    // The swizzle's pattern repeats every 1024 bytes of the address.
    unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
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
        prefetch_map(MODE == kOut || rank == 0 ? &maps.b : &maps.b2);
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
        for (PairUnits<MODE> p(pair, pairs, a); p.there(); p.advance()) {
            const Unit t = unit_of<MODE>(p.u, a);
            const int m = t.m0 + static_cast<int>(rank) * 128;
            const int b_rows = MODE == kOut ? a.width / 2 : t.half;  // of B in each CTA
            const int n = MODE == kOut ? t.n0 + static_cast<int>(rank) * b_rows : t.n0;
            // Rows behind the last one are not copied: what the shared memory holds there reaches rows of the
            // accumulator that nothing reads.
            auto a_bytes = [&](int first) -> uint32_t {
                return t.weight ? kOperandBytes : first < a.rows ? static_cast<uint32_t>(a.row_box) * 128 : 0;
            };
            const CUtensorMap* b_map = t.half == a.half ? (rank == 0 ? &maps.b : &maps.b2) : rank == 0 ? &maps.wa : &maps.wa2;
            const uint32_t bytes = 2 * b_rows * 128 + a_bytes(t.m0) + a_bytes(t.m0 + 128);  // of both CTAs
            const bool has_a = a_bytes(m) > 0;
            for (int kb0 = 0; kb0 < t.kbs; kb0 += BLOCKS, ++it) {
                const uint32_t s = it % kCount;
                if (!wait_bar(empty + s, ((it / kCount) & 1) ^ 1, &dead)) break;
                if (elect_one()) {
                    const int blocks = BLOCKS == 1 ? 1 : min(BLOCKS, t.kbs - kb0);
                    if (rank == 0) mbar_arrive_expect_tx(full + s, blocks * bytes);
                    const uint32_t bar = map_rank(full + s, 0);
#pragma unroll
                    for (int j = 0; j < BLOCKS; ++j) {
                        if (j >= blocks) break;
                        const int kb = kb0 + j;
                        unsigned char* pa = smem + s * kBytes + j * kOperandBytes;
                        unsigned char* pb = smem + s * kBytes + BLOCKS * kOperandBytes + j * kStepB;
                        if constexpr (MODE != kOut) {
                            const int k = kb * kBlockK;
                            if (has_a) tma_load_2d(pa, &maps.a, k, m, bar);
                            tma_load_2d(pb, b_map, k, n, bar);
                        } else if (!t.weight) {
                            int b = t.kb0 + kb;  // of dg, du, and the second numbers of both
                            const bool low = b >= 2 * a.f_blocks;
                            if (low) b -= 2 * a.f_blocks;
                            const bool up = b >= a.f_blocks;
                            const int k = (b - (up ? a.f_blocks : 0)) * kBlockK;
                            const CUtensorMap* w = up ? &maps.b2 : &maps.b;
                            const CUtensorMap* d = low ? (up ? &maps.a2_low : &maps.a_low) : up ? &maps.a2 : &maps.a;
                            if (has_a) tma_load_2d(pa, d, k, m, bar);
                            tma_load_2d(pb, w, n, k, bar);
                            if (b_rows > 64) tma_load_2d(pb + kOperandBytes / 2, w, n + 64, k, bar);
                        } else if (a.pairs) {  // 32 rows of the first numbers, the same of the second ones; x twice
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const CUtensorMap* d = t.weight == 2 ? (h ? &maps.wa2_low : &maps.wa2) : h ? &maps.wa_low : &maps.wa;
                                unsigned char* const da = pa + h * (kPairRows * 128);
                                unsigned char* const db = pb + h * (kPairRows * 128);
                                tma_load_2d(da, d, m, 0, bar);
                                tma_load_2d(da + kOperandBytes / 2, d, m + 64, 0, bar);
                                tma_load_2d(db, &maps.wb, n, 0, bar);
                                if (b_rows > 64) tma_load_2d(db + kOperandBytes / 2, &maps.wb, n + 64, 0, bar);
                            }
                        } else {
                            const int k = (t.kb0 + kb) * kBlockK;
                            const CUtensorMap* d = t.weight == 2 ? &maps.wa2 : &maps.wa;
                            tma_load_2d(pa, d, m, k, bar);
                            tma_load_2d(pa + kOperandBytes / 2, d, m + 64, k, bar);
                            tma_load_2d(pb, &maps.wb, n, k, bar);
                            if (b_rows > 64) tma_load_2d(pb + kOperandBytes / 2, &maps.wb, n + 64, k, bar);
                        }
                    }
                }
                __syncwarp();
            }
            if (dead) break;
        }
        // After a failed wait: the copies in flight land before the CTA ends.
        if (dead && rank == 0)
            for (uint32_t s = 0; s < kCount && s < it; ++s) {
                const uint32_t uses = (it - 1 - s) / kCount;  // its last use, counted from 0
                for (uint32_t i = 0; i < kWaitPolls; ++i)
                    if (mbar_try_wait(full + s, uses & 1)) break;
            }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr bool kBf16 = std::is_same<T, bf16>::value;
            const uint64_t kmajor = desc_base(16), mnmajor = desc_base(kOperandBytes / 2);
            uint32_t it = 0, tile = 0;
            int done = 0;  // K blocks of the tile that are in its first accumulator
            for (PairUnits<MODE> p(pair, pairs, a); p.there(); ++tile) {
                const Unit t = unit_of<MODE>(p.u, a);
                const int kbs = PARTS == 1 ? t.kbs : done > 0 ? t.kbs - done : a.part_blocks;
                const uint32_t acc = tile & 1;
                if (!wait_bar(acc_empty + acc, ((tile >> 1) & 1) ^ 1, &dead)) break;
                tc_fence_after();
                // Which operands have M or N as their contiguous axis.
                const bool a_mn = MODE == kOut && t.weight, b_mn = MODE == kOut;
                const uint32_t idesc = instr_desc(kBf16, a_mn, b_mn, kTileM, MODE == kOut ? a.width : 2 * t.half);
                const uint64_t da = desc_at(a_mn ? mnmajor : kmajor, smem_u32(smem));
                const uint64_t db = desc_at(b_mn ? mnmajor : kmajor, smem_u32(smem) + BLOCKS * kOperandBytes);
                // 16 values of K further on, in the descriptors' units of 16 bytes
                const uint32_t step_a = a_mn ? 128 : 2, step_b = b_mn ? 128 : 2;
                const uint32_t d = tmem + acc * kTileN;
                for (int kb0 = 0; kb0 < kbs; kb0 += BLOCKS, ++it) {
                    const uint32_t s = it % kCount;
                    if (!wait_bar(full + s, (it / kCount) & 1, &dead)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = s * (kBytes >> 4);
#pragma unroll
                        for (int j = 0; j < BLOCKS; ++j) {
                            if (kb0 + j >= kbs) break;
                            const uint64_t ja = da + (at + j * (kOperandBytes >> 4)), jb = db + (at + j * (kStepB >> 4));
#pragma unroll
                            for (int k = 0; k < kBlockK / 16; ++k)
                                tc_mma(d, ja + k * step_a, jb + k * step_b, idesc, kb0 + j + k > 0);
                        }
                        tc_commit(empty + s);
                    }
                    __syncwarp();
                }
                if (dead) break;
                if (elect_one()) tc_commit(acc_full + acc);
                __syncwarp();
                done = PARTS == 1 || done > 0 ? 0 : kbs;
                if (done == 0) p.advance();
            }
            if (dead) {  // the products in flight end before their operands' memory is given back
                if (elect_one()) tc_commit(&drained);
                __syncwarp();
                for (uint32_t i = 0; i < kWaitPolls; ++i)
                    if (mbar_try_wait(&drained, 0)) break;
            }
        }
        __syncwarp();
    } else {
        const int quad = warp & 3;         // the TMEM lanes this warp may read
        const int part = (warp - 2) >> 2;  // its part of the tile's columns
        unsigned char* const boxes = smem + kStages * kStageBytes + (warp - 2) * kWarpBoxes * kStoreBytes;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        uint32_t tile = 0, opened = 0;
        for (PairUnits<MODE> p(pair, pairs, a); p.there(); p.advance(), tile += PARTS) {
            const Unit t = unit_of<MODE>(p.u, a);
            const uint32_t acc = tile & 1;
            const int row0 = t.m0 + static_cast<int>(rank) * 128 + quad * 32;  // this warp's first row
            const int row = row0 + lane;
            auto release = [&]() {  // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_rank(acc_empty + acc, 0));
                if (PARTS == 2 && lane == 0) mbar_arrive_cluster(map_rank(acc_empty + 1, 0));
            };
            if constexpr (MODE != kOut) {
                const int chunks = t.half / 32, per = (chunks + 1) / 2;
                const int c0 = part * per, cs = min(per, chunks - c0);  // its groups of 32 columns, 0 to 2
                uint4 dh[2][4];
                if constexpr (MODE == kGrad) {  // on its way while the products end
                    const T* d = static_cast<const T*>(a.dh) + static_cast<int64_t>(row) * a.ffn;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const int f = t.n0 + (c0 + c) * 32 + v * kVec;
                            dh[c][v] = c < cs && row < a.rows && f < a.ffn ? ld16(d + f) : make_uint4(0, 0, 0, 0);
                        }
                }
                if constexpr (MODE == kGrad) {  // and the next tile's on its way to L2
                    PairUnits<MODE> q = p;
                    q.advance();
                    if (q.there()) {
                        const Unit n = unit_of<MODE>(q.u, a);
                        const int np = (n.half / 32 + 1) / 2, nc = part * np;
                        const int r = n.m0 + static_cast<int>(rank) * 128 + quad * 32 + lane, f = n.n0 + nc * 32;
                        if (r < a.rows && f < a.ffn && nc * 32 < n.half) {
                            const T* d = static_cast<const T*>(a.dh) + static_cast<int64_t>(r) * a.ffn + f;
                            prefetch_l2(d);
                            prefetch_l2(d + min(min(np * 32, n.half - nc * 32), a.ffn - f) - 1);
                        }
                    }
                }
                if (!wait_bar(acc_full + acc, (tile >> 1) & 1, &dead)) break;
                if (PARTS == 2 && !wait_bar(acc_full + 1, (tile >> 1) & 1, &dead)) break;  // of two, acc is 0
                tc_fence_after();
                const uint32_t cols = lanes + acc * kTileN;
                const bool boxed = t.half == kMostHalf;
                unsigned char* box = boxes;
                if (boxed) {  // the boxes are free: one of two for h, both for dg and du
                    if constexpr (MODE == kFwd) box += (opened++ % kWarpBoxes) * kStoreBytes;
                    if (lane == 0) bulk_wait_read<MODE == kFwd ? 1 : 0>();
                    __syncwarp();
                }
                if (cs <= 0) release();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (c >= cs) break;
                    float zg[32], zu[32];
                    tmem_ld32(zg, cols + (c0 + c) * 32);
                    tmem_ld32(zu, cols + t.half + (c0 + c) * 32);
                    tmem_ld_wait(zg);
                    tmem_ld_wait(zu);
                    if constexpr (PARTS == 2) {
                        add_columns(zg, cols + kTileN + (c0 + c) * 32);
                        add_columns(zu, cols + kTileN + t.half + (c0 + c) * 32);
                    }
                    if (c + 1 == cs) release();
                    combine_act<MODE, T>(a.act, zg, zu, dh[c]);
                    if (boxed) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            put16(box, lane, c * 4 + j, pack8<T>(zg, 8 * j, 1.f));
                            if constexpr (MODE == kGrad) put16(box + kStoreBytes, lane, c * 4 + j, pack8<T>(zu, 8 * j, 1.f));
                        }
                    } else if (row < a.rows) {
                        const int f = t.n0 + (c0 + c) * 32;
                        const int64_t e = static_cast<int64_t>(row) * a.ffn + f;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (f + 8 * j < a.ffn) {
                                st16(static_cast<T*>(a.out) + e + 8 * j, pack8<T>(zg, 8 * j, 1.f));
                                if constexpr (MODE == kGrad)
                                    st16(static_cast<T*>(a.out2) + e + 8 * j, pack8<T>(zu, 8 * j, 1.f));
                            }
                    }
                }
                if (boxed) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (row0 < a.rows && t.n0 + c0 * 32 < a.ffn) {
                            tma_store_2d(&maps.out, t.n0 + c0 * 32, row0, box);
                            if constexpr (MODE == kGrad) tma_store_2d(&maps.out2, t.n0 + c0 * 32, row0, box + kStoreBytes);
                        }
                        bulk_commit();
                    }
                }
            } else {
                if (!wait_bar(acc_full + acc, (tile >> 1) & 1, &dead)) break;
                tc_fence_after();
                const int n0 = t.n0 + part * (a.width / 2);
                const uint32_t cols = lanes + part * (a.width / 2) + acc * kTileN;  // two of the four groups behind a narrow tile's
                const bool f32 = t.weight ? a.w_f32 : a.x_partial;
                const int n = min(a.width / 2, a.hidden - n0);
                const bool stores = row0 < (t.weight ? a.ffn : a.rows);
                const CUtensorMap* w_out = t.weight == 2 ? &maps.out3 : &maps.out2;
                unsigned char* box = boxes;
                auto open_box = [&]() {  // the next store box, free to be written
                    box = boxes + (opened++ % kWarpBoxes) * kStoreBytes;
                    if (lane == 0) bulk_wait_read<kWarpBoxes - 1>();
                    __syncwarp();
                };
                auto close_box = [&](auto&& store) {  // and on its way to memory
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (stores) store();
                        bulk_commit();
                    }
                };
                if (f32)
                    sweep(cols, release, [&](int c, float (&z)[32]) {
                        if (c * 32 >= n) return;
                        open_box();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            put16(box, lane, j, f2u4(make_float4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3])));
                        close_box([&] {
                            if (!t.weight || a.w_partial)
                                tma_store_3d(t.weight ? w_out : &maps.out, n0 + c * 32, row0, t.slice, box);
                            else if (a.w_add)
                                tma_add_2d(w_out, n0 + c * 32, row0, box);
                            else
                                tma_store_2d(w_out, n0 + c * 32, row0, box);
                        });
                    });
                else
                    sweep(cols, release, [&](int c, float (&z)[32]) {
                        if (c * 32 >= n) return;
                        if ((c & 1) == 0) open_box();
#pragma unroll
                        for (int j = 0; j < 4; ++j) put16(box, lane, (c & 1) * 4 + j, pack8<T>(z, 8 * j, 1.f));
                        if ((c & 1) == 1 || c * 32 + 32 >= n)
                            close_box([&] { tma_store_2d(t.weight ? w_out : &maps.out, n0 + (c & ~1) * 32, row0, box); });
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

// Self-test of the waits' failure path: two warps wait, as those of gated_kernel do, on a barrier that expects
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

// out (+)= the sum over the slices' FP32 sums, in slice order: those of dWg, dWu and dx, blockIdx.y one of them.
struct JoinArgs {
    void* out[3];
    const float* part[3];
    int slices[3];
    int64_t vecs[3];
    bool f32[3];  // FP32 to be added to, or the storage type to be written
};
template <typename O> __device__ __forceinline__ void join_vec(O* out, const float* part, int slices, int64_t vecs, int64_t v, bool add) {
    float acc[kVec];
    load8f<float>(part + v * kVec, acc);
    for (int s = 1; s < slices; ++s) {
        float f[kVec];
        load8f<float>(part + (s * vecs + v) * kVec, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) acc[j] += f[j];
    }
    if (add) {
        float f[kVec];
        load8f<O>(out + v * kVec, f);
#pragma unroll
        for (int j = 0; j < kVec; ++j) acc[j] += f[j];
    }
    store8f<O>(out + v * kVec, acc);
}
template <typename T> __global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs a) {
    pdl_enter();
    const int k = blockIdx.y;
    const int64_t v = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (v >= a.vecs[k]) return;
    if (a.f32[k])
        join_vec(static_cast<float*>(a.out[k]), a.part[k], a.slices[k], a.vecs[k], v, true);
    else
        join_vec(static_cast<T*>(a.out[k]), a.part[k], a.slices[k], a.vecs[k], v, false);
}

// --- host ----------------------------------------------------------------------
constexpr int64_t kMaxSlices = 16;
// Tensor cores drop low bits as they accumulate: a sum of terms of one sign loses about 5.6e-9 of itself for
// each of them.  No accumulator adds up more than these (of kFwd and kGrad kMostColumns of hidden); what it has then is
// added in FP32.
constexpr int64_t kMostRows = 16384;
constexpr int64_t kMostColumns = 32768;
static_assert(kMaxGatedCols <= 2 * kMostColumns, "a tile of kFwd and kGrad has two accumulators");

// Columns of h in a tile: fewer than 128 for one or two tiles of rows where the busiest pair has less to do that
// way.  A K block's time goes with the columns down to 64 of each projection, and a tile costs about one K block more.
int half_columns(int64_t rows, int64_t hidden, int64_t ffn) {
    if (rows > 2 * kTileM) return kMostHalf;
    const int64_t m_tiles = ceil_div(rows, kTileM), k_blocks = ceil_div(hidden, kBlockK);
    int best_half = kMostHalf;
    int64_t best = INT64_MAX;
    for (int half = kMostHalf; half >= 32; half -= 32) {
        const int64_t t = ceil_div(m_tiles * ceil_div(ffn, half), kPairs) *
                          ((std::max(2 * half, 128) + 8) * k_blocks + 2 * half + 256);
        if (t < best) {
            best = t;
            best_half = half;
        }
    }
    return best_half;
}

// Units of two lengths dealt to the pairs: the longer ones in turn, the shorter ones so that the pair with the
// most to do has as little as can be: `each1` for each of the first `pairs1` pairs, which have one more of the
// longer, the rest for the others.
struct Deal {
    int64_t pairs1, short1, most;  // short1: shorter units for the first pairs
    Deal(int64_t n_long, int64_t len_long, int64_t n_short, int64_t len_short) {
        const int64_t pairs = std::min<int64_t>(kPairs, n_long + n_short), base = n_long / pairs;
        pairs1 = n_long % pairs;
        most = INT64_MAX;
        // both kinds of pairs end together near this number, which the rounding up moves by one at most
        const int64_t even = (n_short * len_short - len_long * (pairs - pairs1)) / (len_short * pairs);
        for (int64_t each1 = std::max<int64_t>(0, even - 1); each1 <= std::max<int64_t>(0, even + 2); ++each1) {
            const int64_t s1 = std::min(n_short, pairs1 * each1);
            const int64_t load1 = pairs1 ? (base + 1) * len_long + ceil_div(s1, pairs1) * len_short : 0;
            const int64_t load0 = base * len_long + ceil_div(n_short - s1, pairs - pairs1) * len_short;
            if (std::max(load1, load0) >= most) continue;
            most = std::max(load1, load0);
            short1 = s1;
        }
    }
};

// The tiles' width, slices and workspace layout; they depend on the shapes alone.  Time is counted in 20ths of a K
// block of a pair's tile (256 x 256 x 64 products, about 0.3 us); one of 128 columns takes 15 of them.
int64_t unit_length(int64_t width, int64_t blocks, bool joined) {
    return blocks * (width == kTileN ? 20 : 15) + (joined ? 2 : 1) * (width == kTileN ? 20 : 14);
}

GatedPlan make_plan(int64_t rows, int64_t hidden, int64_t ffn) {
    GatedPlan p = {};
    const int64_t m_tiles = ceil_div(rows, kTileM);
    p.pairs = rows <= kPairRows && rows * ffn <= kPairElements;
    const int64_t kb = (p.pairs ? 4 : 2) * ceil_div(ffn, kBlockK), row_blocks = ceil_div(rows, kBlockK);
    // joining slices: a launch, and their bytes at about 1.7 MB for a K block's time
    auto join = [](int64_t n, int64_t elements) { return n > 1 ? n * elements * 4 / 85000 : 0; };
    int64_t best = INT64_MAX;
    for (int64_t wide = kTileN; wide >= kTileN / 2; wide /= 2) {
        const int64_t h_tiles = ceil_div(hidden, wide), w_tiles = 2 * ceil_div(ffn, kTileM) * h_tiles;
        // Rows are cut where a small model's weights would leave most pairs without a tile of dW.
        const int64_t most_w = w_tiles < kPairs && rows <= kMostRows ? std::min<int64_t>(row_blocks, 8) : 1;
        for (int64_t sw = 1; sw <= most_w; ++sw) {
            const int64_t w_part = ceil_div(row_blocks, sw), wl = unit_length(wide, w_part, sw > 1);
            if (ceil_div(row_blocks, w_part) != sw) continue;
            for (int64_t s = 1; s <= std::min(kb, kMaxSlices); ++s) {
                const int64_t len = ceil_div(kb, s);
                if (ceil_div(kb, len) != s || len * kBlockK > kMostColumns) continue;
                const int64_t x_units = s * m_tiles * h_tiles, xl = unit_length(wide, len, s > 1), w_units = sw * w_tiles;
                const int64_t out = wl > xl ? Deal(w_units, wl, x_units, xl).most : Deal(x_units, xl, w_units, wl).most;
                const int64_t t = out + (s > 1 || sw > 1 ? 240 : 0) + join(s, rows * hidden) + join(sw, 2 * ffn * hidden);
                if (t >= best) continue;
                best = t;
                p.width = wide;
                p.slices = s;
                p.slice_blocks = len;
                p.w_slices = sw;
                p.w_slice_blocks = w_part;
                p.x_len = xl;
                p.w_first = wl > xl;
            }
        }
    }
    p.du = round256(static_cast<size_t>(rows * ffn) * 2);
    p.partial = (p.pairs ? 4 : 2) * p.du;
    p.w_partial = p.partial + (p.slices > 1 ? round256(static_cast<size_t>(p.slices * rows * hidden) * 4) : 0);
    const bool scratch = p.w_slices > 1 || rows > kMostRows;
    p.bytes = p.w_partial + (scratch ? round256(static_cast<size_t>(2 * p.w_slices * ffn * hidden) * 4) : 0);
    return p;
}

template <typename T, int MODE, int BLOCKS, int PARTS = 1>
cudaError_t launch_gated(const GatedMaps& maps, const GatedArgs& a, int64_t units, cudaStream_t s) {
    static int done[kMaxDevices];
    const cudaError_t e = allow_max_dynamic_smem(gated_kernel<T, MODE, BLOCKS, PARTS>, done);
    if (e != cudaSuccess) return e;
    const int64_t pairs = std::min<int64_t>(units, kPairs);
    return launch_pdl(gated_kernel<T, MODE, BLOCKS, PARTS>, dim3(static_cast<unsigned>(2 * pairs)), dim3(kThreads), kSmemBytes, s, maps, a);
}

// The forward's tiles, or with dh those of dg (out) and du (out2).
template <typename T, int MODE>
cudaError_t launch_tiles(void* out, void* out2, const void* dh, const void* x, const void* wg, const void* wu,
                         const GatedShape& sh, cudaStream_t s) {
    GatedArgs a = {};
    a.rows = static_cast<int>(sh.rows);
    a.hidden = static_cast<int>(sh.hidden);
    a.ffn = static_cast<int>(sh.ffn);
    a.act = static_cast<int>(sh.act);
    a.half = half_columns(sh.rows, sh.hidden, sh.ffn);
    a.m_tiles = static_cast<int>(ceil_div(sh.rows, kTileM));
    a.n_tiles = static_cast<int>(ceil_div(sh.ffn, a.half));
    // The last round's tiles, where there are no more than half as many as pairs, are halved: all pairs have a share
    // of them (forward 772 x 2008 x 664: 24 tiles, 48 halves, 17.5 -> 13.4 us).
    const int tiles = a.m_tiles * a.n_tiles, last = tiles % kPairs;
    a.whole_tiles = a.half == kMostHalf && 2 * last <= kPairs ? tiles - last : tiles;
    a.k_blocks = static_cast<int>(ceil_div(sh.hidden, kBlockK));
    a.row_box = static_cast<int>(std::min<int64_t>(sh.rows, 128));
    a.dh = dh;
    a.out = out;
    a.out2 = out2;
    GatedMaps maps = {};
    LS_CUDA(make_map<T>(&maps.a, x, sh.hidden, sh.rows, sh.hidden, a.row_box));
    LS_CUDA(make_map<T>(&maps.b, wg, sh.hidden, sh.ffn, sh.hidden, a.half));
    LS_CUDA(make_map<T>(&maps.b2, wu, sh.hidden, sh.ffn, sh.hidden, a.half));
    if (a.whole_tiles < tiles) {
        LS_CUDA(make_map<T>(&maps.wa, wg, sh.hidden, sh.ffn, sh.hidden, a.half / 2));
        LS_CUDA(make_map<T>(&maps.wa2, wu, sh.hidden, sh.ffn, sh.hidden, a.half / 2));
    }
    LS_CUDA(make_map<T>(&maps.out, out, sh.ffn, sh.rows, sh.ffn, 32));
    if (MODE == kGrad) LS_CUDA(make_map<T>(&maps.out2, out2, sh.ffn, sh.rows, sh.ffn, 32));
    const int64_t units = 2 * static_cast<int64_t>(tiles) - a.whole_tiles;
    if (sh.hidden > kMostColumns) {  // half of the sums in each accumulator, which the epilogue adds in FP32
        a.part_blocks = static_cast<int>(2 * ceil_div(a.k_blocks, 4));  // even, as a stage may have two
        return a.half <= 64 ? launch_gated<T, MODE, 2, 2>(maps, a, units, s) : launch_gated<T, MODE, 1, 2>(maps, a, units, s);
    }
    return a.half <= 64 ? launch_gated<T, MODE, 2>(maps, a, units, s) : launch_gated<T, MODE, 1>(maps, a, units, s);
}

template <typename T>
cudaError_t bwd(void* dx, void* dwg, void* dwu, bool f32, const void* dh, const void* x, const void* wg, const void* wu,
                const GatedShape& sh, const GatedPlan& p, void* workspace, cudaStream_t s) {
    char* ws = static_cast<char*>(workspace);
    void *dg = ws, *du = ws + p.du;
    void *dg_low = p.pairs ? ws + 2 * p.du : nullptr, *du_low = p.pairs ? ws + 3 * p.du : nullptr;
    float* partial = reinterpret_cast<float*>(ws + p.partial);
    float* w_partial = reinterpret_cast<float*>(ws + p.w_partial);
    if (gated_few_rows(sh.rows, sh.hidden, sh.ffn))
        LS_CUDA(launch_gated_few(std::is_same<T, bf16>::value ? LS_BF16 : LS_F16, dg, du, dh, x, wg, wu, sh, dg_low, du_low, s));
    else
        LS_CUDA((launch_tiles<T, kGrad>(dg, du, dh, x, wg, wu, sh, s)));
    GatedArgs a = {};
    a.rows = static_cast<int>(sh.rows);
    a.hidden = static_cast<int>(sh.hidden);
    a.ffn = static_cast<int>(sh.ffn);
    a.row_box = static_cast<int>(std::min<int64_t>(sh.rows, 128));
    a.width = static_cast<int>(p.width);
    a.h_tiles = static_cast<int>(ceil_div(sh.hidden, p.width));
    a.f_blocks = static_cast<int>(ceil_div(sh.ffn, kBlockK));
    a.pairs = p.pairs;
    a.x_blocks = (p.pairs ? 4 : 2) * a.f_blocks;
    a.slices = static_cast<int>(p.slices);
    a.slice_blocks = static_cast<int>(p.slice_blocks);
    a.x_units = dx ? static_cast<int>(ceil_div(sh.rows, kTileM)) * a.h_tiles : 0;
    a.w_tiles = static_cast<int>(ceil_div(sh.ffn, kTileM)) * a.h_tiles;
    a.w_slice_blocks = static_cast<int>(p.w_slice_blocks);
    a.w_partial = dwg && p.w_slices > 1;
    a.w_units = dwg ? static_cast<int>(p.w_slices) * 2 * a.w_tiles : 0;
    a.w_first = p.w_first;
    a.x_partial = p.slices > 1;
    GatedMaps m = {};
    LS_CUDA(make_map<T>(&m.a, dg, sh.ffn, sh.rows, sh.ffn, a.row_box));
    LS_CUDA(make_map<T>(&m.a2, du, sh.ffn, sh.rows, sh.ffn, a.row_box));
    LS_CUDA(make_map<T>(&m.b, wg, sh.hidden, sh.ffn, sh.hidden, 64));
    LS_CUDA(make_map<T>(&m.b2, wu, sh.hidden, sh.ffn, sh.hidden, 64));
    const int w_rows = p.pairs ? kPairRows : kBlockK;
    LS_CUDA(make_map<T>(&m.wa, dg, sh.ffn, sh.rows, sh.ffn, w_rows));
    LS_CUDA(make_map<T>(&m.wa2, du, sh.ffn, sh.rows, sh.ffn, w_rows));
    LS_CUDA(make_map<T>(&m.wb, x, sh.hidden, sh.rows, sh.hidden, w_rows));
    if (p.pairs) {
        LS_CUDA(make_map<T>(&m.a_low, dg_low, sh.ffn, sh.rows, sh.ffn, a.row_box));
        LS_CUDA(make_map<T>(&m.a2_low, du_low, sh.ffn, sh.rows, sh.ffn, a.row_box));
        LS_CUDA(make_map<T>(&m.wa_low, dg_low, sh.ffn, sh.rows, sh.ffn, w_rows));
        LS_CUDA(make_map<T>(&m.wa2_low, du_low, sh.ffn, sh.rows, sh.ffn, w_rows));
    }
    if (dx && a.x_partial)
        LS_CUDA(make_map<float>(&m.out, partial, sh.hidden, sh.rows, sh.hidden, 32, p.slices));
    else if (dx)
        LS_CUDA(make_map<T>(&m.out, dx, sh.hidden, sh.rows, sh.hidden, 32));
    // dW's sums over the rows, kMostRows of them at a time: added to FP32 gradients, or to scratch.
    const bool scratch = dwg && (a.w_partial || (!f32 && sh.rows > kMostRows));
    const int64_t w_elements = sh.ffn * sh.hidden;
    a.w_f32 = f32 || scratch;
    if (scratch) {
        const int64_t depth = a.w_partial ? p.w_slices : 0;
        LS_CUDA(make_map<float>(&m.out2, w_partial, sh.hidden, sh.ffn, sh.hidden, 32, depth));
        LS_CUDA(make_map<float>(&m.out3, w_partial + p.w_slices * w_elements, sh.hidden, sh.ffn, sh.hidden, 32, depth));
    } else if (dwg && f32) {
        LS_CUDA(make_map<float>(&m.out2, dwg, sh.hidden, sh.ffn, sh.hidden, 32));
        LS_CUDA(make_map<float>(&m.out3, dwu, sh.hidden, sh.ffn, sh.hidden, 32));
    } else if (dwg) {
        LS_CUDA(make_map<T>(&m.out2, dwg, sh.hidden, sh.ffn, sh.hidden, 32));
        LS_CUDA(make_map<T>(&m.out3, dwu, sh.hidden, sh.ffn, sh.hidden, 32));
    }
    a.w_add = f32 && !a.w_partial;
    const int64_t row_blocks = ceil_div(sh.rows, kBlockK), most = kMostRows / kBlockK;
    for (int64_t kb = 0; kb < (dwg ? row_blocks : 1); kb += most) {
        a.w_kb0 = static_cast<int>(kb);
        a.w_k_blocks = static_cast<int>(std::min(most, row_blocks - kb));
        const int64_t x_units = static_cast<int64_t>(a.slices) * a.x_units;
        if (!a.w_partial) a.w_slice_blocks = a.w_k_blocks;
        const int64_t w_len = unit_length(p.width, a.w_slice_blocks, p.w_slices > 1);
        const Deal d(a.w_first ? a.w_units : x_units, a.w_first ? w_len : p.x_len, a.w_first ? x_units : a.w_units,
                     a.w_first ? p.x_len : w_len);
        a.pairs1 = static_cast<int>(d.pairs1);
        a.first_short1 = static_cast<int>((a.w_first ? x_units : a.w_units) - d.short1);
        if (a.width == kTileN)
            LS_CUDA((launch_gated<T, kOut, 1>(m, a, x_units + a.w_units, s)));
        else
            LS_CUDA((launch_gated<T, kOut, 2>(m, a, x_units + a.w_units, s)));
        a.x_units = 0;
        a.w_add = true;
    }
    JoinArgs j = {};
    unsigned joins = 0;
    int64_t vecs = 0;
    auto add = [&](void* out, const float* part, int64_t slices, int64_t elements, bool to_f32) {
        j.out[joins] = out;
        j.part[joins] = part;
        j.slices[joins] = static_cast<int>(slices);
        j.vecs[joins] = elements / kVec;
        j.f32[joins++] = to_f32;
        vecs = std::max(vecs, elements / kVec);
    };
    if (scratch) add(dwg, w_partial, p.w_slices, w_elements, f32);
    if (scratch) add(dwu, w_partial + p.w_slices * w_elements, p.w_slices, w_elements, f32);
    if (dx && a.x_partial) add(dx, partial, p.slices, sh.rows * sh.hidden, false);
    if (joins > 0)
        LS_CUDA(launch_pdl(join_kernel<T>, dim3(static_cast<unsigned>(ceil_div(vecs, 256)), joins), dim3(256), 0, s, j));
    return cudaSuccess;
}

}  // namespace

GatedPlan gated_plan(int64_t rows, int64_t hidden, int64_t ffn) { return make_plan(rows, hidden, ffn); }

cudaError_t launch_gated_fwd(ls_dtype dt, void* h, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, cudaStream_t s) {
    if (gated_few_rows(sh.rows, sh.hidden, sh.ffn)) return launch_gated_few(dt, h, nullptr, nullptr, x, wg, wu, sh, nullptr, nullptr, s);
    if (dt == LS_F16) return launch_tiles<__half, kFwd>(h, nullptr, nullptr, x, wg, wu, sh, s);
    return launch_tiles<bf16, kFwd>(h, nullptr, nullptr, x, wg, wu, sh, s);
}

cudaError_t launch_gated_bwd(ls_dtype dt, void* dx, void* dwg, void* dwu, bool f32_dweight,
                             const void* dh, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, const GatedPlan& p, void* workspace, cudaStream_t s) {
    if (dt == LS_F16) return bwd<__half>(dx, dwg, dwu, f32_dweight, dh, x, wg, wu, sh, p, workspace, s);
    return bwd<bf16>(dx, dwg, dwu, f32_dweight, dh, x, wg, wu, sh, p, workspace, s);
}

cudaError_t launch_block_wait_selftest(uint32_t polls, cudaStream_t s) {
    wait_selftest_kernel<<<1, 64, 0, s>>>(polls);
    return cudaGetLastError();
}

cudaError_t gated_take_device_error(unsigned int* flags) { return take_device_error_word(flags); }

}  // namespace ls
