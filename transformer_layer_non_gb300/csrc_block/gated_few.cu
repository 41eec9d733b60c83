// gated_few.cu -- the gated block's forward, and dg and du, for the few rows of a
// decoding step or a small batch.
//
// Reading both weights once bounds it: 4 products for each weight and row are
// far below what any unit of the GPU does meanwhile.  So what matters is that all
// SMs read, in even shares, with as many loads in flight as there can be; a tile
// of 256 rows would leave most pairs of SMs without one (1 x 1280 x 5120: 40
// tiles for 76 pairs).  A CTA takes 8 columns of h, its warps parts of the sums.
// The products are those of one warp's matrix instruction, m16n8k16, because it
// takes its operands from registers, where 16-byte loads have put them: 16 rows
// are the 8 gate and the 8 up columns, so that a thread ends up with both sums of
// an element; 8 columns are rows of x.  The sum does not mind which of its terms
// is called k = 0, so a thread gives its 8 neighbours of a row of weights, and the
// same 8 of x, to two instructions' places.
//
// One row of 1280 x 5120 BF16 takes 4.0 us where the 26 MB of weights are in L2 (6.6
// TB/s), and 6.0 in a step that goes through 16 blocks' weights (400 MB): 4.3 TB/s of
// DRAM, of whose rate a kernel this short does not see much more than its beginning
// and end.  4096 x 14336: 35.8 us, 6.57 TB/s.  16 rows of 1280 x 5120: 6.4 and 9.1.
//
// Times of small weights are out of L2.  Up to 32 rows, and up to 64 where x is short and h has no more columns than 32
// for each pair of SMs, so that the tiles' one round is a chain of K blocks.  BF16
// forward, and by tiles of 256 rows: 24 x 496 x 1848 3.0 us and 4.6; 32 x 4096 x
// 1024 7.1 and 11.7; 32 x 1280 x 5120 7.4 and 8.7; 64 x 512 x 2048 4.1 and 4.7; 64 x
// 1280 x 2400 7.2 and 6.5; 64 x 1280 x 5120 16.1 and 9.0.
#include <algorithm>

#include "../csrc_vocab/vec.cuh"
#include "block_internal.h"
#include "gated_act.cuh"

namespace ls {
namespace {

constexpr int kFewThreads = 128, kFewWarps = kFewThreads / 32;
constexpr int kFewStep = 32;    // values of K for a warp's load: 8 for each of four lanes of a row
constexpr int64_t kFewColumns = 2432;  // 32 for each of 76 pairs
constexpr int64_t kFewHidden = 1024;   // behind it each CTA's own reads of more than 32 rows of x cost more than they save

// c += a b, with a 16 x 16 (rows), b 16 x 8 (columns) and c 16 x 8 in the instruction's layout.
template <typename T> __device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                               uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<bf16>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                 uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct FewArgs {
    int rows, hidden, ffn, act;
};

// NT: groups of 8 rows of x.  MT: groups of 8 columns of h of a CTA, which share its reads of x.  U: a warp's steps in
// flight.  GRAD: with dh, and dg and du in the place of h.
template <typename T, bool GRAD, int NT, int MT, int U, int CTAS>
__global__ void __launch_bounds__(kFewThreads, CTAS)
few_kernel(T* __restrict__ h, T* __restrict__ du, const T* __restrict__ dh, const T* __restrict__ x, const T* __restrict__ wg,
           const T* __restrict__ wu, T* __restrict__ dg_low, T* __restrict__ du_low, const __grid_constant__ FewArgs a) {
    __shared__ float part[kFewWarps][32][4 * NT * MT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, k8 = (lane & 3) * kVec;  // this lane's row of a group of 8, and its place in a step
    const int f0 = blockIdx.x * 8 * MT;
    const int steps = (a.hidden + kFewStep - 1) / kFewStep;
    const int begin = steps * warp / kFewWarps, end = steps * (warp + 1) / kFewWarps;
    const int64_t at = static_cast<int64_t>(f0 + r) * a.hidden;
    pdl_enter();
    uint4 g[U][MT], u[U][MT], b[U][NT];
    auto load = [&](int slot, int step) {
        const int k = step * kFewStep + k8;
        const bool there = step < end && k < a.hidden;
        const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const bool column = there && (MT == 1 || f0 + 8 * m < a.ffn);
            g[slot][m] = column ? ld16(wg + at + static_cast<int64_t>(8 * m) * a.hidden + k) : zero;
            u[slot][m] = column ? ld16(wu + at + static_cast<int64_t>(8 * m) * a.hidden + k) : zero;
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
            b[slot][n] = there && n * 8 + r < a.rows ? ld16(x + static_cast<int64_t>(n * 8 + r) * a.hidden + k) : zero;
    };
#pragma unroll
    for (int i = 0; i < U; ++i) load(i, begin + i);
    float c[MT][NT][4] = {};
    for (int s = begin; s < end; s += U) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma16816<T>(c[m][n], g[i][m].x, u[i][m].x, g[i][m].y, u[i][m].y, b[i][n].x, b[i][n].y);
                    mma16816<T>(c[m][n], g[i][m].z, u[i][m].z, g[i][m].w, u[i][m].w, b[i][n].z, b[i][n].w);
                }
            load(i, s + i + U);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[warp][lane][4 * (m * NT + n) + j] = c[m][n][j];
    __syncthreads();
    // One thread for each element: column f of 8 MT, row t of x.
    for (int i = threadIdx.x; i < 8 * MT * 8 * NT; i += kFewThreads) {
        const int f = i % (8 * MT), t = i / (8 * MT);
        if (t >= a.rows || (MT > 1 && f0 + f >= a.ffn)) continue;
        // the lane that has it, and where
        const int from = f % 8 * 4 + t % 8 / 2, e = 4 * (f / 8 * NT + t / 8) + (t & 1);
        float sg = part[0][from][e], su = part[0][from][e + 2];
        for (int w = 1; w < kFewWarps; ++w) {
            sg += part[w][from][e];
            su += part[w][from][e + 2];
        }
        const ActValue v = a.act == LS_ACT_SILU        ? act_of<LS_ACT_SILU>(sg)
                           : a.act == LS_ACT_GELU      ? act_of<LS_ACT_GELU>(sg)
                           : a.act == LS_ACT_GELU_TANH ? act_of<LS_ACT_GELU_TANH>(sg)
                                                       : act_of<LS_ACT_RELU>(sg);
        const int64_t o = static_cast<int64_t>(t) * a.ffn + f0 + f;
        if constexpr (GRAD) {
            const float d = to_f32(dh[o]);
            const float gg = d * su * v.slope, gu = d * v.a;
            h[o] = from_f32<T>(gg);
            du[o] = from_f32<T>(gu);
            if (dg_low) {  // what the rounding left; nothing of an infinity
                const float rg = gg - to_f32(from_f32<T>(gg)), ru = gu - to_f32(from_f32<T>(gu));
                dg_low[o] = from_f32<T>(fabsf(rg) < INFINITY ? rg : 0.f);
                du_low[o] = from_f32<T>(fabsf(ru) < INFINITY ? ru : 0.f);
            }
        } else {
            h[o] = from_f32<T>(v.a * su);
        }
    }
}

template <typename T, bool GRAD>
cudaError_t launch(void* h, void* du, const void* dh, const void* x, const void* wg, const void* wu, const GatedShape& sh,
                   void* dg_low, void* du_low, cudaStream_t s) {
    const FewArgs a{static_cast<int>(sh.rows), static_cast<int>(sh.hidden), static_cast<int>(sh.ffn),
                    static_cast<int>(sh.act)};
    // With six CTAs of four warps on an SM (fewer for more rows, whose registers hold more of x) 4 steps in flight are
    // best; 8 warps or 8 steps are slower (1 x 1280 x 5120: 4.0 us; 5.8 and 4.7).  From 17 rows on reading x costs as
    // well: 16 columns for a CTA, unless that left SMs without one (32 x 1280 x 5120: 7.4 us, of 8 columns 8.5; 32 x
    // 4096 x 1024: 10.4 and 7.0).
    auto kernel = few_kernel<T, GRAD, 1, 1, 4, 6>;
    int columns = 8;
    if (sh.rows > 32) {
        kernel = few_kernel<T, GRAD, 8, 1, 2, 4>;
    } else if (sh.rows > 16 && sh.ffn > kFewColumns) {
        kernel = few_kernel<T, GRAD, 4, 2, 2, 3>;
        columns = 16;
    } else if (sh.rows > 16) {
        kernel = few_kernel<T, GRAD, 4, 1, 3, 4>;
    } else if (sh.rows > 8) {
        kernel = few_kernel<T, GRAD, 2, 1, 4, 4>;
    }
    return launch_pdl(kernel, dim3(static_cast<unsigned>((sh.ffn + columns - 1) / columns)), dim3(kFewThreads), 0, s,
                      static_cast<T*>(h), static_cast<T*>(du), static_cast<const T*>(dh), static_cast<const T*>(x),
                      static_cast<const T*>(wg), static_cast<const T*>(wu), static_cast<T*>(dg_low), static_cast<T*>(du_low), a);
}

}  // namespace

bool gated_few_rows(int64_t rows, int64_t hidden, int64_t ffn) {
    return rows <= 32 || (rows <= 64 && ffn <= kFewColumns && hidden <= kFewHidden);
}

cudaError_t launch_gated_few(ls_dtype dt, void* h, void* du, const void* dh, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, void* dg_low, void* du_low, cudaStream_t s) {
    if (dt == LS_F16)
        return dh ? launch<__half, true>(h, du, dh, x, wg, wu, sh, dg_low, du_low, s)
                  : launch<__half, false>(h, du, dh, x, wg, wu, sh, dg_low, du_low, s);
    return dh ? launch<bf16, true>(h, du, dh, x, wg, wu, sh, dg_low, du_low, s)
              : launch<bf16, false>(h, du, dh, x, wg, wu, sh, dg_low, du_low, s);
}

}  // namespace ls
