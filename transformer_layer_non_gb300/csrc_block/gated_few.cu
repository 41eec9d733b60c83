// gated_few.cu -- the gated block's forward for the few rows of a decoding step.
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
#include <algorithm>

#include "../csrc_vocab/vec.cuh"
#include "block_internal.h"
#include "gated_act.cuh"

namespace ls {
namespace {

constexpr int kFewThreads = 128, kFewWarps = kFewThreads / 32;
constexpr int kFewStep = 32;    // values of K for a warp's load: 8 for each of four lanes of a row
constexpr int64_t kMostFew = 16;  // rows of x

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

// NT: groups of 8 rows of x.  U: a warp's steps in flight; with six CTAs of four warps on an SM (four for NT = 2,
// whose registers hold more of x) 4 of them, 8 warps or 8 steps are slower (1 x 1280 x 5120: 4.0 us; 5.8 and 4.7).
template <typename T, int NT, int U>
__global__ void __launch_bounds__(kFewThreads, NT == 1 ? 6 : 4)
few_kernel(T* __restrict__ h, const T* __restrict__ x, const T* __restrict__ wg, const T* __restrict__ wu,
           const __grid_constant__ FewArgs a) {
    __shared__ float part[kFewWarps][32][4 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = lane >> 2, k8 = (lane & 3) * kVec;  // this lane's row of a group of 8, and its place in a step
    const int f0 = blockIdx.x * 8;
    const int steps = (a.hidden + kFewStep - 1) / kFewStep;
    const int begin = steps * warp / kFewWarps, end = steps * (warp + 1) / kFewWarps;
    const T* pg = wg + static_cast<int64_t>(f0 + r) * a.hidden;
    const T* pu = wu + static_cast<int64_t>(f0 + r) * a.hidden;
    pdl_enter();
    uint4 g[U], u[U], b[U][NT];
    auto load = [&](int slot, int step) {
        const int k = step * kFewStep + k8;
        const bool there = step < end && k < a.hidden;
        const uint4 zero = make_uint4(0, 0, 0, 0);
        g[slot] = there ? ld16(pg + k) : zero;
        u[slot] = there ? ld16(pu + k) : zero;
#pragma unroll
        for (int n = 0; n < NT; ++n)
            b[slot][n] = there && n * 8 + r < a.rows ? ld16(x + static_cast<int64_t>(n * 8 + r) * a.hidden + k) : zero;
    };
#pragma unroll
    for (int i = 0; i < U; ++i) load(i, begin + i);
    float c[NT][4] = {};
    for (int s = begin; s < end; s += U) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma16816<T>(c[n], g[i].x, u[i].x, g[i].y, u[i].y, b[i][n].x, b[i][n].y);
                mma16816<T>(c[n], g[i].z, u[i].z, g[i].w, u[i].w, b[i][n].z, b[i][n].w);
            }
            load(i, s + i + U);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[warp][lane][4 * n + j] = c[n][j];
    __syncthreads();
    // One thread for each element: column f of the 8, row t of x.
    const int f = threadIdx.x & 7, t = threadIdx.x >> 3;
    if (t >= 8 * NT || t >= a.rows) return;
    const int from = f * 4 + (t & 7) / 2, e = (t >> 3) * 4 + (t & 1);  // the lane that has it, and where
    float sg = part[0][from][e], su = part[0][from][e + 2];
    for (int w = 1; w < kFewWarps; ++w) {
        sg += part[w][from][e];
        su += part[w][from][e + 2];
    }
    const float v = a.act == LS_ACT_SILU        ? act_of<LS_ACT_SILU>(sg).a
                    : a.act == LS_ACT_GELU      ? act_of<LS_ACT_GELU>(sg).a
                    : a.act == LS_ACT_GELU_TANH ? act_of<LS_ACT_GELU_TANH>(sg).a
                                                : act_of<LS_ACT_RELU>(sg).a;
    h[static_cast<int64_t>(t) * a.ffn + f0 + f] = from_f32<T>(v * su);
}

template <typename T>
cudaError_t launch(void* h, const void* x, const void* wg, const void* wu, const GatedShape& sh, cudaStream_t s) {
    const FewArgs a{static_cast<int>(sh.rows), static_cast<int>(sh.hidden), static_cast<int>(sh.ffn),
                    static_cast<int>(sh.act)};
    return launch_pdl(sh.rows <= 8 ? few_kernel<T, 1, 4> : few_kernel<T, 2, 4>, dim3(static_cast<unsigned>(sh.ffn / 8)),
                      dim3(kFewThreads), 0, s, static_cast<T*>(h), static_cast<const T*>(x), static_cast<const T*>(wg),
                      static_cast<const T*>(wu), a);
}

}  // namespace

bool gated_few_rows(int64_t rows) { return rows <= kMostFew; }

cudaError_t launch_gated_few(ls_dtype dt, void* h, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, cudaStream_t s) {
    return dt == LS_F16 ? launch<__half>(h, x, wg, wu, sh, s) : launch<bf16>(h, x, wg, wu, sh, s);
}

}  // namespace ls
