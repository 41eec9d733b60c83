// gated.cu -- the gated feed-forward block: h = act(x Wg^T) * (x Wu^T), and its
// gradients.
//
// Simple tiles: 64 x 64 outputs for each CTA, FP32 products of operands staged
// through shared memory.  The backward computes both sums again, writes dg and
// du in the storage type, and multiplies them with the weights and with x.
#include <algorithm>

#include "../csrc_vocab/tc_tile.cuh"
#include "block_internal.h"

namespace ls {
namespace {

constexpr int kTile = 64, kStep = 16, kThreads = 256;

struct ActValue {
    float a, slope;  // act(g), act'(g)
};
__device__ __forceinline__ ActValue act_of(float g, int act) {
    if (act == LS_ACT_RELU) return {g > 0.f ? g : 0.f, g > 0.f ? 1.f : 0.f};
    if (act == LS_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-g));
        return {g * s, s * (1.f + g * (1.f - s))};
    }
    if (act == LS_ACT_GELU) {
        const float phi = 0.5f * erfcf(-g * 0.70710678f);
        return {g * phi, phi + g * 0.39894228f * expf(-0.5f * g * g)};
    }
    const float k = 0.79788456f, t = tanhf(k * (g + 0.044715f * g * g * g));
    return {0.5f * g * (1.f + t), 0.5f * (1.f + t) + 0.5f * g * (1.f - t * t) * k * (1.f + 0.134145f * g * g)};
}

// A matrix of which rows or columns are contiguous.
template <typename T> struct Matrix {
    const T* p;
    int64_t row, col;  // strides
    int rows, cols;
    __device__ __forceinline__ float at(int r, int c) const {
        return r < rows && c < cols ? to_f32(p[r * row + c * col]) : 0.f;
    }
};

// Both products of a 64 x 64 tile: a (M x K) with b[0..N) (N x K), each thread 4 x 4 of it.
template <typename T>
__device__ __forceinline__ void multiply(const Matrix<T>& a, const Matrix<T>& b, int m0, int n0, float (&acc)[4][4]) {
    __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
    const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    for (int k0 = 0; k0 < a.cols; k0 += kStep) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTile * kStep; i += kThreads) {
            const int r = i / kStep, k = i % kStep;
            sa[k][r] = a.at(m0 + r, k0 + k);
            sb[k][r] = b.at(n0 + r, k0 + k);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
    }
}

// h, or with dh its gradients dg and du.
template <typename T>
__global__ void __launch_bounds__(kThreads)
gated_kernel(T* __restrict__ h, T* __restrict__ dg, T* __restrict__ du, const T* __restrict__ dh, Matrix<T> x, Matrix<T> wg,
             Matrix<T> wu, int act) {
    pdl_enter();
    const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float g[4][4] = {}, u[4][4] = {};
    multiply(x, wg, m0, n0, g);
    multiply(x, wu, m0, n0, u);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = m0 + ty + 16 * i, f = n0 + tx + 16 * j;
            if (r >= x.rows || f >= wg.rows) continue;
            const int64_t e = static_cast<int64_t>(r) * wg.rows + f;
            const ActValue v = act_of(g[i][j], act);
            if (dh) {
                const float d = to_f32(dh[e]);
                dg[e] = from_f32<T>(d * u[i][j] * v.slope);
                du[e] = from_f32<T>(d * v.a);
            } else {
                h[e] = from_f32<T>(v.a * u[i][j]);
            }
        }
}

// out (+)= a b^T + a2 b2^T
template <typename T, typename O>
__global__ void __launch_bounds__(kThreads)
product_kernel(O* __restrict__ out, Matrix<T> a, Matrix<T> b, Matrix<T> a2, Matrix<T> b2, bool add) {
    pdl_enter();
    const int m0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile, ty = threadIdx.x / 16, tx = threadIdx.x % 16;
    float acc[4][4] = {};
    multiply(a, b, m0, n0, acc);
    if (a2.p) multiply(a2, b2, m0, n0, acc);
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int r = m0 + ty + 16 * i, c = n0 + tx + 16 * j;
            if (r >= a.rows || c >= b.rows) continue;
            const int64_t e = static_cast<int64_t>(r) * b.rows + c;
            out[e] = from_f32<O>(add ? to_f32(out[e]) + acc[i][j] : acc[i][j]);
        }
}

// rows x cols, row-major, and transposed.
template <typename T> Matrix<T> mat(const void* p, int64_t rows, int64_t cols) {
    return Matrix<T>{static_cast<const T*>(p), cols, 1, static_cast<int>(rows), static_cast<int>(cols)};
}
template <typename T> Matrix<T> transposed(const void* p, int64_t rows, int64_t cols) {
    return Matrix<T>{static_cast<const T*>(p), 1, cols, static_cast<int>(cols), static_cast<int>(rows)};
}
dim3 tiles(int64_t rows, int64_t cols) {
    return dim3(static_cast<unsigned>(ceil_div(cols, kTile)), static_cast<unsigned>(ceil_div(rows, kTile)));
}

template <typename T>
cudaError_t fwd(void* h, const void* x, const void* wg, const void* wu, const GatedShape& sh, cudaStream_t s) {
    return launch_pdl(gated_kernel<T>, tiles(sh.rows, sh.ffn), dim3(kThreads), 0, s, static_cast<T*>(h), nullptr, nullptr,
                      nullptr, mat<T>(x, sh.rows, sh.hidden), mat<T>(wg, sh.ffn, sh.hidden), mat<T>(wu, sh.ffn, sh.hidden),
                      static_cast<int>(sh.act));
}

template <typename T, typename O>
cudaError_t product(O* out, const Matrix<T>& a, const Matrix<T>& b, const Matrix<T>& a2, const Matrix<T>& b2, bool add,
                    cudaStream_t s) {
    return launch_pdl(product_kernel<T, O>, tiles(a.rows, b.rows), dim3(kThreads), 0, s, out, a, b, a2, b2, add);
}

template <typename T>
cudaError_t bwd(void* dx, void* dwg, void* dwu, bool f32, const void* dh, const void* x, const void* wg, const void* wu,
                const GatedShape& sh, void* workspace, cudaStream_t s) {
    T* dg = static_cast<T*>(workspace);
    T* du = dg + sh.rows * sh.ffn;
    LS_CUDA(launch_pdl(gated_kernel<T>, tiles(sh.rows, sh.ffn), dim3(kThreads), 0, s, nullptr, dg, du,
                       static_cast<const T*>(dh), mat<T>(x, sh.rows, sh.hidden), mat<T>(wg, sh.ffn, sh.hidden),
                       mat<T>(wu, sh.ffn, sh.hidden), static_cast<int>(sh.act)));
    const Matrix<T> none = {};
    if (dx)
        LS_CUDA(product(static_cast<T*>(dx), mat<T>(dg, sh.rows, sh.ffn), transposed<T>(wg, sh.ffn, sh.hidden),
                        mat<T>(du, sh.rows, sh.ffn), transposed<T>(wu, sh.ffn, sh.hidden), false, s));
    for (int k = 0; k < 2 && dwg; ++k) {
        const Matrix<T> a = transposed<T>(k ? du : dg, sh.rows, sh.ffn), b = transposed<T>(x, sh.rows, sh.hidden);
        void* dw = k ? dwu : dwg;
        if (f32)
            LS_CUDA(product(static_cast<float*>(dw), a, b, none, none, true, s));
        else
            LS_CUDA(product(static_cast<T*>(dw), a, b, none, none, false, s));
    }
    return cudaSuccess;
}

// Self-test of the waits' failure path: two warps wait on a barrier that expects an arrival nobody makes; the
// first whose polls run out flags the failure, the other one sees it.
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

}  // namespace

size_t gated_workspace_bytes(int64_t rows, int64_t hidden, int64_t ffn) {
    return round256(static_cast<size_t>(rows * ffn) * 4);
}

cudaError_t launch_gated_fwd(ls_dtype dt, void* h, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, cudaStream_t s) {
    return dt == LS_F16 ? fwd<__half>(h, x, wg, wu, sh, s) : fwd<bf16>(h, x, wg, wu, sh, s);
}

cudaError_t launch_gated_bwd(ls_dtype dt, void* dx, void* dwg, void* dwu, bool f32_dweight,
                             const void* dh, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, void* workspace, cudaStream_t s) {
    if (dt == LS_F16) return bwd<__half>(dx, dwg, dwu, f32_dweight, dh, x, wg, wu, sh, workspace, s);
    return bwd<bf16>(dx, dwg, dwu, f32_dweight, dh, x, wg, wu, sh, workspace, s);
}

cudaError_t launch_block_wait_selftest(uint32_t polls, cudaStream_t s) {
    wait_selftest_kernel<<<1, 64, 0, s>>>(polls);
    return cudaGetLastError();
}

cudaError_t gated_take_device_error(unsigned int* flags) { return take_device_error_word(flags); }

}  // namespace ls
