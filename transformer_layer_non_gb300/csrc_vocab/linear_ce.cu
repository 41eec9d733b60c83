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
// FP16 has no exponent range for dloss * p (1/rows times 1/vocab), so g is
// stored as g * 2^s with 2^s max|dloss| <= 2^14 and the factor is taken out of
// the FP32 sums again; BF16 has FP32's range and s = 0.
#include <math.h>

#include <type_traits>

#include "vec.cuh"
#include "vocab_internal.h"

namespace ls {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct HeadArgs {
    int64_t rows, hidden, vocab;
    int64_t col0, cols;   // this piece of the vocabulary
    int64_t ldg;
    float eps;
    int32_t ignore_index;
};

__device__ __forceinline__ bool used_target(int32_t y, const HeadArgs& a) {
    return y != a.ignore_index && y >= 0 && y < a.vocab;
}

// 64 x 64 tile of C = A B^T-like products with any strides: A(i, k) = a[i * ai + k * ak],
// B(j, k) = b[j * bj + k * bk]; thread (tx, ty) owns 4 x 4 results.
template <typename T>
__device__ __forceinline__ void tile_product(float (&acc)[4][4], const T* a, int64_t ai, int64_t ak,
                                             const T* b, int64_t bj, int64_t bk, int64_t m,
                                             int64_t n, int64_t k, int64_t i0, int64_t j0) {
    __shared__ float sa[16][kTile + 1], sb[16][kTile + 1];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] = 0.f;
    for (int64_t k0 = 0; k0 < k; k0 += 16) {
        for (int t = threadIdx.x; t < 16 * kTile; t += kThreads) {
            const int kk = t & 15, r = t >> 4;
            const bool in_k = k0 + kk < k;
            sa[kk][r] = in_k && i0 + r < m ? to_f32(a[(i0 + r) * ai + (k0 + kk) * ak]) : 0.f;
            sb[kk][r] = in_k && j0 + r < n ? to_f32(b[(j0 + r) * bj + (k0 + kk) * bk]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    acc[p][q] = fmaf(sa[kk][ty * 4 + p], sb[kk][tx * 4 + q], acc[p][q]);
        __syncthreads();
    }
}

// part: [3][tiles][rows]: maximum, sum of exponentials, plain sum.
template <typename T>
__global__ void __launch_bounds__(kThreads)
logit_stats_kernel(float* __restrict__ part, float* __restrict__ zy, const T* __restrict__ x,
                   const T* __restrict__ w, const int32_t* __restrict__ target,
                   const __grid_constant__ HeadArgs a) {
    __shared__ float z[kTile][kTile + 1];
    pdl_enter();
    const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kTile;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kTile;
    float acc[4][4];
    tile_product<T>(acc, x, a.hidden, 1, w, a.hidden, 1, a.rows, a.vocab, a.hidden, i0, j0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int p = 0; p < 4; ++p)
        for (int q = 0; q < 4; ++q) z[ty * 4 + p][tx * 4 + q] = acc[p][q];
    __syncthreads();
    const int64_t i = i0 + threadIdx.x;
    if (threadIdx.x >= kTile || i >= a.rows) return;
    const int n = static_cast<int>(min(static_cast<int64_t>(kTile), a.vocab - j0));
    float m = -INFINITY, l = 0.f, s = 0.f;
    for (int j = 0; j < n; ++j) m = fmaxf(m, z[threadIdx.x][j]);
    for (int j = 0; j < n; ++j) {
        l += exp2_approx((z[threadIdx.x][j] - m) * kLog2e);
        s += z[threadIdx.x][j];
    }
    const int64_t stride = static_cast<int64_t>(gridDim.x) * a.rows;
    float* o = part + blockIdx.x * a.rows + i;
    o[0] = m;
    o[stride] = l;
    o[2 * stride] = s;
    const int64_t y = target[i];
    if (y >= j0 && y < j0 + n) zy[i] = z[threadIdx.x][y - j0];
}

__global__ void __launch_bounds__(kThreads)
merge_stats_kernel(float* __restrict__ loss, float* __restrict__ lse_out,
                   const float* __restrict__ part, const float* __restrict__ zy,
                   const int32_t* __restrict__ target, int64_t tiles,
                   const __grid_constant__ HeadArgs a) {
    pdl_enter();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (i >= a.rows) return;
    float m = -INFINITY, l = 0.f, s = 0.f;
    const int64_t stride = tiles * a.rows;
    for (int64_t t = 0; t < tiles; ++t) {
        const float m2 = part[t * a.rows + i], l2 = part[stride + t * a.rows + i];
        const float mm = fmaxf(m, m2);
        l = l * exp2_approx((m - mm) * kLog2e) + l2 * exp2_approx((m2 - mm) * kLog2e);
        m = mm;
        s += part[2 * stride + t * a.rows + i];
    }
    const float lse = m + logf(l);
    if (lse_out) lse_out[i] = lse;
    loss[i] = used_target(target[i], a)
                  ? (1.f - a.eps) * (lse - zy[i]) +
                        (a.eps > 0.f ? a.eps * (lse - s / static_cast<float>(a.vocab)) : 0.f)
                  : 0.f;
}

// scale[0] = 2^s, scale[1] = 2^-s.
__global__ void __launch_bounds__(1024)
grad_scale_kernel(float* __restrict__ scale, const float* __restrict__ dloss, int64_t rows,
                  bool scaled) {
    __shared__ float sm[32];
    pdl_enter();
    float m = dloss ? 0.f : 1.f;
    if (dloss && scaled)
        for (int64_t i = threadIdx.x; i < rows; i += 1024) {
            const float d = fabsf(dloss[i]);
            if (d < INFINITY) m = fmaxf(m, d);
        }
    m = group_max<32>(m);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) {
        m = group_max<32>(sm[threadIdx.x]);
        if (threadIdx.x == 0) {
            int s = 0;
            if (scaled && m > 0.f) {
                int ex;
                frexpf(m, &ex);  // m < 2^ex
                s = min(100, max(-100, 14 - ex));
            }
            scale[0] = ldexpf(1.f, s);
            scale[1] = ldexpf(1.f, -s);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
logit_grad_kernel(T* __restrict__ g, const T* __restrict__ x, const T* __restrict__ w,
                  const int32_t* __restrict__ target, const float* __restrict__ lse,
                  const float* __restrict__ dloss, const float* __restrict__ scale,
                  const __grid_constant__ HeadArgs a) {
    pdl_enter();
    const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kTile;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kTile;
    float acc[4][4];
    tile_product<T>(acc, x, a.hidden, 1, w + a.col0 * a.hidden, a.hidden, 1, a.rows, a.cols,
                    a.hidden, i0, j0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const float q0 = a.eps / static_cast<float>(a.vocab);
    for (int p = 0; p < 4; ++p) {
        const int64_t i = i0 + ty * 4 + p;
        if (i >= a.rows) break;
        const int64_t y = target[i];
        const bool used = used_target(static_cast<int32_t>(y), a);
        const float d = (dloss ? dloss[i] : 1.f) * scale[0];
        for (int q = 0; q < 4; ++q) {
            const int64_t j = j0 + tx * 4 + q;
            if (j >= a.cols) break;
            const float t = q0 + (a.col0 + j == y ? 1.f - a.eps : 0.f);
            g[i * a.ldg + j] =
                from_f32<T>(used ? d * (exp2_approx((acc[p][q] - lse[i]) * kLog2e) - t) : 0.f);
        }
    }
}

// dx accumulator (FP32 [rows, hidden]) (+)= g W_piece; the last piece writes dx.
template <typename T>
__global__ void __launch_bounds__(kThreads)
dx_kernel(float* acc_buf, T* __restrict__ dx, const T* __restrict__ g, const T* __restrict__ w,
          const float* __restrict__ scale, bool first, bool last,
          const __grid_constant__ HeadArgs a) {
    pdl_enter();
    const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kTile;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kTile;
    float acc[4][4];
    tile_product<T>(acc, g, a.ldg, 1, w + a.col0 * a.hidden, 1, a.hidden, a.rows, a.hidden, a.cols,
                    i0, j0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int p = 0; p < 4; ++p) {
        const int64_t i = i0 + ty * 4 + p;
        for (int q = 0; q < 4; ++q) {
            const int64_t j = j0 + tx * 4 + q;
            if (i >= a.rows || j >= a.hidden) continue;
            float v = acc[p][q];
            if (!first) v += acc_buf[i * a.hidden + j];
            if (last)
                dx[i * a.hidden + j] = from_f32<T>(v * scale[1]);
            else
                acc_buf[i * a.hidden + j] = v;
        }
    }
}

template <typename T, typename D>
__global__ void __launch_bounds__(kThreads)
dweight_kernel(D* dw, const T* __restrict__ g, const T* __restrict__ x,
               const float* __restrict__ scale, const __grid_constant__ HeadArgs a) {
    pdl_enter();
    const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kTile;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * kTile;
    float acc[4][4];
    tile_product<T>(acc, g, 1, a.ldg, x, 1, a.hidden, a.cols, a.hidden, a.rows, i0, j0);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int p = 0; p < 4; ++p) {
        const int64_t i = i0 + ty * 4 + p;
        for (int q = 0; q < 4; ++q) {
            const int64_t j = j0 + tx * 4 + q;
            if (i >= a.cols || j >= a.hidden) continue;
            D* o = dw + (a.col0 + i) * a.hidden + j;
            float v = acc[p][q] * scale[1];
            if constexpr (sizeof(D) == 4) v += *o;
            *o = from_f32<D>(v);
        }
    }
}

// Pieces: gradients of the logits of `cols` vocabulary entries at a time, about 128 MB.
constexpr int64_t kPieceBytes = int64_t{128} << 20;

struct HeadPlan {
    int64_t tiles, cols;
    size_t part, zy, scale, g, acc, fwd_bytes, bwd_bytes;
    HeadPlan(int64_t rows, int64_t hidden, int64_t vocab) {
        tiles = (vocab + kTile - 1) / kTile;
        part = 0;
        zy = static_cast<size_t>(3 * tiles * rows) * 4;
        fwd_bytes = zy + static_cast<size_t>(rows) * 4;
        cols = kPieceBytes / 2 / rows / 256 * 256;
        if (cols < 2048) cols = 2048;
        const int64_t all = (vocab + 255) / 256 * 256;
        if (cols > all) cols = all;
        scale = 0;
        g = 256;
        acc = g + static_cast<size_t>(rows * cols) * 2;
        bwd_bytes = acc + (cols < vocab ? static_cast<size_t>(rows * hidden) * 4 : 0);
    }
    size_t bytes() const { return fwd_bytes > bwd_bytes ? fwd_bytes : bwd_bytes; }
};

HeadArgs make_args(const HeadShape& sh) {
    HeadArgs a;
    a.rows = sh.rows;
    a.hidden = sh.hidden;
    a.vocab = sh.vocab;
    a.col0 = 0;
    a.cols = sh.vocab;
    a.ldg = 0;
    a.eps = sh.eps;
    a.ignore_index = sh.ignore_index;
    return a;
}

unsigned tiles_of(int64_t n) { return static_cast<unsigned>((n + kTile - 1) / kTile); }

template <typename T>
cudaError_t fwd(float* loss, float* lse, const void* x, const void* w, const int32_t* target,
                const HeadShape& sh, void* workspace, cudaStream_t s) {
    const HeadPlan p(sh.rows, sh.hidden, sh.vocab);
    const HeadArgs a = make_args(sh);
    char* ws = static_cast<char*>(workspace);
    float* part = reinterpret_cast<float*>(ws + p.part);
    float* zy = reinterpret_cast<float*>(ws + p.zy);
    cudaError_t e = launch_pdl(logit_stats_kernel<T>, dim3(tiles_of(sh.vocab), tiles_of(sh.rows)),
                               dim3(kThreads), 0, s, part, zy, static_cast<const T*>(x),
                               static_cast<const T*>(w), target, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(merge_stats_kernel,
                      dim3(static_cast<unsigned>((sh.rows + kThreads - 1) / kThreads)),
                      dim3(kThreads), 0, s, loss, lse, part, zy, target, p.tiles, a);
}

template <typename T>
cudaError_t bwd(void* dx, void* dweight, bool f32_dweight, const void* x, const void* w,
                const int32_t* target, const float* lse, const float* dloss, const HeadShape& sh,
                void* workspace, cudaStream_t s) {
    const HeadPlan p(sh.rows, sh.hidden, sh.vocab);
    HeadArgs a = make_args(sh);
    a.ldg = p.cols;
    char* ws = static_cast<char*>(workspace);
    float* scale = reinterpret_cast<float*>(ws + p.scale);
    T* g = reinterpret_cast<T*>(ws + p.g);
    float* acc = reinterpret_cast<float*>(ws + p.acc);
    const T* xt = static_cast<const T*>(x);
    const T* wt = static_cast<const T*>(w);
    cudaError_t e = launch_pdl(grad_scale_kernel, dim3(1), dim3(1024), 0, s, scale, dloss, sh.rows,
                               std::is_same<T, __half>::value);
    for (int64_t c = 0; e == cudaSuccess && c < sh.vocab; c += p.cols) {
        a.col0 = c;
        a.cols = sh.vocab - c < p.cols ? sh.vocab - c : p.cols;
        e = launch_pdl(logit_grad_kernel<T>, dim3(tiles_of(a.cols), tiles_of(sh.rows)),
                       dim3(kThreads), 0, s, g, xt, wt, target, lse, dloss, scale, a);
        if (e == cudaSuccess && dx)
            e = launch_pdl(dx_kernel<T>, dim3(tiles_of(sh.hidden), tiles_of(sh.rows)),
                           dim3(kThreads), 0, s, acc, static_cast<T*>(dx), g, wt, scale, c == 0,
                           c + a.cols == sh.vocab, a);
        const dim3 wgrid(tiles_of(sh.hidden), tiles_of(a.cols));
        if (e == cudaSuccess && dweight)
            e = f32_dweight ? launch_pdl(dweight_kernel<T, float>, wgrid, dim3(kThreads), 0, s,
                                         static_cast<float*>(dweight), g, xt, scale, a)
                            : launch_pdl(dweight_kernel<T, T>, wgrid, dim3(kThreads), 0, s,
                                         static_cast<T*>(dweight), g, xt, scale, a);
    }
    return e;
}

}  // namespace

size_t linear_ce_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab) {
    return HeadPlan(rows, hidden, vocab).bytes();
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

cudaError_t linear_ce_take_device_error(unsigned int* flags) {
    return take_device_error_word(flags);
}

}  // namespace ls
