// clip.cu -- the global norm of many gradients, gradients scaled by a factor
// in device memory, and the trainer update with such a factor.
//
// All three stream: the norm reads every gradient once, scaling reads and
// writes it, the update moves 22 bytes (16-bit storage) an element.  DRAM
// bounds them, and for small models the launches.
//
// Many tensors go through one launch: a table of addresses and sizes in the
// kernel's arguments (no copy, and a graph captures it by value), 48,
// 320 or 1024 tensors of it.  Tensors are cut into chunks of 32768 elements (of small models
// fewer, down to 8192), dealt to a fixed number of CTAs in turn, so that what a CTA adds depends on the sizes alone, and
// that CTAs that run at the same time read neighbouring memory (1.0 G BF16
// gradients, norm and scaling: 897 us, 6.7 TB/s; an equal run of chunks for each
// CTA 914, chunks of 8192 1035).  Scaling goes through them backwards: what the
// norm read last is still in L2.
//
// Squares of BF16 and FP32 values leave FP32's range at 2^64 and 2^-63.  Each
// thread adds the squares of its part of a chunk in FP32, and goes through it
// again in FP64 if the sum is not between 2^-100 and infinity; everything from
// there on is FP64 (one addition for 64 elements, so its low rate does not show).
#include <math.h>

#include <algorithm>

#include "../csrc_vocab/vec.cuh"
#include "block_internal.h"

namespace ls {
namespace {

constexpr int kThreads = 256;
// CTAs of the norm and of scaling, each of which takes its chunks in turn.  An SM holds three of scaling (72 registers a
// thread), so these are two even rounds, and four of the norm (55), so there they are one and a half.  With the 608 that
// run at once the norm alone is faster (1008 M BF16: 291 us for 300, 137 M FP16 44.5 for 46.5) and scaling slower (norm
// and scaling 1003 for 904, 146 for 136); below 20 M elements nothing changes.
constexpr int kNormCtas = 912;
constexpr int kMostChunk = 15, kLeastChunk = 13;  // log2 of a chunk's elements
constexpr int kSlots = 8;           // vectors in flight for each thread, of the norm
constexpr int kScaleSlots = 4;      // and of scaling (8 of them spill)
constexpr int kFew = 48, kSome = 320, kMany = 1024;  // tensors of a launch, whose table is copied with it: 29 bytes each

struct Entry {
    void* p;         // the gradient, or the output
    const void* in;  // scaling: the input
    int64_t n;
};
template <int N> struct Table {
    Entry e[N];
    uint32_t first[N];  // number of its first chunk
    uint8_t dtype[N];
    int count, shift;   // shift: log2 of a chunk's elements
    uint32_t chunks;
};

// The chunks of this CTA, the last of them first if `backwards`.  f(entry index, first element, elements).
template <int N, typename F>
__device__ __forceinline__ void for_chunks(const Table<N>& t, bool backwards, F&& f) {
    const uint32_t n = t.chunks > blockIdx.x ? (t.chunks - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
    for (uint32_t i = 0; i < n; ++i) {
        const uint32_t c = blockIdx.x + (backwards ? n - 1 - i : i) * gridDim.x;
        int lo = 0, hi = t.count - 1;  // the last tensor whose first chunk is not behind c
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (t.first[mid] <= c)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int64_t e0 = static_cast<int64_t>(c - t.first[lo]) << t.shift;
        f(lo, e0, static_cast<int>(min(int64_t{1} << t.shift, t.e[lo].n - e0)));
    }
}

template <typename T> struct Wide;  // 16 bytes
template <> struct Wide<__half> { static constexpr int n = 8; };
template <> struct Wide<bf16> { static constexpr int n = 8; };
template <> struct Wide<float> { static constexpr int n = 4; };

template <typename T> __device__ __forceinline__ void widen(uint4 v, float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 t = u2f4(v);
        f[0] = t.x; f[1] = t.y; f[2] = t.z; f[3] = t.w;
    } else {
        unpack(Raw8<T>{v}, f);
    }
}

template <typename T> __device__ __forceinline__ float squares(uint4 v, float sum) {
    float f[8];
    widen<T>(v, f);
#pragma unroll
    for (int j = 0; j < Wide<T>::n; ++j) sum = fmaf(f[j], f[j], sum);
    return sum;
}

// The FP32 sum of a few squares, or, where FP32 cannot hold it, `again()`.
template <typename T, typename F> __device__ __forceinline__ double checked(float sum, F&& again) {
    if (sizeof(T) == 2 && !std::is_same<T, bf16>::value) return sum;  // FP16: 2^-48 to 2^32 each
    if (sum > 0x1p-100f && sum < INFINITY) return sum;
    return again();
}

// The squares of n elements from p on, this thread's part of them.
template <typename T> __device__ __forceinline__ double chunk_squares(const T* p, int n) {
    constexpr int W = Wide<T>::n;
    double total = 0.0;
    // up to the first 16-byte border, and behind the last
    const int head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) / sizeof(T)) % W);
    const int vecs = (n - head) / W, tail = n - head - vecs * W;
    const int i = static_cast<int>(threadIdx.x);
    if (i < head + tail) {
        const double x = to_f32(p[i < head ? i : n - tail + (i - head)]);
        total = x * x;
    }
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
    for (int v0 = i; v0 < vecs; v0 += kThreads * kSlots) {
        uint4 r[kSlots];
#pragma unroll
        for (int u = 0; u < kSlots; ++u)
            r[u] = v0 + u * kThreads < vecs ? v[v0 + u * kThreads] : make_uint4(0, 0, 0, 0);
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < kSlots; ++u) sum[u & 1] = squares<T>(r[u], sum[u & 1]);
        total += checked<T>(sum[0] + sum[1], [&] {
            uint32_t any = 0;
#pragma unroll
            for (int u = 0; u < kSlots; ++u) any |= r[u].x | r[u].y | r[u].z | r[u].w;
            double d = 0.0;
            if (any == 0) return d;  // zeros, as rows of an embedding's gradient are
#pragma unroll 1
            for (int u = 0; u < kSlots; ++u) {
                uint4 q = r[0];
#pragma unroll
                for (int k = 1; k < kSlots; ++k) q = u == k ? r[k] : q;
                float f[8];
                widen<T>(q, f);
#pragma unroll
                for (int j = 0; j < W; ++j) d += static_cast<double>(f[j]) * f[j];
            }
            return d;
        });
    }
    return total;
}

// The sum over the CTA's threads, in thread 0.  By its first warp: an FP64 addition of a warp takes about 16 cycles of
// an SM, so that exchanges in all warps would be most of a small tensor's time.
__device__ __forceinline__ double cta_sum(double v, double (&sm)[kThreads]) {
    sm[threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    v = sm[threadIdx.x];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) v += sm[threadIdx.x + 32 * w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// partial[cta] (+)= the squares of the CTA's chunks.
template <int N>
__global__ void __launch_bounds__(kThreads, 4)
square_sum_kernel(const __grid_constant__ Table<N> t, double* __restrict__ partial, bool add) {
    __shared__ double sm[kThreads];
    pdl_enter();
    double total = 0.0;
    for_chunks(t, false, [&](int k, int64_t e0, int n) {
        if (t.dtype[k] == LS_F32)
            total += chunk_squares(static_cast<const float*>(t.e[k].p) + e0, n);
        else if (t.dtype[k] == LS_F16)
            total += chunk_squares(static_cast<const __half*>(t.e[k].p) + e0, n);
        else
            total += chunk_squares(static_cast<const bf16*>(t.e[k].p) + e0, n);
    });
    total = cta_sum(total, sm);
    if (threadIdx.x == 0) partial[blockIdx.x] = add ? partial[blockIdx.x] + total : total;
}

// norm and factor from the CTAs' sums.
__global__ void __launch_bounds__(kThreads)
norm_factor_kernel(float* __restrict__ norm, float* __restrict__ factor, const double* __restrict__ partial, int n,
                   float max_norm, float grad_scale) {
    __shared__ double sm[kThreads];
    pdl_enter();
    double total = 0.0;
    for (int i = threadIdx.x; i < n; i += kThreads) total += partial[i];
    total = cta_sum(total, sm);
    if (threadIdx.x != 0) return;
    const float v = static_cast<float>(sqrt(total) * fabs(static_cast<double>(grad_scale)));
    const float f = max_norm / (v + 1e-6f);
    if (norm) norm[0] = v;
    if (factor) factor[0] = grad_scale * (max_norm == INFINITY && v == v ? 1.f : f > 1.f ? 1.f : f);  // a NaN stays one
}

template <typename T> __device__ __forceinline__ uint4 scaled(uint4 v, float f) {
    float x[8];
    widen<T>(v, x);
#pragma unroll
    for (int j = 0; j < Wide<T>::n; ++j) x[j] *= f;
    if constexpr (sizeof(T) == 4)
        return f2u4(make_float4(x[0], x[1], x[2], x[3]));
    else
        return pack<T>(x).v;
}

template <typename T> __device__ __forceinline__ void scale_chunk(T* out, const T* in, int n, float f) {
    constexpr int W = Wide<T>::n;
    const int i = static_cast<int>(threadIdx.x);
    if ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(in)) & 15) {  // no common border
        for (int e = i; e < n; e += kThreads) out[e] = from_f32<T>(to_f32(in[e]) * f);
        return;
    }
    const int head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(in) & 15)) / sizeof(T)) % W);
    const int vecs = (n - head) / W, tail = n - head - vecs * W;
    if (i < head + tail) {
        const int e = i < head ? i : n - tail + (i - head);
        out[e] = from_f32<T>(to_f32(in[e]) * f);
    }
    const uint4* v = reinterpret_cast<const uint4*>(in + head);
    uint4* w = reinterpret_cast<uint4*>(out + head);
    for (int v0 = i; v0 < vecs; v0 += kThreads * kScaleSlots) {
        uint4 r[kScaleSlots];
#pragma unroll
        for (int u = 0; u < kScaleSlots; ++u)
            if (v0 + u * kThreads < vecs) r[u] = v[v0 + u * kThreads];
#pragma unroll
        for (int u = 0; u < kScaleSlots; ++u)
            if (v0 + u * kThreads < vecs) w[v0 + u * kThreads] = scaled<T>(r[u], f);
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 3)
scale_kernel(const __grid_constant__ Table<N> t, const float* __restrict__ factor) {
    pdl_enter();
    const float f = *factor;
    for_chunks(t, true, [&](int k, int64_t e0, int n) {
        if (f == 1.f && t.e[k].p == t.e[k].in) return;
        if (t.dtype[k] == LS_F32)
            scale_chunk(static_cast<float*>(t.e[k].p) + e0, static_cast<const float*>(t.e[k].in) + e0, n, f);
        else if (t.dtype[k] == LS_F16)
            scale_chunk(static_cast<__half*>(t.e[k].p) + e0, static_cast<const __half*>(t.e[k].in) + e0, n, f);
        else
            scale_chunk(static_cast<bf16*>(t.e[k].p) + e0, static_cast<const bf16*>(t.e[k].in) + e0, n, f);
    });
}

// The update of one element; constants folded on the host as for ls_adam_update.
struct AdamArgs {
    uint64_t nv, n;  // whole vectors of 8, elements
    float b1, b2, omb1, omb2;
    float step_size, inv_sqrt_bc2, eps, decay;
    const float* factor;
    const float* norm;  // nullable: where it is not finite, nothing is written
};
__device__ __forceinline__ void adam1(float& p, float g, float& m, float& v, const AdamArgs& a) {
    m = a.b1 * m + a.omb1 * g;
    v = a.b2 * v + a.omb2 * (g * g);
    p = p * a.decay - a.step_size * m / (sqrtf(v) * a.inv_sqrt_bc2 + a.eps);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
adam_scaled_kernel(T* __restrict__ param, const T* __restrict__ grad, float* __restrict__ m, float* __restrict__ v,
                   const __grid_constant__ AdamArgs a) {
    pdl_enter();
    const float factor = *a.factor;
    if (a.norm && !(fabsf(*a.norm) < INFINITY)) return;
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kThreads;
    for (uint64_t i = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x; i < a.nv; i += step) {
        const uint64_t e = i * kVec;
        const Raw8<T> pr = load8<T>(param + e), gr = load8<T>(grad + e);
        const Raw8<float> mr = load8<float>(m + e), vr = load8<float>(v + e);
        float pf[kVec], gf[kVec], mf[kVec], vf[kVec];
        unpack(pr, pf);
        unpack(gr, gf);
        unpack(mr, mf);
        unpack(vr, vf);
#pragma unroll
        for (int j = 0; j < kVec; ++j) adam1(pf[j], gf[j] * factor, mf[j], vf[j], a);
        store8f<T>(param + e, pf);
        store8f<float>(m + e, mf);
        store8f<float>(v + e, vf);
    }
    const uint64_t j = a.nv * kVec + threadIdx.x;  // the last n % 8
    if (blockIdx.x == 0 && j < a.n) {
        float pf = to_f32(param[j]), mf = m[j], vf = v[j];
        adam1(pf, to_f32(grad[j]) * factor, mf, vf, a);
        param[j] = from_f32<T>(pf);
        m[j] = mf;
        v[j] = vf;
    }
}

// --- host ----------------------------------------------------------------------
// log2 of a chunk's elements: fewer of them where the tensors are too small for two chunks for each SM (norm and scaling
// of 0.5 M BF16 elements 8.2 -> 6.6 us, of 2.5 M FP32 10.0 -> 9.4; smaller chunks, or more of them, cost more CTAs their
// look at the table: 5.2 M FP16 in 107 tensors 10.2 us, with 632 chunks of 8192 13.4).
int chunk_shift(const ls_tensor* t, int64_t count) {
    int64_t n = 0;
    for (int64_t k = 0; k < count; ++k) n += t[k].n;
    int shift = kMostChunk;
    while (shift > kLeastChunk && n >> shift < 2 * 152) --shift;
    return shift;
}

// One launch after the other over tables of at most N tensors and 2^31 chunks: launch(table, number of launches before).
template <int N, typename F> cudaError_t by_tables(const ls_tensor* out, const ls_tensor* in, int64_t count, F&& launch) {
    Table<N> t;
    t.shift = chunk_shift(out, count);
    int64_t k = 0;
    for (int done = 0; k < count; ++done) {
        t.count = 0;
        int64_t chunks = 0;
        for (; k < count && t.count < N; ++k) {
            if (out[k].n == 0) continue;
            const int64_t c = (out[k].n + (int64_t{1} << t.shift) - 1) >> t.shift;
            if (chunks + c > INT32_MAX && t.count > 0) break;
            t.e[t.count] = Entry{out[k].data, in ? in[k].data : nullptr, out[k].n};
            t.dtype[t.count] = static_cast<uint8_t>(out[k].dtype);
            t.first[t.count] = static_cast<uint32_t>(chunks);
            ++t.count;
            chunks += c;
        }
        if (t.count == 0) break;
        t.chunks = static_cast<uint32_t>(chunks);
        const cudaError_t e = launch(t, done);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int N>
cudaError_t grad_norm(float* norm, float* factor, const ls_tensor* grads, int64_t count, float max_norm, float grad_scale,
                      double* partial, cudaStream_t s) {
    int ctas = 0;  // those that have written their sum; the first launch of several has them all
    const cudaError_t e = by_tables<N>(grads, nullptr, count, [&](const Table<N>& t, int done) {
        const int n = done || count > N ? kNormCtas : static_cast<int>(std::min<uint32_t>(t.chunks, kNormCtas));
        ctas = n;
        return launch_pdl(square_sum_kernel<N>, dim3(n), dim3(kThreads), 0, s, t, partial, done > 0);
    });
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_factor_kernel, dim3(1), dim3(kThreads), 0, s, norm, factor, static_cast<const double*>(partial),
                      ctas, max_norm, grad_scale);
}

template <int N>
cudaError_t scale_gradients(const ls_tensor* out, const ls_tensor* in, int64_t count, const float* factor,
                            cudaStream_t s) {
    return by_tables<N>(out, in, count, [&](const Table<N>& t, int) {
        return launch_pdl(scale_kernel<N>, dim3(std::min<uint32_t>(t.chunks, kNormCtas)), dim3(kThreads), 0, s, t, factor);
    });
}

template <typename T>
cudaError_t adam(void* param, const void* grad, float* m, float* v, const AdamArgs& a, cudaStream_t s) {
    // One vector for each thread: the seven streams stay closer together in memory than with a grid that strides
    // (137 M FP16 parameters with the norm: 475 us, with 1216 CTAs 555).
    const int64_t want = static_cast<int64_t>((a.nv + kThreads - 1) / kThreads);
    const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(want, 1 << 30));
    return launch_pdl(adam_scaled_kernel<T>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, static_cast<T*>(param),
                      static_cast<const T*>(grad), m, v, a);
}

}  // namespace

size_t grad_norm_workspace_bytes() { return kNormCtas * sizeof(double); }

cudaError_t launch_grad_norm(float* norm, float* factor, const ls_tensor* grads, int64_t count,
                             float max_norm, float grad_scale, void* workspace, cudaStream_t s) {
    double* partial = static_cast<double*>(workspace);
    if (count <= kFew) return grad_norm<kFew>(norm, factor, grads, count, max_norm, grad_scale, partial, s);
    if (count <= kSome) return grad_norm<kSome>(norm, factor, grads, count, max_norm, grad_scale, partial, s);
    return grad_norm<kMany>(norm, factor, grads, count, max_norm, grad_scale, partial, s);
}

cudaError_t launch_scale_gradients(const ls_tensor* out, const ls_tensor* in, int64_t count,
                                   const float* factor, cudaStream_t s) {
    return count <= kFew    ? scale_gradients<kFew>(out, in, count, factor, s)
           : count <= kSome ? scale_gradients<kSome>(out, in, count, factor, s)
                            : scale_gradients<kMany>(out, in, count, factor, s);
}

cudaError_t launch_adam_scaled(ls_dtype dt, void* param, const void* grad, float* m, float* v,
                               int64_t n, const AdamScaled& h, cudaStream_t s) {
    AdamArgs a;
    a.n = static_cast<uint64_t>(n);
    a.nv = a.n / kVec;
    a.b1 = h.beta1;
    a.b2 = h.beta2;
    a.omb1 = 1.0f - h.beta1;
    a.omb2 = 1.0f - h.beta2;
    const double bc1 = 1.0 - pow(static_cast<double>(h.beta1), static_cast<double>(h.step));
    const double bc2 = 1.0 - pow(static_cast<double>(h.beta2), static_cast<double>(h.step));
    a.step_size = static_cast<float>(static_cast<double>(h.lr) / bc1);
    a.inv_sqrt_bc2 = static_cast<float>(1.0 / sqrt(bc2));
    a.eps = h.eps;
    a.decay = static_cast<float>(1.0 - static_cast<double>(h.lr) * h.weight_decay);
    a.factor = h.factor;
    a.norm = h.norm;
    if (dt == LS_F16) return adam<__half>(param, grad, m, v, a, s);
    if (dt == LS_BF16) return adam<bf16>(param, grad, m, v, a, s);
    return adam<float>(param, grad, m, v, a, s);
}

}  // namespace ls
