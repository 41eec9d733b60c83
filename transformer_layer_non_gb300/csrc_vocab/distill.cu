// distill.cu -- distillation from a teacher's top logits, forward and backward.
//
// Per row, with the student's logits z, the teacher's k entries (index, t) and
// the temperature tau (the loss of Hinton, Vinyals and Dean, "Distilling the
// knowledge in a neural network", 2015, over the stored entries):
//   log q_e = t_e / tau - base,   base = log sum_valid exp(t / tau) or the given teacher_lse
//   log p_j = z_j / tau - lse,    lse  = log sum_j exp(z_j / tau)
//   loss    = tau^2 sum_e q_e (log q_e - log p_index(e))
//   dz_j    = dloss tau (p_j Q - sum_{e: index(e) = j} q_e),   Q = sum_e q_e
//
// The forward reads each row once (online maximum and sum per thread, merged
// across the CTA and its cluster); the backward reads it once and writes it
// once, from the forward's lse.  Both are bound by memory for rows of many
// CTAs.  The k entries are a few hundred bytes: every CTA of a row computes
// their q for itself.
#include <math.h>

#include "vec.cuh"
#include "vocab_internal.h"

namespace ls {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;  // vectors per thread in flight
constexpr int kMaxK = 1024;
constexpr float kLog2e = 1.4426950408889634f;

struct DistillArgs {
    int64_t vocab;
    int k;
    int nvec;       // vocab / 8
    int slice;      // vectors per CTA of a row
    float tau;
    float c;        // log2(e) / tau
};

__device__ __forceinline__ void merge(float& m, float& l, float m2, float l2, float c) {
    const float mm = fmaxf(m, m2);
    if (mm == -INFINITY) {  // nothing but -inf (or NaN sums) so far
        l += l2;
        return;
    }
    l = l * exp2_approx((m - mm) * c) + l2 * exp2_approx((m2 - mm) * c);
    m = mm;
}

// Sum or maximum over the CTA, the same value in every thread; `sm` holds kWarps floats.
__device__ __forceinline__ float cta_sum(float v, float* sm) {
    v = group_sum<32>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sm[w];
    return s;
}
__device__ __forceinline__ float cta_max(float v, float* sm) {
    v = group_max<32>(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = sm[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s = fmaxf(s, sm[w]);
    return s;
}

// The row's entries: sm_logq[e] = log q_e (-inf where q is 0) and sm_ix[e]
// (-1 where the entry is not valid).
template <typename T>
__device__ __forceinline__ void load_entries(float* sm_logq, int* sm_ix, float* sm_red,
                                             const int32_t* index, const T* teacher,
                                             const float* teacher_lse, int64_t row,
                                             const DistillArgs& a) {
    float tmax = -INFINITY;
    for (int e = threadIdx.x; e < a.k; e += kThreads) {
        const int32_t j = index[row * a.k + e];
        const bool there = j >= 0 && j < a.vocab;
        const float t = there ? to_f32(teacher[row * a.k + e]) / a.tau : -INFINITY;
        sm_ix[e] = there ? j : -1;
        sm_logq[e] = t;
        tmax = t != t ? INFINITY : fmaxf(tmax, t);  // a NaN reaches q either way
    }
    float base;
    if (teacher_lse) {
        base = teacher_lse[row];
    } else {
        tmax = cta_max(tmax, sm_red);
        float s = 0.f;
        if (tmax > -INFINITY)
            for (int e = threadIdx.x; e < a.k; e += kThreads) s += expf(sm_logq[e] - tmax);
        s = cta_sum(s, sm_red);
        base = tmax > -INFINITY ? tmax + logf(s) : 0.f;
    }
    for (int e = threadIdx.x; e < a.k; e += kThreads)
        if (sm_ix[e] >= 0 && sm_logq[e] != -INFINITY) sm_logq[e] -= base;
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
distill_fwd_kernel(float* __restrict__ loss, float* __restrict__ lse_out,
                   const T* __restrict__ logits, const int32_t* __restrict__ index,
                   const T* __restrict__ teacher, const float* __restrict__ teacher_lse,
                   const __grid_constant__ DistillArgs a) {
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_red[kWarps];
    __shared__ float sm_logq[kMaxK];
    __shared__ int sm_ix[kMaxK];
    pdl_enter();
    const int64_t row = blockIdx.x;
    const T* z = logits + row * a.vocab;
    float m = -INFINITY, l = 0.f;
    for (int v0 = threadIdx.x; v0 < a.nvec; v0 += kThreads * kUnroll) {
        Raw8<T> r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int v = v0 + u * kThreads;
            if (v < a.nvec) r[u] = load8<T>(z + static_cast<int64_t>(v) * kVec);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (v0 + u * kThreads >= a.nvec) break;
            float f[kVec];
            unpack(r[u], f);
            const float vm = vmax8(r[u]);
            if (vm > m) {
                l *= exp2_approx((m - vm) * a.c);
                m = vm;
            }
            const float mc = m * a.c;
            if (fabsf(mc) < INFINITY) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) l += exp2_approx(fmaf(f[j], a.c, -mc));
            } else if (m != -INFINITY) {  // m is finite and m c is not (FP32's lowest values as a mask)
#pragma unroll
                for (int j = 0; j < kVec; ++j) l += exp2_approx((f[j] - m) * a.c);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const float l2 = __shfl_xor_sync(0xffffffffu, l, o);
        merge(m, l, m2, l2, a.c);
    }
    if ((threadIdx.x & 31) == 0) {
        sm_m[threadIdx.x >> 5] = m;
        sm_l[threadIdx.x >> 5] = l;
    }
    load_entries(sm_logq, sm_ix, sm_red, index, teacher, teacher_lse, row, a);
    m = sm_m[0];
    l = sm_l[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) merge(m, l, sm_m[w], sm_l[w], a.c);
    const float lse = m / a.tau + logf(l);
    float s = 0.f;
    for (int e = threadIdx.x; e < a.k; e += kThreads) {
        const float lq = sm_logq[e];
        const float q = expf(lq);
        if (sm_ix[e] < 0 || q == 0.f) continue;
        s += q * (lq - (to_f32(z[sm_ix[e]]) / a.tau - lse));
    }
    s = cta_sum(s, sm_red);
    if (threadIdx.x == 0) {
        loss[row] = a.tau * a.tau * s;
        if (lse_out) lse_out[row] = lse;
    }
}

// CTA (row, slice): the slice's vectors of the row, then the entries that fall into it.
template <typename T>
__global__ void __launch_bounds__(kThreads)
distill_bwd_kernel(T* dlogits, const T* logits, const int32_t* __restrict__ index,
                   const T* __restrict__ teacher, const float* __restrict__ lse,
                   const float* __restrict__ teacher_lse, const float* __restrict__ dloss,
                   const __grid_constant__ DistillArgs a) {
    __shared__ float sm_red[kWarps];
    __shared__ float sm_q[kMaxK], sm_z[kMaxK];
    __shared__ int sm_ix[kMaxK];
    pdl_enter();
    const int64_t row = blockIdx.x;
    const T* z = logits + row * a.vocab;
    T* dz = dlogits + row * a.vocab;
    load_entries(sm_q, sm_ix, sm_red, index, teacher, teacher_lse, row, a);
    float Q = 0.f;
    for (int e = threadIdx.x; e < a.k; e += kThreads) {
        const float q = sm_ix[e] >= 0 ? expf(sm_q[e]) : 0.f;
        sm_q[e] = q;
        sm_z[e] = q != 0.f ? to_f32(z[sm_ix[e]]) : 0.f;  // before the slice is overwritten (in place)
        Q += q;
    }
    Q = cta_sum(Q, sm_red);  // its barriers also put every gather before the first store
    const float g = a.tau * (dloss ? dloss[row] : 1.f);
    const float gq = g * Q;
    const float row_lse = lse[row];
    const bool some = Q != 0.f;
    // exp(z / tau - lse) by one FMA, unless the FMA's terms overflow (FP32's
    // lowest values in a whole row).
    const float ll = row_lse * kLog2e;
    const bool tame = fabsf(ll) < INFINITY;
    auto prob = [&](float f) {
        return exp2_approx(tame ? fmaf(f, a.c, -ll) : (f / a.tau - row_lse) * kLog2e);
    };
    const int lo = blockIdx.y * a.slice;
    const int hi = min(a.nvec, lo + a.slice);
    for (int v0 = lo + threadIdx.x; v0 < hi; v0 += kThreads * kUnroll) {
        Raw8<T> r[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int v = v0 + u * kThreads;
            if (v < hi && some) r[u] = load8<T>(z + static_cast<int64_t>(v) * kVec);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int v = v0 + u * kThreads;
            if (v >= hi) break;
            float o[kVec];
            if (some) {
                float f[kVec];
                unpack(r[u], f);
#pragma unroll
                for (int j = 0; j < kVec; ++j) o[j] = gq * prob(f[j]);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j) o[j] = 0.f;
            }
            store8f<T>(dz + static_cast<int64_t>(v) * kVec, o);
        }
    }
    if (!some) return;
    __syncthreads();
    // The entries' columns again, from the FP32 values.  The first of several
    // entries with one index writes it, with their q added in entry order.
    for (int e = threadIdx.x; e < a.k; e += kThreads) {
        const int j = sm_ix[e];
        if (j < 0 || j / kVec < lo || j / kVec >= hi || sm_q[e] == 0.f) continue;
        float q = 0.f;
        bool first = true;
        for (int f = 0; f < a.k; ++f) {
            if (sm_ix[f] != j || sm_q[f] == 0.f) continue;
            if (f < e) {
                first = false;
                break;
            }
            q += sm_q[f];
        }
        if (first) dz[j] = from_f32<T>(g * (Q * prob(sm_z[e]) - q));
    }
}

DistillArgs make_args(const DistillShape& sh) {
    DistillArgs a;
    a.vocab = sh.vocab;
    a.k = sh.k;
    a.nvec = static_cast<int>(sh.vocab / kVec);
    a.slice = a.nvec;
    a.tau = sh.tau;
    a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(sh.tau));
    return a;
}

template <typename T>
cudaError_t fwd(float* loss, float* lse, const void* logits, const int32_t* index,
                const void* teacher, const float* teacher_lse, const DistillShape& sh,
                cudaStream_t s) {
    return launch_pdl(distill_fwd_kernel<T>, dim3(static_cast<unsigned>(sh.rows)), dim3(kThreads),
                      0, s, loss, lse, static_cast<const T*>(logits), index,
                      static_cast<const T*>(teacher), teacher_lse, make_args(sh));
}

template <typename T>
cudaError_t bwd(void* dlogits, const void* logits, const int32_t* index, const void* teacher,
                const float* lse, const float* teacher_lse, const float* dloss,
                const DistillShape& sh, cudaStream_t s) {
    return launch_pdl(distill_bwd_kernel<T>, dim3(static_cast<unsigned>(sh.rows)), dim3(kThreads),
                      0, s, static_cast<T*>(dlogits), static_cast<const T*>(logits), index,
                      static_cast<const T*>(teacher), lse, teacher_lse, dloss, make_args(sh));
}

}  // namespace

cudaError_t launch_distill_fwd(ls_dtype dt, float* loss, float* lse, const void* logits,
                               const int32_t* index, const void* teacher, const float* teacher_lse,
                               const DistillShape& sh, cudaStream_t s) {
    if (dt == LS_F16) return fwd<__half>(loss, lse, logits, index, teacher, teacher_lse, sh, s);
    if (dt == LS_BF16) return fwd<bf16>(loss, lse, logits, index, teacher, teacher_lse, sh, s);
    return fwd<float>(loss, lse, logits, index, teacher, teacher_lse, sh, s);
}

cudaError_t launch_distill_bwd(ls_dtype dt, void* dlogits, const void* logits,
                               const int32_t* index, const void* teacher, const float* lse,
                               const float* teacher_lse, const float* dloss,
                               const DistillShape& sh, cudaStream_t s) {
    if (dt == LS_F16)
        return bwd<__half>(dlogits, logits, index, teacher, lse, teacher_lse, dloss, sh, s);
    if (dt == LS_BF16)
        return bwd<bf16>(dlogits, logits, index, teacher, lse, teacher_lse, dloss, sh, s);
    return bwd<float>(dlogits, logits, index, teacher, lse, teacher_lse, dloss, sh, s);
}

}  // namespace ls
