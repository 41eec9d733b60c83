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
// across the CTA and its cluster), the backward reads it once and writes it
// once, from the forward's lse: bound by memory when the rows fill the GPU.
// Few rows are cut over more CTAs: a cluster of up to 8 per row in the
// forward, any number of slices in the backward, which needs no merging.
//
// The k entries are a few hundred bytes.  Warp 0 works them out by shuffles
// while the row's first vectors are on their way to all warps:
// each lane, of its entries,
//   r = max_e z_index(e) / tau,   E = sum_e q_e (log q_e + r - z_index(e) / tau),   Q = sum_e q_e,
// and   loss = tau^2 sum_lanes (E + Q (lse - r))   then needs one barrier, the
// merging of the warps' sums.  (Without r the loss would be a difference of two
// numbers of lse's size: 1e23 instead of 2 in a row of logits near -1e30.)
#include <float.h>
#include <math.h>

#include <algorithm>

#include "vec.cuh"
#include "vocab_internal.h"

namespace ls {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// exp((z - m) / tau) = 2^(z c - m c), c = log2(e) / tau, by one FMA as long as the rounding of m c, at most
// 2^-24 of it, is harmless: below 2^17 (FP16's lowest value at tau = 1) it is at most 2^-8, less than the
// rounding of the row's FP32 lse.  At 1e10 it is hundreds, and the exponential of the maximum itself, which is
// 1, would be infinite or 0.
constexpr float kMostFma = 131072.f;
// Vectors per thread in flight.
template <typename T> constexpr int unroll_fwd() { return sizeof(T) == 2 ? 6 : 3; }
template <typename T> constexpr int unroll_bwd() { return sizeof(T) == 2 ? 8 : 4; }

struct DistillArgs {
    int64_t vocab;
    int k;
    int nvec;       // vocab / 8
    int slice;      // vectors per CTA of a row
    int table;      // backward: slots of the hash table, a power of two >= 2 k, or 0:
    int words;      //   a bit for each column of the slice, in so many words
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

constexpr int kBatch = 4;  // entries per lane whose loads are in flight together

// The student's logits at a lane's entries e0, e0 + 32, ..., 0 where the index is not in [lo, hi) (or -1).
template <typename T>
__device__ __forceinline__ void gather(float (&f)[kBatch], const T* z, const int* ix, int e0, int k, int lo, int hi) {
    T w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
        const int j = ix[min(e0 + 32 * u, k - 1)];
        w[u] = j >= lo && j < hi ? z[j] : from_f32<T>(0.f);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) f[u] = to_f32(w[u]);
}

// log q of the row's entries: e = lane, lane + 32, ... of warp 0.  ix[e] gets
// the index, -1 where the entry has q = 0; logq[e] the value.
template <typename T>
__device__ __forceinline__ void load_entries(float* logq, int* ix, const int32_t* index,
                                             const T* teacher, const float* teacher_lse,
                                             int64_t row, const DistillArgs& a) {
    const int lane = threadIdx.x & 31;
    index += row * a.k;
    teacher += row * a.k;
    float tmax = -INFINITY;
    for (int e0 = lane; e0 < a.k; e0 += 32 * kBatch) {
        int32_t j[kBatch];
        T w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int e = min(e0 + 32 * u, a.k - 1);
            j[u] = index[e];
            w[u] = teacher[e];
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int e = e0 + 32 * u;
            if (e >= a.k) break;
            const bool there = j[u] >= 0 && j[u] < a.vocab;
            const float t = there ? to_f32(w[u]) / a.tau : -INFINITY;
            logq[e] = t;
            ix[e] = t == -INFINITY ? -1 : j[u];
            tmax = t != t ? INFINITY : fmaxf(tmax, t);  // a NaN reaches q either way
        }
    }
    float base = 0.f;
    if (teacher_lse) {
        base = teacher_lse[row];
    } else {
        tmax = group_max<32>(tmax);
        if (tmax > -INFINITY) {
            float s = 0.f;
            for (int e = lane; e < a.k; e += 32) s += expf(logq[e] - tmax);
            base = tmax + logf(group_sum<32>(s));
        }
    }
    for (int e = lane; e < a.k; e += 32) {
        logq[e] -= base;
        if (expf(logq[e]) == 0.f) ix[e] = -1;
    }
}

// The vectors v, v + THREADS, ... of a row below hi, into registers; -inf behind it.
template <typename T, int U, int THREADS>
__device__ __forceinline__ void load_batch(Raw8<T> (&r)[U], const T* z, int v0, int hi) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = v0 + u * THREADS;
        r[u] = v < hi ? load8<T>(z + static_cast<int64_t>(v) * kVec) : lowest8<T>();
    }
}

// Dynamic shared memory: logq [k], ix [k].
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
distill_fwd_kernel(float* __restrict__ loss, float* __restrict__ lse_out,
                   const T* __restrict__ logits, const int32_t* __restrict__ index,
                   const T* __restrict__ teacher, const float* __restrict__ teacher_lse,
                   const __grid_constant__ DistillArgs a, int cluster) {
    constexpr int U = unroll_fwd<T>(), kWarps = THREADS / 32;
    extern __shared__ float sm_k[];
    __shared__ float sm_m[kWarps], sm_l[kWarps];
    __shared__ float sm_part[2];
    pdl_enter();
    const int64_t row = blockIdx.x / cluster;
    const int rank = static_cast<int>(blockIdx.x - row * cluster);
    const T* z = logits + row * a.vocab;
    const int lo = rank * a.slice, hi = min(a.nvec, lo + a.slice);
    Raw8<T> r[U];
    int v0 = lo + threadIdx.x;
    load_batch<T, U, THREADS>(r, z, v0, hi);
    float E = 0.f, Q = 0.f, ref = -FLT_MAX;
    if (rank == 0 && threadIdx.x < 32) {
        float* logq = sm_k;
        int* ix = reinterpret_cast<int*>(sm_k + a.k);
        load_entries(logq, ix, index, teacher, teacher_lse, row, a);
        __syncwarp();
        for (int e0 = threadIdx.x; e0 < a.k; e0 += 32 * kBatch) {
            float f[kBatch];
            gather(f, z, ix, e0, a.k, 0, static_cast<int>(a.vocab));
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int e = e0 + 32 * u;
                if (e >= a.k || ix[e] < 0) continue;
                const float q = expf(logq[e]), zu = f[u] / a.tau;
                if (zu > ref) {
                    if (Q != 0.f) E += Q * (zu - ref);
                    ref = zu;
                }
                E += q * (logq[e] + (ref - zu));
                Q += q;
            }
        }
    }
    float m = -INFINITY;
    float2 l2 = make_float2(0.f, 0.f);
    const float2 cc = make_float2(a.c, a.c);
    for (; v0 < hi; v0 += U * THREADS) {
        Raw8<T> top = r[0];
#pragma unroll
        for (int u = 1; u < U; ++u) top = vmax(top, r[u]);
        const float bm = vmax8(top);
        if (bm > m) {  // rescale the running sum to the new maximum
            const float c = exp2_approx((m - bm) * a.c);
            l2 = mul2(l2, make_float2(c, c));
            m = bm;
        }
        const float mc = m * a.c;
        const bool tame = fabsf(mc) < kMostFma;
        const float2 mm = make_float2(-mc, -mc);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[kVec];
            unpack(r[u], f);
            // The next vector into this one's place at once: U loads stay in flight.
            const int next = v0 + (U + u) * THREADS;
            r[u] = next < hi ? load8<T>(z + static_cast<int64_t>(next) * kVec) : lowest8<T>();
            if (tame) {
#pragma unroll
                for (int j = 0; j < kVec; j += 2) {
                    const float2 t = fma2(make_float2(f[j], f[j + 1]), cc, mm);
                    l2 = add2(l2, make_float2(exp2_approx(t.x), exp2_approx(t.y)));
                }
            } else {  // large finite values as a mask (m c may overflow), or m is infinite: -inf adds nothing, a NaN stays
                for (int j = 0; j < kVec; ++j)
                    if (f[j] != -INFINITY) l2.x += exp2_approx((f[j] - m) * a.c);
            }
        }
    }
    float l = l2.x + l2.y;
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
    __syncthreads();
    if (threadIdx.x >= 32 && cluster == 1) return;
    m = sm_m[0];
    l = sm_l[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) merge(m, l, sm_m[w], sm_l[w], a.c);
    if (cluster > 1) {
        if (threadIdx.x == 0) {
            sm_part[0] = m;
            sm_part[1] = l;
        }
        cluster_sync();
        if (rank == 0)
            for (int c = 1; c < cluster; ++c) {
                const uint32_t p = map_rank(sm_part, c);
                merge(m, l, ld_cluster(p), ld_cluster(p + 4), a.c);
            }
        cluster_sync();  // a CTA's shared memory lives until the first one has read it
        if (rank != 0 || threadIdx.x >= 32) return;
    }
    const float lse = m / a.tau + logf(l);
    if (Q != 0.f) E += Q * (lse - ref);
    E = group_sum<32>(E);
    Q = group_sum<32>(Q);
    if (threadIdx.x == 0) {
        loss[row] = Q == 0.f ? 0.f : a.tau * a.tau * E;
        if (lse_out) lse_out[row] = lse;
    }
}

// A CTA for each slice of each row, a row's side by side: the slice's vectors, then the entries that fall
// into it.  Rows run from the last to the first: the forward, which runs the
// other way, has left the last ones in L2.
// Indexes that a row holds twice are found by a hash table, or where the slice is short against k by a bit
// for each column (8192 x 4096 BF16, k = 256: 68 us with the table, 45 with the bits;
// 8192 x 1000: 38 and 23, and 38 where a row has about 30 indexes twice).
// Dynamic shared memory: q, z, ix, slot [k]; then hash table, twice [table]; or seen, twice [words].
template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS)
distill_bwd_kernel(T* dlogits, const T* logits, const int32_t* __restrict__ index,
                   const T* __restrict__ teacher, const float* __restrict__ lse,
                   const float* __restrict__ teacher_lse, const float* __restrict__ dloss,
                   const __grid_constant__ DistillArgs a, int parts) {
    constexpr int U = unroll_bwd<T>();
    extern __shared__ float sm_k[];
    __shared__ float sm_sum;
    __shared__ int sm_repeated;
    float* sm_q = sm_k;
    float* sm_z = sm_k + a.k;
    int* sm_ix = reinterpret_cast<int*>(sm_k + 2 * a.k);
    int* sm_slot = sm_ix + a.k;
    int* sm_table = sm_slot + a.k;
    int* sm_twice = sm_table + a.table;  // [table]: the slot's index came more than once
    uint32_t* sm_seen = reinterpret_cast<uint32_t*>(sm_table);
    uint32_t* sm_more = sm_seen + a.words;  // columns that came more than once
    pdl_enter();
    const int64_t unit = gridDim.x - 1 - blockIdx.x, row = unit / parts;
    const T* z = logits + row * a.vocab;
    T* dz = dlogits + row * a.vocab;
    const int lo = static_cast<int>(unit - row * parts) * a.slice, hi = min(a.nvec, lo + a.slice);
    Raw8<T> r[U];
    int v0 = lo + threadIdx.x;
    load_batch<T, U, THREADS>(r, z, v0, hi);
    const float row_lse = lse[row];
    const float g = a.tau * (dloss ? dloss[row] : 1.f);
    // Warp 0: the slice's entries' logits, and the hash table of their indexes.  Logits of other slices are
    // not read: in place, their CTAs may have written gradients over them.
    auto place_entries = [&]() {
        bool any_twice = false;
        for (int e0 = threadIdx.x; e0 < a.k; e0 += 32 * kBatch) {
            float f[kBatch];
            gather(f, z, sm_ix, e0, a.k, lo * kVec, hi * kVec);
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int e = e0 + 32 * u;
                if (e >= a.k) continue;
                const int j = sm_ix[e];
                sm_z[e] = f[u];
                if (j < 0 || j / kVec < lo || j / kVec >= hi) {
                    sm_ix[e] = -1;
                    continue;
                }
                if (a.table == 0) {
                    const int c = j - lo * kVec;
                    const uint32_t bit = 1u << (c & 31);
                    if (atomicOr(sm_seen + (c >> 5), bit) & bit) {
                        atomicOr(sm_more + (c >> 5), bit);
                        any_twice = true;
                    }
                    continue;
                }
                uint32_t h = ((static_cast<uint32_t>(j) * 2654435761u) >> 16) & (a.table - 1);
                for (;; h = (h + 1) & (a.table - 1)) {  // at most k of the table's 2 k slots are taken
                    const int was = atomicCAS(sm_table + h, -1, j);
                    if (was == -1) break;
                    if (was == j) {
                        sm_twice[h] = 1;
                        any_twice = true;
                        break;
                    }
                }
                sm_slot[e] = h;
            }
        }
        // The entries whose index came more than once: in order into a list, over the slots that are no
        // longer needed, and marked by -2 - index.
        int n = 0;
        __syncwarp();
        if (__any_sync(0xffffffffu, any_twice))
            for (int e0 = 0; e0 < a.k; e0 += 32) {
                const int e = e0 + threadIdx.x;
                const int j = e < a.k ? sm_ix[e] : -1;
                const int c = j - lo * kVec;
                const bool more =
                    j >= 0 && (a.table == 0 ? sm_more[c >> 5] >> (c & 31) & 1 : sm_twice[sm_slot[e]]);
                const unsigned all = __ballot_sync(0xffffffffu, more);
                if (more) {
                    sm_ix[e] = -2 - j;
                    sm_slot[n + __popc(all & ((1u << threadIdx.x) - 1u))] = e;
                }
                n += __popc(all);
                __syncwarp();
            }
        if (threadIdx.x == 0) sm_repeated = n;
    };
    const bool in_place = dlogits == logits;
    if (threadIdx.x < 32) {
        for (int t = threadIdx.x; t < a.table; t += 32) {
            sm_table[t] = -1;
            sm_twice[t] = 0;
        }
        for (int t = threadIdx.x; t < 2 * a.words; t += 32) sm_seen[t] = 0;
        __syncwarp();
        load_entries(sm_q, sm_ix, index, teacher, teacher_lse, row, a);
        float Q = 0.f;
        for (int e = threadIdx.x; e < a.k; e += 32) {
            const float q = sm_ix[e] >= 0 ? expf(sm_q[e]) : 0.f;
            sm_q[e] = q;
            Q += q;
        }
        Q = group_sum<32>(Q);
        if (threadIdx.x == 0) sm_sum = Q;
        __syncwarp();
        if (in_place) place_entries();  // before anything is stored over the entries' logits
    }
    __syncthreads();
    if (!in_place && threadIdx.x < 32) place_entries();  // while the other warps go ahead
    const float Q = sm_sum;
    const float gq = g * Q;
    const bool some = Q != 0.f;
    // exp(z / tau - lse) by one FMA, unless lse is too far from zero for that (large finite values in a
    // whole row); the difference is then at most 0, because the forward's lse is no less than z / tau.
    const float ll = row_lse * kLog2e;
    const bool tame = fabsf(ll) < kMostFma;
    auto prob = [&](float f) {
        return exp2_approx(tame ? fmaf(f, a.c, -ll) : (f / a.tau - row_lse) * kLog2e);
    };
    if (some && tame) {
        const float2 cc = make_float2(a.c, a.c), mm = make_float2(-ll, -ll), gg = make_float2(gq, gq);
        for (; v0 < hi; v0 += U * THREADS) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int v = v0 + u * THREADS;
                if (v >= hi) break;
                float f[kVec];
                unpack(r[u], f);
#pragma unroll
                for (int j = 0; j < kVec; j += 2) {
                    const float2 t = fma2(make_float2(f[j], f[j + 1]), cc, mm);
                    const float2 o = mul2(make_float2(exp2_approx(t.x), exp2_approx(t.y)), gg);
                    f[j] = o.x;
                    f[j + 1] = o.y;
                }
                store8f<T>(dz + static_cast<int64_t>(v) * kVec, f);
            }
            load_batch<T, U, THREADS>(r, z, v0 + U * THREADS, hi);
        }
    } else {
#pragma unroll 1
        for (; v0 < hi; v0 += THREADS) {
            float f[kVec];
            load8f<T>(z + static_cast<int64_t>(v0) * kVec, f);
            for (int j = 0; j < kVec; ++j) f[j] = some ? gq * prob(f[j]) : 0.f;
            store8f<T>(dz + static_cast<int64_t>(v0) * kVec, f);
        }
    }
    if (!some) return;
    __syncthreads();
    // The entries' columns again, from the FP32 values.
    for (int e = threadIdx.x; e < a.k; e += THREADS) {
        const int j = sm_ix[e];
        if (j >= 0) dz[j] = from_f32<T>(g * (Q * prob(sm_z[e]) - sm_q[e]));
    }
    // Where a row holds an index more than once, its first entry writes the sum of their q, in entry order.
    const int n = sm_repeated;
    for (int i = threadIdx.x; i < n; i += THREADS) {
        const int e = sm_slot[i], mark = sm_ix[e];
        float q = 0.f;
        bool first = true;
        for (int m0 = 0; m0 < n && first; m0 += kBatch) {
            int e2[kBatch], mark2[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) e2[u] = sm_slot[min(m0 + u, n - 1)];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) mark2[u] = sm_ix[e2[u]];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (m0 + u >= n || mark2[u] != mark) continue;
                first = first && m0 + u >= i;
                q += sm_q[e2[u]];
            }
        }
        if (first) dz[-2 - mark] = from_f32<T>(g * (Q * prob(sm_z[e]) - q));
    }
}

// A row is cut into `parts` slices.
DistillArgs make_args(const DistillShape& sh, int parts) {
    DistillArgs a;
    a.vocab = sh.vocab;
    a.k = sh.k;
    a.nvec = static_cast<int>(sh.vocab / kVec);
    a.slice = (a.nvec + parts - 1) / parts;
    a.table = 2;
    while (a.table < 2 * sh.k) a.table *= 2;
    a.words = (a.slice * kVec + 31) / 32;
    if (a.words <= std::min(2 * a.table, 3584))  // 44 KB in all at the most
        a.table = 0;
    else
        a.words = 0;
    a.tau = sh.tau;
    a.c = static_cast<float>(1.4426950408889634 / static_cast<double>(sh.tau));
    return a;
}

// One warp for slices below 8K values where there are many: they spend their time on the entries'
// latencies, and an SM then has 32 of them at once (8192 x 4096 FP16, k = 32: step 62 us with 128
// threads, 38 with 32; 8192 x 1000: 54 and 23; 100 x 50264 FP32 in slices, backward: 10.6 and 8.4).
// Few slices have the SMs to themselves (5 x 50264 FP32, forward: 4.9 us with 128 threads, 6.4 with 32).
constexpr int kShortSlice = 1024, kManySlices = 608;

// Threads of a CTA otherwise: 128, and 256 for slices of 64K values or more (measured at
// 4096 x 30528 FP16: forward 47 us with 128, 51 with 256; 2047 x 131072 BF16: 104 and 92).
int threads_of(const DistillArgs& a, int64_t slices) {
    if (a.slice < kShortSlice && slices >= kManySlices) return 32;
    return a.slice >= 8192 ? 256 : 128;
}

// Slices of a row, for about `ctas` CTAs in all; none below two vectors for a thread.
int parts_of(const DistillShape& sh, int ctas, int most) {
    const int64_t want = ctas / sh.rows;
    const int64_t can = sh.vocab / kVec / 256;
    int64_t n = 1;
    while (2 * n <= want && 2 * n <= can && 2 * n <= most) n *= 2;
    return static_cast<int>(n);
}

template <typename T>
cudaError_t fwd(float* loss, float* lse, const void* logits, const int32_t* index,
                const void* teacher, const float* teacher_lse, const DistillShape& sh,
                cudaStream_t s) {
    // A grid's x extent ends at 2^31 - 1 CTAs.
    const int cluster = sh.rows > (1 << 20) ? 1 : parts_of(sh, 608, 8);
    const DistillArgs a = make_args(sh, cluster);
    const int threads = threads_of(a, sh.rows * cluster);
    return launch_cluster(threads == 32    ? distill_fwd_kernel<T, 32>
                          : threads == 128 ? distill_fwd_kernel<T, 128>
                                           : distill_fwd_kernel<T, 256>,
                          dim3(static_cast<unsigned>(sh.rows * cluster)), cluster, dim3(threads),
                          static_cast<size_t>(sh.k) * 8, s, loss, lse, static_cast<const T*>(logits),
                          index, static_cast<const T*>(teacher), teacher_lse, a, cluster);
}

template <typename T>
cudaError_t bwd(void* dlogits, const void* logits, const int32_t* index, const void* teacher,
                const float* lse, const float* teacher_lse, const float* dloss,
                const DistillShape& sh, cudaStream_t s) {
    // Each slice reads and writes its own columns alone, in place too.  (777 x 32000 FP32: 49 us whole,
    // 40 in four slices; FP16 rows, half as long, gain nothing.)
    int parts = parts_of(sh, sizeof(T) == 4 ? 3648 : 1216, 64);
    // And none above 32 KB (64 with many entries, which each slice looks through): whole rows in flight on
    // all SMs spread over so much memory that some placements of the two buffers take 195 us instead of 78
    // (4096 x 30528 FP16; 76.5 in two slices wherever they lie; 2047 x 131072 BF16: 166 whole, 157 in eight).
    const int64_t most = (sh.k > 128 ? 65536 : 32768) / (kVec * static_cast<int64_t>(sizeof(T)));
    while (sh.vocab / kVec > parts * most) parts *= 2;
    const DistillArgs a = make_args(sh, parts);
    const int threads = threads_of(a, sh.rows * parts);
    const size_t smem = static_cast<size_t>(4 * sh.k + 2 * (a.table ? a.table : a.words)) * 4;
    return launch_pdl(threads == 32    ? distill_bwd_kernel<T, 32>
                      : threads == 128 ? distill_bwd_kernel<T, 128>
                                       : distill_bwd_kernel<T, 256>,
                      dim3(static_cast<unsigned>(sh.rows * parts)),
                      dim3(threads), smem, s,
                      static_cast<T*>(dlogits), static_cast<const T*>(logits), index,
                      static_cast<const T*>(teacher), lse, teacher_lse, dloss, a, parts);
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
