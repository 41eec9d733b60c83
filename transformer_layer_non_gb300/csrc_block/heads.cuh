// heads.cuh -- rotary positions of queries and keys, and the norm of each
// head's row with the rotation in the same pass; forward and backward in one
// kernel.
//
//   forward   y = R(w u),  u = x r,  r = 1 / sqrt(mean x^2 + eps)     (without the norm: y = R x)
//   backward  g = R^T dy, dw = sum g u, dx = r (w g - u mean(w g u))  (without the norm: dx = R^T dy)
//
// Every element is read once and written once, so memory bounds it: a few FP32
// operations an element.  What else could cost is the angles.  An angle is
// turns * position in 64-bit fixed point, a full circle being 2^64, so the
// reduction to one turn is the multiplication's overflow and exact at any
// position; sincospif gets at most an eighth of a turn.  A warp takes a few tokens
// with all their heads (or, of few tokens, some of them), works out its tokens'
// cosines and sines once, while its first rows are on their way, and each lane
// keeps those of its token in registers while it goes through the heads.  Warps
// share nothing until the end, so none waits for another.
//
// A group of LPR lanes holds a row, each lane two 16-byte vectors (of 16-bit
// elements) that contain both members of its pairs: vectors (s, s + r/16) of the
// half layout, any two of the interleaved one, so that the rotation needs no
// exchange.  Rotary dimensions whose halves are no multiple of a vector (a
// quarter of a head of 80, say) take the narrow layout: a warp for a row, single
// elements.
//
// The weights' gradients are summed per lane over the warp's rows, then over the
// CTA's groups, then over the CTAs by a second launch, each in a fixed order; the
// number of CTAs depends on the shapes alone.
#pragma once

#include <algorithm>

#include "../csrc_vocab/vec.cuh"
#include "block_internal.h"

namespace ls {
namespace {

constexpr int kHeadsThreads = 128;
constexpr int kHeadsWarps = kHeadsThreads / 32;

enum HeadsLayout { kHalf = 0, kInterleaved = 1, kNarrow = 2 };
enum HeadsMode { kRotate = 0, kNormFwd = 1, kNormBwd = 2 };

struct HeadsView {
    const void* p;
    int64_t bs, ss, hs;
};

struct HeadsArgs {
    HeadsView x[2], g[2], y[2];
    const void* w[2];
    int heads[2];
    int tok_shift[2];    // log2 of a unit's tokens
    int split_shift[2];  // log2 of the units that share a token's heads
    int units[2];        // of a warp
    int iters[2];        // heads that a group goes through
    int ctas0;           // CTAs of the first tensor; the others have the second
    int tokens;
    FastDiv by_seq;
    int dim, vecs, pairs;    // head_dim, its vectors, rotary_dim / 2
    FastDiv by_pairs;
    bool interleaved;        // for the narrow layout
    bool skip_rest[2];       // in place without the norm: elements behind rotary_dim stay untouched
    const uint64_t* turns;
    const int32_t* positions;
    int64_t first;
    float scale, sign;       // sign: -1 transposes the rotation
    float eps, inv_dim;
    float* partial;          // [kPartialCtas][dim]
};

// sin and cos of frac * 2^-64 of a circle.
__device__ __forceinline__ void turn_sincos(uint64_t frac, float& s, float& c) {
    const uint32_t q = static_cast<uint32_t>((frac + (uint64_t{1} << 61)) >> 62);  // the nearest quarter
    const int64_t r = static_cast<int64_t>(frac - (static_cast<uint64_t>(q) << 62));
    // |r| <= 2^61, an eighth of a turn; its upper half, in units of half a turn
    float sr, cr;
    sincospif(static_cast<float>(static_cast<int32_t>(r >> 32)) * 0x1p-31f, &sr, &cr);
    s = q & 1 ? cr : sr;
    c = q & 1 ? sr : cr;
    if (q & 2) s = -s;
    if ((q + 1) & 2) c = -c;
}

// What a lane holds of a row: the places of its 8 pairs.  The lanes' first vectors lie side by side, and so do
// their second ones: a group's access covers whole sectors of memory.
template <int LAYOUT> struct LanePlace {
    int a, b;        // wide: first elements of its two vectors, -1 if there is none; narrow: the lane
    uint32_t rot;    // bit j: pair j is rotated
};

template <int LAYOUT> __device__ __forceinline__ LanePlace<LAYOUT> lane_place(int s, const HeadsArgs& a) {
    LanePlace<LAYOUT> l;
    if constexpr (LAYOUT == kHalf) {
        const int hv = a.pairs / kVec;  // vectors of half of the rotated part
        const int rest = a.vecs - 2 * hv, v = s < hv ? s : s + hv, v2 = s < hv ? s + hv : v + (rest + 1) / 2;
        l.a = s < hv || s - hv < (rest + 1) / 2 ? v * kVec : -1;
        l.b = l.a >= 0 && v2 < a.vecs ? v2 * kVec : -1;
        l.rot = s < hv ? 0xffu : 0u;
    } else if constexpr (LAYOUT == kInterleaved) {
        const int v = s, v2 = s + (a.vecs + 1) / 2;
        l.a = v < (a.vecs + 1) / 2 ? v * kVec : -1;
        l.b = l.a >= 0 && v2 < a.vecs ? v2 * kVec : -1;
        l.rot = (l.a >= 0 && v * (kVec / 2) < a.pairs ? 0x0fu : 0u) | (l.b >= 0 && v2 * (kVec / 2) < a.pairs ? 0xf0u : 0u);
    } else {
        l.a = l.b = s;
        l.rot = 0;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            if (s + 32 * j < a.pairs) l.rot |= 1u << j;
    }
    return l;
}

// Narrow: the elements of pair number p (of dim / 2), the rotated ones first.
__device__ __forceinline__ int2 narrow_pair(int p, const HeadsArgs& a) {
    if (p >= a.pairs || a.interleaved) return make_int2(2 * p, 2 * p + 1);
    return make_int2(p, p + a.pairs);
}

template <typename T, int LAYOUT> struct RowRaw {
    Raw8<T> a, b;
};
template <typename T> struct RowRaw<T, kNarrow> {
    float a[kVec], b[kVec];
};

// A lane's part of the row at p; zeros for what does not exist.
template <typename T, int LAYOUT>
__device__ __forceinline__ void load_row(RowRaw<T, LAYOUT>& r, const T* p, bool on, const LanePlace<LAYOUT>& l,
                                         const HeadsArgs& a) {
    if constexpr (LAYOUT != kNarrow) {
        r.a = on && l.a >= 0 ? load8<T>(p + l.a) : zero8<T>();
        r.b = on && l.b >= 0 ? load8<T>(p + l.b) : zero8<T>();
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int n = l.a + 32 * j;
            const bool there = on && 2 * n < a.dim;
            const int2 e = narrow_pair(n, a);
            r.a[j] = there ? to_f32(p[e.x]) : 0.f;
            r.b[j] = there ? to_f32(p[e.y]) : 0.f;
        }
    }
}
// Its 8 pairs in FP32: the first members, and the second ones.  Two neighbours share a float2, so that the
// arithmetic takes one instruction for both.
constexpr int kHalfVec = kVec / 2;
struct Pairs {
    float2 x[kHalfVec], y[kHalfVec];
};
template <typename T, int LAYOUT> __device__ __forceinline__ Pairs pairs_of(const RowRaw<T, LAYOUT>& r) {
    Pairs p;
    float u[kVec], v[kVec];
    if constexpr (LAYOUT == kNarrow) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            u[j] = r.a[j];
            v[j] = r.b[j];
        }
    } else {
        unpack(r.a, u);
        unpack(r.b, v);
    }
#pragma unroll
    for (int j = 0; j < kHalfVec; ++j) {
        if constexpr (LAYOUT == kInterleaved) {
            const float* w = j < kHalfVec / 2 ? u : v;
            const int k = 4 * (j % (kHalfVec / 2));
            p.x[j] = make_float2(w[k], w[k + 2]);
            p.y[j] = make_float2(w[k + 1], w[k + 3]);
        } else {
            p.x[j] = make_float2(u[2 * j], u[2 * j + 1]);
            p.y[j] = make_float2(v[2 * j], v[2 * j + 1]);
        }
    }
    return p;
}
// Back to the lane's two vectors, in the row's order (narrow: first and second members).
template <int LAYOUT> __device__ __forceinline__ void vectors_of(const Pairs& p, float (&u)[kVec], float (&v)[kVec]) {
#pragma unroll
    for (int j = 0; j < kHalfVec; ++j) {
        if constexpr (LAYOUT == kInterleaved) {
            float* w = j < kHalfVec / 2 ? u : v;
            const int k = 4 * (j % (kHalfVec / 2));
            w[k] = p.x[j].x;
            w[k + 1] = p.y[j].x;
            w[k + 2] = p.x[j].y;
            w[k + 3] = p.y[j].y;
        } else {
            u[2 * j] = p.x[j].x;
            u[2 * j + 1] = p.x[j].y;
            v[2 * j] = p.y[j].x;
            v[2 * j + 1] = p.y[j].y;
        }
    }
}
template <typename T, int LAYOUT>
__device__ __forceinline__ void store_row(T* p, const Pairs& r, bool skip_rest, const LanePlace<LAYOUT>& l,
                                          const HeadsArgs& a) {
    float u[kVec], v[kVec];
    vectors_of<LAYOUT>(r, u, v);
    if constexpr (LAYOUT == kNarrow) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int n = l.a + 32 * j;
            if (2 * n >= a.dim || (skip_rest && n >= a.pairs)) continue;
            const int2 e = narrow_pair(n, a);
            p[e.x] = from_f32<T>(u[j]);
            p[e.y] = from_f32<T>(v[j]);
        }
    } else {
        // in place without the norm, vectors that hold nothing rotated are left
        const uint32_t first = LAYOUT == kHalf ? 0xffu : 0x0fu, second = LAYOUT == kHalf ? 0xffu : 0xf0u;
        if (l.a >= 0 && !(skip_rest && !(l.rot & first))) store8f<T>(p + l.a, u);
        if (l.b >= 0 && !(skip_rest && !(l.rot & second))) store8f<T>(p + l.b, v);
    }
}

// Where the cosine of pair f of a warp's token k stands in its table, its sine two floats on: a float4 holds the
// cosines and the sines of two neighbours of a lane, those of the lanes side by side.
template <int LAYOUT, int LPR> __device__ __forceinline__ int table_place(int k, int f, const HeadsArgs& a) {
    int lane, j;
    if constexpr (LAYOUT == kHalf) {
        lane = f / kVec, j = f % kVec;
    } else if constexpr (LAYOUT == kInterleaved) {
        const int v = f / (kVec / 2), first = (a.vecs + 1) / 2;
        lane = v < first ? v : v - first;
        j = f % (kVec / 2) + (v < first ? 0 : kVec / 2);
    } else {
        lane = f % 32, j = f / 32;
    }
    return ((k * kHalfVec + j / 2) * LPR + lane) * 4 + (j & 1);
}

// Rows in flight for each lane, with 16 warps on an SM.  The backward has two inputs and the weights' sums in its
// registers: two rows for each lane spill, and more warps with fewer registers are slower too (8199 x 40 x 128
// BF16, both directions: 88 us; two rows 91, five CTAs on an SM 86, but 30 instead of 20 at 4096 x 24 x 64 FP16).
template <typename T, int LAYOUT, int MODE> constexpr int heads_unroll() {
    return LAYOUT == kNarrow || MODE == kNormBwd ? 1 : sizeof(T) == 2 ? 4 : 2;
}
constexpr int kHeadsCtas = 4;  // on an SM

template <typename T, int LAYOUT, int LPR, int MODE>
__global__ void __launch_bounds__(kHeadsThreads, kHeadsCtas) heads_kernel(const __grid_constant__ HeadsArgs a) {
    constexpr int G = kHeadsThreads / LPR, GW = 32 / LPR;  // groups of a CTA, of a warp
    constexpr int U = heads_unroll<T, LAYOUT, MODE>();
    constexpr bool kCsRegs = MODE == kRotate;  // cosines and sines in registers
    constexpr int kTable = 32 * kVec;  // GW tokens of LPR * 8 pairs, at the most
    __shared__ __align__(16) float tables[kHeadsWarps * 2 * kTable];
    const int lane = threadIdx.x % LPR, warp = threadIdx.x / 32, in_warp = threadIdx.x % 32, group = in_warp / LPR;
    float* const table = tables + warp * 2 * kTable;
    const int which = blockIdx.x >= a.ctas0;
    const int cta = blockIdx.x - (which ? a.ctas0 : 0), ctas = which ? gridDim.x - a.ctas0 : a.ctas0;
    const HeadsView vx = a.x[which], vg = a.g[which], vy = a.y[which];
    const T* x = static_cast<const T*>(vx.p);
    const T* gy = static_cast<const T*>(vg.p);
    T* y = static_cast<T*>(const_cast<void*>(vy.p));
    const int shift = a.tok_shift[which], split = a.split_shift[which], heads = a.heads[which], iters = a.iters[which];
    const int side = GW >> shift, head_step = side << split, my_token = group & ((1 << shift) - 1);
    const bool skip_rest = a.skip_rest[which];
    const LanePlace<LAYOUT> place = lane_place<LAYOUT>(lane, a);
    pdl_enter();

    Pairs sum = {};  // of the weights' gradients
    __shared__ float4 ws[MODE != kRotate ? kHalfVec : 1][LPR];
    if constexpr (MODE != kRotate) {
        const T* pw = static_cast<const T*>(a.w[which]);
        Pairs w;
        if (pw) {
            RowRaw<T, LAYOUT> r;
            load_row<T, LAYOUT>(r, pw, true, place, a);
            w = pairs_of<T, LAYOUT>(r);
        } else {
#pragma unroll
            for (int j = 0; j < kHalfVec; ++j) w.x[j] = w.y[j] = make_float2(1.f, 1.f);
        }
        if (threadIdx.x < LPR)
#pragma unroll
            for (int j = 0; j < kHalfVec; ++j) ws[j][lane] = make_float4(w.x[j].x, w.x[j].y, w.y[j].x, w.y[j].y);
        __syncthreads();
    }

    for (int unit = cta * kHeadsWarps + warp; unit < a.units[which]; unit += ctas * kHeadsWarps) {
        const int t0 = (unit >> split) << shift, t = t0 + my_token;
        const int head0 = (group >> shift) + side * (unit & ((1 << split) - 1));
        const bool on = t < a.tokens;
        const int64_t b = fdiv(on ? t : 0, a.by_seq), l = fmod_(on ? t : 0, a.by_seq);
        const T* px = x + b * vx.bs + l * vx.ss;
        const T* pg = gy + b * vg.bs + l * vg.ss;
        T* py = y + b * vy.bs + l * vy.ss;
        // Rows on their way, each loaded into the place of the one that has just been used.
        RowRaw<T, LAYOUT> rx[U], rg[MODE == kNormBwd ? U : 1];
        auto load = [&](int u, int i) {
            const int h = head0 + i * head_step;
            const bool there = on && h < heads;
            load_row<T, LAYOUT>(rx[u], px + h * vx.hs, there, place, a);
            if constexpr (MODE == kNormBwd) load_row<T, LAYOUT>(rg[u], pg + h * vg.hs, there, place, a);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) load(u, u);
        __syncwarp();  // the table's readers are done
        for (int i = in_warp; i < a.pairs << shift; i += 32) {
            const int k = static_cast<int>(fdiv(i, a.by_pairs)), f = i - k * a.pairs;
            const int tk = min(t0 + k, a.tokens - 1);
            const int64_t at = a.positions ? a.positions[tk] : a.first + static_cast<int64_t>(fmod_(tk, a.by_seq));
            float s, c;
            turn_sincos(static_cast<uint64_t>(at) * a.turns[f], s, c);
            float* e = table + table_place<LAYOUT, LPR>(k, f, a);
            e[0] = c * a.scale;
            e[2] = s * a.scale * a.sign;
        }
        __syncwarp();
        const float4* turns = reinterpret_cast<const float4*>(table) + my_token * kHalfVec * LPR + lane;
        float4 cs[kCsRegs ? kHalfVec : 1];
        if constexpr (kCsRegs)
#pragma unroll
            for (int j = 0; j < kHalfVec; ++j) cs[j] = turns[j * LPR];
        auto turn = [&](Pairs& p) {
            if (place.rot == 0) return;
            const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
            for (int j = 0; j < kHalfVec; ++j) {
                const float4 q = kCsRegs ? cs[kCsRegs ? j : 0] : turns[j * LPR];
                const float2 c = make_float2(q.x, q.y), s = make_float2(q.z, q.w);
                const float2 u = fma2(mul2(p.y[j], s), minus, mul2(p.x[j], c)), v = fma2(p.x[j], s, mul2(p.y[j], c));
                if (place.rot == 0xffu) {
                    p.x[j] = u;
                    p.y[j] = v;
                } else {  // what the others hold (a NaN, say) stays out of them
                    if (place.rot >> (2 * j) & 1u) {
                        p.x[j].x = u.x;
                        p.y[j].x = v.x;
                    }
                    if (place.rot >> (2 * j + 1) & 1u) {
                        p.x[j].y = u.y;
                        p.y[j].y = v.y;
                    }
                }
            }
        };
        for (int i0 = 0; i0 < iters; i0 += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = head0 + (i0 + u) * head_step;
                const bool there = on && h < heads;
                Pairs p = pairs_of<T, LAYOUT>(rx[u]), g;
                if constexpr (MODE == kNormBwd) g = pairs_of<T, LAYOUT>(rg[u]);
                load(u, i0 + u + U);
                if constexpr (MODE != kRotate) {
                    float2 q = make_float2(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < kHalfVec; ++j) q = fma2(p.x[j], p.x[j], fma2(p.y[j], p.y[j], q));
                    const float r = rsqrtf(group_sum<LPR>(q.x + q.y) * a.inv_dim + a.eps);
                    const float2 rr = make_float2(r, r);
                    if constexpr (MODE == kNormFwd) {
#pragma unroll
                        for (int j = 0; j < kHalfVec; ++j) {
                            const float4 wj = ws[j][lane];
                            p.x[j] = mul2(mul2(p.x[j], rr), make_float2(wj.x, wj.y));
                            p.y[j] = mul2(mul2(p.y[j], rr), make_float2(wj.z, wj.w));
                        }
                        turn(p);
                    } else {
                        turn(g);
                        // with g r and w g r in the place of g: dw = sum (g r) x, dx = w g r - x r^2 mean(w g r x)
                        q = make_float2(0.f, 0.f);
#pragma unroll
                        for (int j = 0; j < kHalfVec; ++j) {
                            g.x[j] = mul2(g.x[j], rr);
                            g.y[j] = mul2(g.y[j], rr);
                            if (there) {  // r of a row that does not exist is infinite for eps = 0
                                sum.x[j] = fma2(g.x[j], p.x[j], sum.x[j]);
                                sum.y[j] = fma2(g.y[j], p.y[j], sum.y[j]);
                            }
                            const float4 wj = ws[j][lane];
                            g.x[j] = mul2(g.x[j], make_float2(wj.x, wj.y));
                            g.y[j] = mul2(g.y[j], make_float2(wj.z, wj.w));
                            q = fma2(g.x[j], p.x[j], fma2(g.y[j], p.y[j], q));
                        }
                        const float d = -group_sum<LPR>(q.x + q.y) * a.inv_dim * r * r;
                        const float2 dd = make_float2(d, d);
#pragma unroll
                        for (int j = 0; j < kHalfVec; ++j) {
                            p.x[j] = fma2(p.x[j], dd, g.x[j]);
                            p.y[j] = fma2(p.y[j], dd, g.y[j]);
                        }
                    }
                } else {
                    turn(p);
                }
                if (there) store_row<T, LAYOUT>(py + h * vy.hs, p, skip_rest, place, a);
            }
        }
    }
    if constexpr (MODE == kNormBwd) {
        if (!a.partial) return;
        // the groups' sums, in the row's order, added in the groups' order
        __syncthreads();
        float* mine = tables + (warp * GW + group) * a.dim;
        float u[kVec], v[kVec];
        vectors_of<LAYOUT>(sum, u, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if constexpr (LAYOUT == kNarrow) {
                const int n = lane + 32 * j;
                if (2 * n >= a.dim) continue;
                const int2 e = narrow_pair(n, a);
                mine[e.x] = u[j];
                mine[e.y] = v[j];
            } else {
                if (place.a >= 0) mine[place.a + j] = u[j];
                if (place.b >= 0) mine[place.b + j] = v[j];
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < a.dim; j += kHeadsThreads) {
            float total = 0.f;
            for (int k = 0; k < G; ++k) total += tables[k * a.dim + j];
            a.partial[static_cast<int64_t>(blockIdx.x) * a.dim + j] = total;
        }
    }
}

// dweight = the CTAs' sums added in their order: 32 slices of them, then the slices.  One CTA for 32 columns of
// one tensor.
template <typename T>
__global__ void __launch_bounds__(1024)
heads_dweight_kernel(T* __restrict__ dw0, T* __restrict__ dw1, const float* __restrict__ partial, int dim, int ctas0,
                     int ctas) {
    __shared__ float part[32][33];
    pdl_enter();
    T* dw = blockIdx.y ? dw1 : dw0;
    if (!dw) return;
    const int first = blockIdx.y ? ctas0 : 0, n = blockIdx.y ? ctas - ctas0 : ctas0;
    const int j = blockIdx.x * 32 + threadIdx.x;
    const int begin = n * threadIdx.y / 32, end = n * (threadIdx.y + 1) / 32;
    float sum = 0.f;
    if (j < dim)
#pragma unroll 4
        for (int k = begin; k < end; ++k) sum += partial[static_cast<int64_t>(first + k) * dim + j];
    part[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y == 0 && j < dim) {
        for (int k = 1; k < 32; ++k) sum += part[k][threadIdx.x];
        dw[j] = from_f32<T>(sum);
    }
}

template <typename T, int LAYOUT, int LPR>
cudaError_t launch_mode(const HeadsArgs& a, const HeadsCall& c, int ctas, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(ctas)), block(kHeadsThreads);
    if (!c.norm) return launch_pdl(heads_kernel<T, LAYOUT, LPR, kRotate>, grid, block, 0, s, a);
    if (!c.backward) return launch_pdl(heads_kernel<T, LAYOUT, LPR, kNormFwd>, grid, block, 0, s, a);
    return launch_pdl(heads_kernel<T, LAYOUT, LPR, kNormBwd>, grid, block, 0, s, a);
}

template <typename T, int LAYOUT>
cudaError_t launch_width(int lpr, const HeadsArgs& a, const HeadsCall& c, int ctas, cudaStream_t s) {
    if (lpr == 4) return launch_mode<T, LAYOUT, 4>(a, c, ctas, s);
    if (lpr == 8) return launch_mode<T, LAYOUT, 8>(a, c, ctas, s);
    if (lpr == 16) return launch_mode<T, LAYOUT, 16>(a, c, ctas, s);
    return launch_mode<T, LAYOUT, 32>(a, c, ctas, s);
}

HeadsView view_of(const ls_head_view* v) {
    return v ? HeadsView{v->data, v->batch_stride, v->seq_stride, v->head_stride} : HeadsView{nullptr, 0, 0, 0};
}

// A unit's tokens, and the units that share their heads.  The groups that share a token go through its heads
// side by side: few of them leave each more heads to use its cosines on, many end sooner.  Counted in rounds of
// the warps that the GPU holds (`slots` of them are this tensor's), a round being the heads that a group goes
// through and about one and a half more for the angles.
void plan_units(HeadsArgs& a, int which, int groups, int64_t slots) {
    int64_t best = INT64_MAX;
    for (int split = 0; split <= 5; ++split)
        for (int shift = 0; (1 << shift) <= groups; ++shift) {
            const int64_t step = static_cast<int64_t>(groups >> shift) << split;
            if (split > 0 && step >= 2 * a.heads[which]) continue;
            const int64_t iters = (a.heads[which] + step - 1) / step;
            const int64_t units = ((static_cast<int64_t>(a.tokens) + (1 << shift) - 1) >> shift) << split;
            const int64_t t = (units + slots - 1) / slots * (2 * iters + 3);
            if (units > INT32_MAX / 2 || t > best || (t == best && split > a.split_shift[which])) continue;
            best = t;
            a.tok_shift[which] = shift;
            a.split_shift[which] = split;
            a.iters[which] = static_cast<int>(iters);
            a.units[which] = static_cast<int>(units);
        }
}

}  // namespace

template <typename T> cudaError_t launch_heads(const HeadsCall& c, cudaStream_t s) {
    HeadsArgs a = {};
    a.tokens = static_cast<int>(c.batch * c.seq);
    a.by_seq = make_fastdiv(static_cast<uint32_t>(c.seq));
    a.dim = static_cast<int>(c.dim);
    a.vecs = a.dim / kVec;
    a.eps = c.eps;
    a.inv_dim = 1.f / static_cast<float>(a.dim);
    a.sign = c.backward ? -1.f : 1.f;
    a.scale = 1.f;
    if (const ls_rotation* r = c.rotation) {
        a.pairs = static_cast<int>(r->rotary_dim / 2);
        a.interleaved = r->interleaved != 0;
        a.turns = r->turns;
        a.positions = r->positions;
        a.first = r->first_position;
        a.scale = r->scale;
    }
    a.by_pairs = make_fastdiv(static_cast<uint32_t>(std::max(a.pairs, 1)));
    const int layout = a.pairs % (a.interleaved ? kVec / 2 : kVec) ? kNarrow : a.interleaved ? kInterleaved : kHalf;
    int lpr = 32;
    if (layout != kNarrow)
        for (lpr = 4; 2 * lpr < a.vecs;) lpr *= 2;
    const bool partial = c.norm && c.backward && (c.dweight[0] || c.dweight[1]);
    int64_t rows[2] = {0, 0};
    for (int k = 0; k < 2; ++k) {
        if (!c.x[k]) continue;
        a.x[k] = view_of(c.x[k]);
        a.g[k] = view_of(c.g[k]);
        a.y[k] = view_of(c.y[k]);
        a.w[k] = c.weight[k];
        a.heads[k] = static_cast<int>(c.x[k]->heads);
        a.skip_rest[k] = !c.norm && c.x[k]->data == c.y[k]->data;
        rows[k] = static_cast<int64_t>(a.tokens) * a.heads[k];
    }
    int64_t ctas[2] = {0, 0};
    for (int k = 0; k < 2; ++k) {
        if (!rows[k]) continue;
        plan_units(a, k, 32 / lpr, std::max<int64_t>(1, 152 * 16 * rows[k] / (rows[0] + rows[1])));
        ctas[k] = (a.units[k] + kHeadsWarps - 1) / kHeadsWarps;
    }
    if (partial && ctas[0] + ctas[1] > kPartialCtas) {  // in proportion to the rows, at least one each
        const int64_t share = (kPartialCtas * rows[0] + (rows[0] + rows[1]) / 2) / (rows[0] + rows[1]);
        const int64_t most0 = kPartialCtas - std::min<int64_t>(ctas[1], 1);
        ctas[0] = std::min(ctas[0], std::min(most0, std::max<int64_t>(share, std::min<int64_t>(ctas[0], 1))));
        ctas[1] = std::min(ctas[1], kPartialCtas - ctas[0]);
    }
    a.ctas0 = static_cast<int>(ctas[0]);
    a.partial = partial ? static_cast<float*>(c.workspace) : nullptr;
    const int all = static_cast<int>(ctas[0] + ctas[1]);
    cudaError_t e = cudaSuccess;
    if (all > 0) {
        e = layout == kNarrow         ? launch_mode<T, kNarrow, 32>(a, c, all, s)
            : layout == kInterleaved ? launch_width<T, kInterleaved>(lpr, a, c, all, s)
                                     : launch_width<T, kHalf>(lpr, a, c, all, s);
    }
    if (e != cudaSuccess || !partial) return e;
    // zeros for a tensor without rows
    return launch_pdl(heads_dweight_kernel<T>, dim3(static_cast<unsigned>((c.dim + 31) / 32), 2), dim3(32, 32), 0, s,
                      static_cast<T*>(c.dweight[0]), static_cast<T*>(c.dweight[1]), static_cast<const float*>(a.partial), a.dim,
                      a.ctas0, all);
}

}  // namespace ls
