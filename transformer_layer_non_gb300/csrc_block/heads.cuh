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
// position; sincospif gets at most an eighth of a turn.  A CTA takes a tile of
// tokens with all their heads, works out its tokens' cosines and sines once into
// shared memory, and each group of lanes keeps those of its token in registers
// while it goes through the heads.
//
// A group of LPR lanes holds a row, each lane two 16-byte vectors (of 16-bit
// elements) that contain both members of its pairs: vectors (s, s + r/16) of the
// half layout, (2s, 2s + 1) of the interleaved one, so that the rotation needs
// no exchange.  Rotary dimensions whose halves are no multiple of a vector (a
// quarter of a head of 80, say) take the narrow layout: a warp for a row, single
// elements.
//
// The weights' gradients are summed per lane over the CTA's rows, then over the
// CTA's groups, then over the CTAs by a second launch, each in a fixed order; the
// number of CTAs depends on the shapes alone.
#pragma once

#include <algorithm>

#include "../csrc_vocab/vec.cuh"
#include "block_internal.h"

namespace ls {
namespace {

constexpr int kHeadsThreads = 256;

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
    int tok[2];       // tokens of a tile, a power of two
    int tok_shift[2];
    int tiles[2];
    int iters[2];     // heads that a group goes through
    int ctas0;        // CTAs of the first tensor; the others have the second
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

// What a lane holds of a row: the places of its 8 pairs.
template <int LAYOUT> struct LanePlace {
    int a, b;        // wide: first elements of its two vectors, -1 if there is none; narrow: the lane
    uint32_t rot;    // bit j: pair j is rotated
    int freq;        // wide: the first pair's number
};

template <int LAYOUT> __device__ __forceinline__ LanePlace<LAYOUT> lane_place(int s, const HeadsArgs& a) {
    LanePlace<LAYOUT> l;
    l.freq = s * kVec;
    if constexpr (LAYOUT == kHalf) {
        const int hv = a.pairs / kVec;  // vectors of half of the rotated part
        const int v = s < hv ? s : 2 * s;  // behind it (2 hv + 2 (s - hv)) two neighbours each
        const int v2 = s < hv ? s + hv : 2 * s + 1;
        l.a = v < a.vecs ? v * kVec : -1;
        l.b = v2 < a.vecs ? v2 * kVec : -1;
        l.rot = s < hv ? 0xffu : 0u;
    } else if constexpr (LAYOUT == kInterleaved) {
        const int v = 2 * s;
        l.a = v < a.vecs ? v * kVec : -1;
        l.b = v + 1 < a.vecs ? (v + 1) * kVec : -1;
        l.rot = (v * (kVec / 2) < a.pairs ? 0x0fu : 0u) | ((v + 1) * (kVec / 2) < a.pairs ? 0xf0u : 0u);
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
// Its pairs in FP32.
template <typename T, int LAYOUT>
__device__ __forceinline__ void pairs_of(const RowRaw<T, LAYOUT>& r, float (&x)[kVec], float (&y)[kVec]) {
    if constexpr (LAYOUT == kHalf) {
        unpack(r.a, x);
        unpack(r.b, y);
    } else if constexpr (LAYOUT == kInterleaved) {
        float u[kVec], v[kVec];
        unpack(r.a, u);
        unpack(r.b, v);
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j) {
            x[j] = u[2 * j];
            y[j] = u[2 * j + 1];
            x[j + kVec / 2] = v[2 * j];
            y[j + kVec / 2] = v[2 * j + 1];
        }
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            x[j] = r.a[j];
            y[j] = r.b[j];
        }
    }
}
template <typename T, int LAYOUT>
__device__ __forceinline__ void store_row(T* p, const float (&x)[kVec], const float (&y)[kVec], bool skip_rest,
                                          const LanePlace<LAYOUT>& l, const HeadsArgs& a) {
    if constexpr (LAYOUT == kHalf) {
        if (skip_rest && !l.rot) return;
        if (l.a >= 0) store8f<T>(p + l.a, x);
        if (l.b >= 0) store8f<T>(p + l.b, y);
    } else if constexpr (LAYOUT == kInterleaved) {
        float u[kVec], v[kVec];
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j) {
            u[2 * j] = x[j];
            u[2 * j + 1] = y[j];
            v[2 * j] = x[j + kVec / 2];
            v[2 * j + 1] = y[j + kVec / 2];
        }
        if (l.a >= 0 && !(skip_rest && !(l.rot & 0x0fu))) store8f<T>(p + l.a, u);
        if (l.b >= 0 && !(skip_rest && !(l.rot & 0xf0u))) store8f<T>(p + l.b, v);
    } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int n = l.a + 32 * j;
            if (2 * n >= a.dim || (skip_rest && n >= a.pairs)) continue;
            const int2 e = narrow_pair(n, a);
            p[e.x] = from_f32<T>(x[j]);
            p[e.y] = from_f32<T>(y[j]);
        }
    }
}

// (x, y) <- the rotated pairs.
__device__ __forceinline__ void rotate(float (&x)[kVec], float (&y)[kVec], const float (&c)[kVec],
                                       const float (&s)[kVec], uint32_t rot) {
    if (rot == 0) return;
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        const float u = x[j] * c[j] - y[j] * s[j], v = x[j] * s[j] + y[j] * c[j];
        if (rot == 0xffu || (rot >> j & 1u)) {  // what the others hold (a NaN, say) stays out of them
            x[j] = u;
            y[j] = v;
        }
    }
}

// Rows in flight for each lane.
template <typename T, int LAYOUT, int MODE> constexpr int heads_unroll() {
    return LAYOUT == kNarrow ? 1 : MODE == kNormBwd ? (sizeof(T) == 2 ? 2 : 1) : sizeof(T) == 2 ? 4 : 2;
}

template <typename T, int LAYOUT, int LPR, int MODE>
__global__ void __launch_bounds__(kHeadsThreads) heads_kernel(const __grid_constant__ HeadsArgs a) {
    constexpr int G = kHeadsThreads / LPR;  // groups
    constexpr int U = heads_unroll<T, LAYOUT, MODE>();
    constexpr int kTable = kHeadsThreads * kVec;  // G tokens of LPR * 8 pairs, at the most
    __shared__ __align__(16) float table[2 * kTable];
    const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
    const int which = blockIdx.x >= a.ctas0;
    const int cta = blockIdx.x - (which ? a.ctas0 : 0), ctas = which ? gridDim.x - a.ctas0 : a.ctas0;
    const HeadsView vx = a.x[which], vg = a.g[which], vy = a.y[which];
    const T* x = static_cast<const T*>(vx.p);
    const T* gy = static_cast<const T*>(vg.p);
    T* y = static_cast<T*>(const_cast<void*>(vy.p));
    const int tok = a.tok[which], shift = a.tok_shift[which], heads = a.heads[which], iters = a.iters[which];
    const int head_groups = G >> shift, head0 = group >> shift, my_token = group & (tok - 1);
    const bool skip_rest = a.skip_rest[which];
    const LanePlace<LAYOUT> place = lane_place<LAYOUT>(lane, a);
    const int stride = (a.pairs + kVec - 1) & ~(kVec - 1);  // of a token's cosines
    pdl_enter();

    float w1[kVec], w2[kVec], s1[kVec], s2[kVec];
    if constexpr (MODE != kRotate) {
        const T* w = static_cast<const T*>(a.w[which]);
        if (w) {
            RowRaw<T, LAYOUT> r;
            load_row<T, LAYOUT>(r, w, true, place, a);
            pairs_of<T, LAYOUT>(r, w1, w2);
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) w1[j] = w2[j] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) s1[j] = s2[j] = 0.f;
    }

    for (int tile = cta; tile < a.tiles[which]; tile += ctas) {
        const int t0 = tile << shift;
        __syncthreads();  // the table's readers are done
        for (int i = threadIdx.x; i < a.pairs << shift; i += kHeadsThreads) {
            const int k = static_cast<int>(fdiv(i, a.by_pairs)), f = i - k * a.pairs;
            const int t = min(t0 + k, a.tokens - 1);
            const int64_t at = a.positions ? a.positions[t] : a.first + static_cast<int64_t>(fmod_(t, a.by_seq));
            float s, c;
            turn_sincos(static_cast<uint64_t>(at) * a.turns[f], s, c);
            table[k * stride + f] = c * a.scale;
            table[kTable + k * stride + f] = s * a.scale * a.sign;
        }
        __syncthreads();
        const int t = t0 + my_token;
        const bool on = t < a.tokens;
        float c[kVec], s[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const int f = LAYOUT == kNarrow ? lane + 32 * j : place.freq + j;
            const bool there = place.rot >> j & 1u;
            c[j] = there ? table[my_token * stride + f] : 1.f;
            s[j] = there ? table[kTable + my_token * stride + f] : 0.f;
        }
        const int64_t b = fdiv(on ? t : 0, a.by_seq), l = fmod_(on ? t : 0, a.by_seq);
        const int64_t ox = b * vx.bs + l * vx.ss, og = b * vg.bs + l * vg.ss, oy = b * vy.bs + l * vy.ss;
        for (int i0 = 0; i0 < iters; i0 += U) {
            RowRaw<T, LAYOUT> rx[U], rg[MODE == kNormBwd ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = head0 + (i0 + u) * head_groups;
                const bool there = on && h < heads;
                load_row<T, LAYOUT>(rx[u], x + ox + h * vx.hs, there, place, a);
                if constexpr (MODE == kNormBwd) load_row<T, LAYOUT>(rg[u], gy + og + h * vg.hs, there, place, a);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = head0 + (i0 + u) * head_groups;
                const bool there = on && h < heads;
                float x1[kVec], x2[kVec];
                pairs_of<T, LAYOUT>(rx[u], x1, x2);
                if constexpr (MODE != kRotate) {
                    float sum = 0.f;
#pragma unroll
                    for (int j = 0; j < kVec; ++j) sum = fmaf(x1[j], x1[j], fmaf(x2[j], x2[j], sum));
                    const float r = rsqrtf(group_sum<LPR>(sum) * a.inv_dim + a.eps);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        x1[j] *= r;
                        x2[j] *= r;
                    }
                    if constexpr (MODE == kNormFwd) {
#pragma unroll
                        for (int j = 0; j < kVec; ++j) {
                            x1[j] *= w1[j];
                            x2[j] *= w2[j];
                        }
                        rotate(x1, x2, c, s, place.rot);
                    } else {
                        float g1[kVec], g2[kVec];
                        pairs_of<T, LAYOUT>(rg[u], g1, g2);
                        rotate(g1, g2, c, s, place.rot);
                        float dot = 0.f;
#pragma unroll
                        for (int j = 0; j < kVec; ++j) {
                            if (there) {  // a row that does not exist has u = 0 / sqrt(eps), a NaN for eps = 0
                                s1[j] = fmaf(g1[j], x1[j], s1[j]);
                                s2[j] = fmaf(g2[j], x2[j], s2[j]);
                            }
                            g1[j] *= w1[j];
                            g2[j] *= w2[j];
                            dot = fmaf(g1[j], x1[j], fmaf(g2[j], x2[j], dot));
                        }
                        dot = group_sum<LPR>(dot) * a.inv_dim;
#pragma unroll
                        for (int j = 0; j < kVec; ++j) {
                            x1[j] = (g1[j] - x1[j] * dot) * r;
                            x2[j] = (g2[j] - x2[j] * dot) * r;
                        }
                    }
                } else {
                    rotate(x1, x2, c, s, place.rot);
                }
                if (there) store_row<T, LAYOUT>(y + oy + h * vy.hs, x1, x2, skip_rest, place, a);
            }
        }
    }
    if constexpr (MODE == kNormBwd) {
        if (!a.partial) return;
        // the groups' sums, in the row's order, added in the groups' order
        __syncthreads();
        float* mine = table + group * a.dim;
        if constexpr (LAYOUT == kNarrow) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const int n = lane + 32 * j;
                if (2 * n >= a.dim) continue;
                const int2 e = narrow_pair(n, a);
                mine[e.x] = s1[j];
                mine[e.y] = s2[j];
            }
        } else if constexpr (LAYOUT == kHalf) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                if (place.a >= 0) mine[place.a + j] = s1[j];
                if (place.b >= 0) mine[place.b + j] = s2[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec / 2; ++j) {
                if (place.a >= 0) {
                    mine[place.a + 2 * j] = s1[j];
                    mine[place.a + 2 * j + 1] = s2[j];
                }
                if (place.b >= 0) {
                    mine[place.b + 2 * j] = s1[j + kVec / 2];
                    mine[place.b + 2 * j + 1] = s2[j + kVec / 2];
                }
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < a.dim; j += kHeadsThreads) {
            float sum = 0.f;
            for (int k = 0; k < G; ++k) sum += table[k * a.dim + j];
            a.partial[static_cast<int64_t>(blockIdx.x) * a.dim + j] = sum;
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

// Tokens of a tile: the groups that share a token go through its heads side by side.  Few groups a token leave
// each more heads to use its cosines on; many make more tiles.  Counted in rounds of the GPU's 152 x 6 CTAs, a
// round being the heads that a group goes through and about one more for the angles.
void plan_tile(HeadsArgs& a, int which, int groups, int64_t most_ctas) {
    int64_t best = INT64_MAX;
    for (int shift = 0; (1 << shift) <= groups; ++shift) {
        const int side = groups >> shift;
        const int64_t iters = (a.heads[which] + side - 1) / side;
        const int64_t tiles = (static_cast<int64_t>(a.tokens) + (1 << shift) - 1) >> shift;
        const int64_t t = (tiles + most_ctas - 1) / most_ctas * (iters + 1);
        if (t <= best) {
            best = t;
            a.tok[which] = 1 << shift;
            a.tok_shift[which] = shift;
            a.iters[which] = static_cast<int>(iters);
            a.tiles[which] = static_cast<int>(tiles);
        }
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
        if (rows[k]) plan_tile(a, k, kHeadsThreads / lpr, partial ? kPartialCtas : 152 * 6);
    }
    int64_t ctas[2] = {a.tiles[0], a.tiles[1]};
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
