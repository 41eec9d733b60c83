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
// position; the polynomials get at most an eighth of a turn.  A warp takes a few
// tokens with all their heads (or, of few tokens, some of them), works out its
// tokens' cosines and sines once, while its first rows are on their way, and goes
// through the rows.  Warps share nothing until the end, so none waits for another.
//
// A group of LPR lanes holds a row, each lane 8 pairs of its elements, so that the
// rotation needs no exchange.  Interleaved: any two vectors of 8 elements.  Halves:
// as many chunks of W elements of the first half as of the second, W being what
// divides the half, 8 or fewer: chunk n and chunk n + half / W.  What is not rotated
// is paired the same way.
//
// The weights' gradients are summed per lane over the warp's rows, then over the
// CTA's groups, then over the CTAs by a second launch, each in a fixed order; the
// number of CTAs depends on the shapes alone.
#pragma once

#include <string.h>

#include <algorithm>
#include <type_traits>

#include "../csrc_vocab/vec.cuh"
#include "block_internal.h"

namespace ls {
namespace {

constexpr int kHeadsThreads = 128;
constexpr int kHeadsWarps = kHeadsThreads / 32;

// A layout is the chunks' width of halves, 8 (16-bit storage), 4, 2 or 1, or
constexpr int kInterleaved = 0;
enum HeadsMode { kRotate = 0, kNormFwd = 1, kNormBwd = 2 };

struct HeadsView {
    const void* p;
    int64_t bs, ss, hs;
};

struct HeadsArgs {
    HeadsView x[2], g[2], y[2];
    const void* w[2];
    int heads[2];
    int tok_shift[2];    // log2 of a unit's tokens that are side by side
    int sub_shift[2];    // and of those that a group goes through one after the other
    int split_shift[2];  // log2 of the units that share a token's heads
    uint32_t units[2];   // of a warp
    int iters[2];        // heads of a token that a group goes through
    int ctas0;           // CTAs of the first tensor; the others have the second
    int tokens;
    FastDiv by_seq;
    int dim, pairs;          // head_dim, rotary_dim / 2
    FastDiv by_pairs;
    bool skip_rest[2];       // in place without the norm: elements behind rotary_dim stay untouched
    const uint64_t* turns;
    const int32_t* positions;
    int32_t first;
    float scale, sign;       // sign: -1 transposes the rotation
    float eps, inv_dim;
    float* partial;          // [kPartialCtas][dim]
};

// sin and cos of turns * position * 2^-64 of a circle: the upper 32 bits of the product (below them 1.5e-9 of an angle).
__device__ __forceinline__ void turn_sincos(uint64_t turns, int32_t position, float& s, float& c) {
    const uint32_t lo = static_cast<uint32_t>(turns), hi = static_cast<uint32_t>(turns >> 32);
    const uint32_t at = static_cast<uint32_t>(position);
    const uint32_t frac = __umulhi(lo, at) + hi * at - (position < 0 ? lo : 0u);
    const uint32_t q = (frac + (1u << 29)) >> 30;  // the nearest quarter
    const int32_t r = static_cast<int32_t>(frac - (q << 30));
    // at most an eighth of a turn; in radians, and Taylor's series, whose next terms are below 2e-9 and 1e-10
    const float x = static_cast<float>(r) * 1.4629180792671596e-9f, z = x * x;
    const float sr = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), x);
    const float cr = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
    // quarters turn (c, s) into (-s, c), (-c, -s) and (s, -c)
    s = __uint_as_float(__float_as_uint(q & 1 ? cr : sr) ^ ((q << 30) & 0x80000000u));
    c = __uint_as_float(__float_as_uint(q & 1 ? sr : cr) ^ (((q + 1) << 30) & 0x80000000u));
}

// W elements of the storage type, as they lie in memory.
template <typename T, int W> struct Chunk {
    using Word = std::conditional_t<W * sizeof(T) == 2, uint16_t, uint32_t>;
    static constexpr int kWords = W * sizeof(T) / sizeof(Word);
    Word w[kWords];
};
template <typename T, int W> __device__ __forceinline__ Chunk<T, W> load_chunk(const T* p) {
    Chunk<T, W> c;
    if constexpr (W * sizeof(T) >= 16) {
#pragma unroll
        for (int i = 0; i < c.kWords; i += 4) {
            const uint4 v = ld16(reinterpret_cast<const uint32_t*>(p) + i);
            c.w[i] = v.x, c.w[i + 1] = v.y, c.w[i + 2] = v.z, c.w[i + 3] = v.w;
        }
    } else if constexpr (W * sizeof(T) == 8) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        c.w[0] = v.x, c.w[1] = v.y;
    } else {
        c.w[0] = *reinterpret_cast<const typename Chunk<T, W>::Word*>(p);
    }
    return c;
}
template <typename T, int W> __device__ __forceinline__ void store_chunk(T* p, const Chunk<T, W>& c) {
    if constexpr (W * sizeof(T) >= 16) {
#pragma unroll
        for (int i = 0; i < c.kWords; i += 4)
            st16(reinterpret_cast<uint32_t*>(p) + i, make_uint4(c.w[i], c.w[i + 1], c.w[i + 2], c.w[i + 3]));
    } else if constexpr (W * sizeof(T) == 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
    } else {
        *reinterpret_cast<typename Chunk<T, W>::Word*>(p) = c.w[0];
    }
}
// Into f[k .. k + W), and back.
template <typename T, int W> __device__ __forceinline__ void unpack_chunk(const Chunk<T, W>& c, float (&f)[kVec], int k) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) f[k + i] = __uint_as_float(c.w[i]);
    } else if constexpr (W == 1) {
        T v;
        memcpy(&v, &c.w[0], 2);
        f[k] = to_f32(v);
    } else {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const float2 t = std::is_same<T, bf16>::value ? b2f(c.w[i]) : h2f(c.w[i]);
            f[k + 2 * i] = t.x, f[k + 2 * i + 1] = t.y;
        }
    }
}
template <typename T, int W> __device__ __forceinline__ Chunk<T, W> pack_chunk(const float (&f)[kVec], int k) {
    Chunk<T, W> c;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) c.w[i] = __float_as_uint(f[k + i]);
    } else if constexpr (W == 1) {
        const T v = from_f32<T>(f[k]);
        memcpy(&c.w[0], &v, 2);
    } else {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) c.w[i] = pack2<T>(f[k + 2 * i], f[k + 2 * i + 1]);
    }
    return c;
}

// Where a lane's 8 pairs are: J chunks of W elements with the first members and J with the second ones (halves), or
// 2 J vectors of neighbours (interleaved).  The lanes' chunks j lie side by side: a group's access covers whole sectors
// of memory.
template <typename T, int LAYOUT> constexpr int chunk_width() { return LAYOUT == kInterleaved ? 16 / sizeof(T) : LAYOUT; }
template <typename T, int LAYOUT, int LPR> struct LanePlace {
    static constexpr int W = chunk_width<T, LAYOUT>(), J = kVec / W;
    int lane, all;   // chunks of a row
    int turned;      // halves: chunk pairs that are rotated
    int apart;       // halves: the chunks from a pair that is not rotated to its second one
    uint32_t rot;    // bit k: pair k is rotated

    __device__ __forceinline__ LanePlace(int s, const HeadsArgs& a) : lane(s), all(a.dim / W), turned(0), apart(0), rot(0) {
        if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
            for (int k = 0; k < kVec; ++k) {
                const int n = s + LPR * (k / (W / 2));
                if (n < all && n * (W / 2) + k % (W / 2) < a.pairs) rot |= 1u << k;
            }
        } else {
            turned = a.pairs / W;
            apart = (all - 2 * turned + 1) / 2;
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (s + LPR * j < turned) rot |= ((1u << W) - 1) << (j * W);
        }
    }
    // The elements where its chunks j begin, and whether they exist.
    __device__ __forceinline__ int first(int j, bool& there) const {
        const int n = lane + LPR * j;
        there = n < (LAYOUT == kInterleaved ? all : turned + apart);
        return (LAYOUT == kInterleaved || n < turned ? n : n + turned) * W;
    }
    __device__ __forceinline__ int second(int j, bool& there) const {
        const int n = lane + LPR * j;
        const int c = LAYOUT == kInterleaved ? n + LPR * J : n < turned ? n + turned : n + turned + apart;
        there = c < all && (LAYOUT == kInterleaved || n < turned + apart);
        return c * W;
    }
    // Which of the W elements of a first chunk j (with `later` a second one) are rotated: a bit for each, or for each
    // two (interleaved).
    static constexpr uint32_t kWhole = (1u << (LAYOUT == kInterleaved ? W / 2 : W)) - 1;
    __device__ __forceinline__ uint32_t rotated(int j, bool later) const {
        return rot >> (LAYOUT == kInterleaved ? (j + (later ? J : 0)) * (W / 2) : j * W) & kWhole;
    }
};

// Its 8 pairs in FP32: the first members, and the second ones.  Two neighbours share a float2, so that the
// arithmetic takes one instruction for both.
constexpr int kHalfVec = kVec / 2;
struct Pairs {
    float2 x[kHalfVec], y[kHalfVec];
};
// A lane's chunks, in order: the first members' and the second ones'.
template <typename T, int LAYOUT> struct RowRaw {
    static constexpr int W = chunk_width<T, LAYOUT>(), J = kVec / W;
    Chunk<T, W> a[J], b[J];
};
template <typename T, int LAYOUT> __device__ __forceinline__ Pairs pairs_of(const RowRaw<T, LAYOUT>& r) {
    Pairs p;
    float u[kVec], v[kVec];
#pragma unroll
    for (int j = 0; j < r.J; ++j) {
        unpack_chunk(r.a[j], u, j * r.W);
        unpack_chunk(r.b[j], v, j * r.W);
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
// Back to the lane's chunks, one after the other.
template <int LAYOUT> __device__ __forceinline__ void chunks_of(const Pairs& p, float (&u)[kVec], float (&v)[kVec]) {
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

// 16 bytes from memory to shared memory, without registers.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// At most N of this thread's groups of copies are still under way.
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The ring that a warp's rows come through: slots of a row for each group, in memory's vectors of 16 bytes.  Where
// chunks are such vectors (kOwn) each lane copies, reads and stores its own ones, and no lane waits for another;
// narrower chunks are read from, and put back into, the row as it lies in memory.
template <typename T, int LAYOUT, int LPR> struct Ring {
    using Place = LanePlace<T, LAYOUT, LPR>;
    static constexpr int W = Place::W, J = Place::J;
    static constexpr bool kOwn = W * sizeof(T) == 16;
    static constexpr int kVecs = sizeof(T);            // vectors of a lane: 16 elements
    static constexpr int kElems = 16 / sizeof(T);      // elements of a vector
    // 16 bytes more for a row that lanes read across, so that not all of a warp's rows begin in the same bank.
    static constexpr uint32_t kRowBytes = LPR * kVecs * 16 + (kOwn ? 0 : 16);
    static constexpr uint32_t kSlotBytes = 32 / LPR * kRowBytes;

    // The elements where a lane's vector i begins, whether it exists, and where it is in a slot.
    static __device__ __forceinline__ int element(const Place& l, int i, bool& there) {
        if constexpr (kOwn) {
            return i < J ? l.first(i, there) : l.second(i - J, there);
        } else {
            const int v = l.lane + LPR * i;
            there = v < l.all * W / kElems;
            return v * kElems;
        }
    }
    static __device__ __forceinline__ uint32_t place(const Place& l, int i) {
        const uint32_t in_warp = threadIdx.x % 32;
        if constexpr (kOwn) return (i * 32 + in_warp) * 16;
        return in_warp / LPR * kRowBytes + (l.lane + LPR * i) * 16;
    }
    static __device__ __forceinline__ T* row(unsigned char* slot) {
        return reinterpret_cast<T*>(slot + threadIdx.x % 32 / LPR * kRowBytes);
    }
    // Zeros for vectors that do not exist: they are never copied over.
    static __device__ __forceinline__ void clear(unsigned char* slot, const Place& l) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            bool there;
            element(l, i, there);
            if (!there) st16(slot + place(l, i), make_uint4(0, 0, 0, 0));
        }
    }
    static __device__ __forceinline__ void load(unsigned char* slot, const T* p, const Place& l) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            bool there;
            const int e = element(l, i, there);
            if (there) copy16(smem_u32(slot + place(l, i)), p + e);
        }
    }
    // A lane's chunks of the row in the slot; zeros for those that do not exist.
    static __device__ __forceinline__ RowRaw<T, LAYOUT> read(unsigned char* slot, const Place& l) {
        RowRaw<T, LAYOUT> r;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if constexpr (kOwn) {
                r.a[j] = load_chunk<T, W>(reinterpret_cast<const T*>(slot + place(l, j)));
                r.b[j] = load_chunk<T, W>(reinterpret_cast<const T*>(slot + place(l, J + j)));
            } else {
                bool ta, tb;
                const int a = l.first(j, ta), b = l.second(j, tb);
                r.a[j] = ta ? load_chunk<T, W>(row(slot) + a) : Chunk<T, W>{};
                r.b[j] = tb ? load_chunk<T, W>(row(slot) + b) : Chunk<T, W>{};
            }
        }
        return r;
    }
    // From registers to memory.  keep: what is not rotated is stored as it was read (raw); skip: it is not stored.
    static __device__ __forceinline__ void store(unsigned char* slot, T* p, const Pairs& r, const RowRaw<T, LAYOUT>& raw,
                                                 bool there, bool keep, bool skip, int rotated, const Place& l) {
        float u[kVec], v[kVec];
        chunks_of<LAYOUT>(r, u, v);
        if constexpr (kOwn) {
            if (!there) return;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                bool is;
                const int e = element(l, i, is), j = i % J;
                const float(&f)[kVec] = i < J ? u : v;
                const uint32_t bits = l.rotated(j, i >= J);
                Chunk<T, W> c = pack_chunk<T, W>(f, j * W);
                if (keep && sizeof(T) == 2 && bits != Place::kWhole) {
#pragma unroll
                    for (int k = 0; k < c.kWords; ++k)  // two neighbours; of halves, all or nothing
                        if (!(bits >> k & 1u)) c.w[k] = (i < J ? raw.a[j] : raw.b[j]).w[k];
                }
                if (!is) continue;
                if (!skip || bits == Place::kWhole) {
                    store_chunk<T, W>(p + e, c);
                } else if (LAYOUT == kInterleaved) {
#pragma unroll
                    for (int k = 0; k < W; ++k)
                        if (bits >> k / 2 & 1u) p[e + k] = from_f32<T>(f[j * W + k]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                bool ta, tb;
                const int a = l.first(j, ta), b = l.second(j, tb);
                if (keep && !l.rotated(j, false)) continue;
                if (ta) store_chunk<T, W>(row(slot) + a, pack_chunk<T, W>(u, j * W));
                if (tb) store_chunk<T, W>(row(slot) + b, pack_chunk<T, W>(v, j * W));
            }
            __syncwarp();
            if (there) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    bool is;
                    const int e = element(l, i, is);
                    if (!is || (skip && e >= rotated)) continue;
                    if (!skip || e + kElems <= rotated)
                        st16(p + e, ld16(row(slot) + e));
                    else
                        for (int k = e; k < rotated; ++k) p[k] = row(slot)[k];
                }
            }
            __syncwarp();  // the slot is free
        }
    }
};

// Where the cosine of pair f of a warp's token k stands in its table, its sine two floats on: a float4 holds the
// cosines and the sines of two neighbours of a lane, those of the lanes and tokens side by side.
template <typename T, int LAYOUT, int LPR> __device__ __forceinline__ int table_place(int k, int f, int unit_shift) {
    constexpr int W = LAYOUT == kInterleaved ? chunk_width<T, LAYOUT>() / 2 : chunk_width<T, LAYOUT>();
    const int n = f / W, j = n / LPR * W + f % W;
    return (((j / 2 << unit_shift) + k) * LPR + n % LPR) * 4 + (j & 1);
}

// Slots of a warp's ring: 128 bytes for each lane, and two rows at least.  With four CTAs on an SM that is enough in
// flight (rotation 16411 x 40 x 128 BF16: 51 us, 6.6 TB/s; norm forward and backward 8199 x 40 x 128 BF16 78, with three
// slots for the backward 82, with five CTAs 88, three 93).
template <typename T, int MODE> constexpr int ring_slots() { return sizeof(T) == 2 && MODE != kNormBwd ? 4 : 2; }
constexpr int kHeadsCtas = 4;  // on an SM
// Tokens that a group goes through one after the other, at the most (161805 x 4 x 96 BF16: 73 us; of two 80, of eight 73).
constexpr int kMostSub = 2;  // log2

template <typename T, int LAYOUT, int LPR, int MODE>
__global__ void __launch_bounds__(kHeadsThreads, kHeadsCtas) heads_kernel(const __grid_constant__ HeadsArgs a) {
    constexpr int G = kHeadsThreads / LPR, GW = 32 / LPR;  // groups of a CTA, of a warp
    constexpr int D = ring_slots<T, MODE>();
    constexpr bool kCsRegs = MODE == kRotate;  // cosines and sines in registers
    using R = Ring<T, LAYOUT, LPR>;
    constexpr uint32_t kRow = R::kSlotBytes * (MODE == kNormBwd ? 2 : 1);  // x, and the gradient behind it
    // For each warp its ring; behind them its table of cosines and sines.
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x % LPR, warp = threadIdx.x / 32, in_warp = threadIdx.x % 32, group = in_warp / LPR;
    unsigned char* const ring = smem + warp * D * kRow;
    const int which = blockIdx.x >= a.ctas0;
    const uint32_t cta = blockIdx.x - (which ? a.ctas0 : 0), ctas = which ? gridDim.x - a.ctas0 : a.ctas0;
    const HeadsView vx = a.x[which], vg = a.g[which], vy = a.y[which];
    const T* x = static_cast<const T*>(vx.p);
    const T* gy = static_cast<const T*>(vg.p);
    T* y = static_cast<T*>(const_cast<void*>(vy.p));
    const int shift = a.tok_shift[which], unit_shift = shift + a.sub_shift[which];
    const int turn_shift = unit_shift + __popc(LPR - 1);
    const int split = a.split_shift[which], heads = a.heads[which], iters = a.iters[which];
    const int side = GW >> shift, head_step = side << split, my_token = group & ((1 << shift) - 1);
    const bool skip_rest = a.skip_rest[which];
    const LanePlace<T, LAYOUT, LPR> place(lane, a);
    float* const table = reinterpret_cast<float*>(smem + kHeadsWarps * D * kRow) + (warp << unit_shift) * (LPR * 2 * kVec);
    if constexpr (R::kOwn)
#pragma unroll
        for (uint32_t at = 0; at < D * kRow; at += R::kSlotBytes) R::clear(ring + at, place);
    pdl_enter();

    Pairs sum = {};  // of the weights' gradients
    __shared__ float4 ws[MODE != kRotate ? kHalfVec : 1][LPR];
    if constexpr (MODE != kRotate) {
        const T* pw = static_cast<const T*>(a.w[which]);
        Pairs w;
        if (pw) {
            RowRaw<T, LAYOUT> r;
#pragma unroll
            for (int j = 0; j < r.J; ++j) {
                bool ta, tb;
                const int ea = place.first(j, ta), eb = place.second(j, tb);
                r.a[j] = ta ? load_chunk<T, r.W>(pw + ea) : Chunk<T, r.W>{};
                r.b[j] = tb ? load_chunk<T, r.W>(pw + eb) : Chunk<T, r.W>{};
            }
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

    const float sine_scale = a.scale * a.sign;
    const int seq = static_cast<int>(a.by_seq.d), table_tokens = a.pairs ? 1 << unit_shift : 0;
    const int first_k = static_cast<int>(fdiv(in_warp, a.by_pairs)), first_f = in_warp - first_k * a.pairs;
    const int step_k = static_cast<int>(fdiv(32, a.by_pairs)), step_f = 32 - step_k * a.pairs;
    for (uint32_t unit = cta * kHeadsWarps + warp; unit < a.units[which]; unit += ctas * kHeadsWarps) {
        const int t0 = static_cast<int>(unit >> split) << unit_shift;
        const int head0 = (group >> shift) + side * static_cast<int>(unit & ((1u << split) - 1));
        // The rows of a group: heads head0, head0 + head_step, .. of token t0 + my_token, then of the one 2^shift
        // further on.  Two places in them: of the row to be loaded next, and of the one to be stored next.
        const T *px, *pg;
        T* py;
        int load_t = t0 + my_token, load_head = head0, to_load = iters << a.sub_shift[which];
        int t = load_t, head = head0, to_store = to_load, load_i = iters, store_i = iters;
        bool load_on, on;
        auto open_load = [&] {
            load_on = load_t < a.tokens;
            const int64_t b = fdiv(load_on ? load_t : 0, a.by_seq), l = fmod_(load_on ? load_t : 0, a.by_seq);
            px = x + (b * vx.bs + l * vx.ss + head0 * vx.hs);
            if constexpr (MODE == kNormBwd) pg = gy + (b * vg.bs + l * vg.ss + head0 * vg.hs);
        };
        auto open_store = [&] {
            on = t < a.tokens;
            const int64_t b = fdiv(on ? t : 0, a.by_seq), l = fmod_(on ? t : 0, a.by_seq);
            py = y + (b * vy.bs + l * vy.ss + head0 * vy.hs);
        };
        // Rows on their way; each goes into the slot of one that has been used.
        uint32_t load_slot = 0, slot = 0;
        auto load = [&] {
            if (to_load > 0) {
                --to_load;
                if (load_on && load_head < heads) {
                    R::load(ring + load_slot, px, place);
                    if constexpr (MODE == kNormBwd) R::load(ring + load_slot + R::kSlotBytes, pg, place);
                }
                load_head += head_step;
                px += head_step * vx.hs;
                if constexpr (MODE == kNormBwd) pg += head_step * vg.hs;
                if (--load_i == 0 && to_load > 0) {
                    load_i = iters;
                    load_head = head0;
                    load_t += 1 << shift;
                    open_load();
                }
                load_slot = load_slot + kRow == D * kRow ? 0 : load_slot + kRow;
            }
            copies_commit();
        };
        open_load();
        open_store();
#pragma unroll
        for (int u = 0; u < D; ++u) load();
        __syncwarp();  // the table's readers are done
        // pair f of token k, and 32 pairs on
        const int l0 = static_cast<int>(fmod_(t0, a.by_seq));
        for (int k = first_k, f = first_f; k < table_tokens;) {
            int32_t at;
            if (a.positions) {
                at = a.positions[min(t0 + k, a.tokens - 1)];
            } else {
                const int l = l0 + k;
                at = a.first + (l < seq ? l : static_cast<int>(fmod_(l, a.by_seq)));
            }
            float s, c;
            turn_sincos(a.turns[f], at, s, c);
            float* e = table + table_place<T, LAYOUT, LPR>(k, f, unit_shift);
            e[0] = c * a.scale;
            e[2] = s * sine_scale;
            f += step_f;
            k += step_k;
            if (f >= a.pairs) {
                f -= a.pairs;
                ++k;
            }
        }
        __syncwarp();
        const float4* turns = reinterpret_cast<const float4*>(table) + my_token * LPR + lane;  // its tokens' j'th at j << turn_shift
        float4 cs[kCsRegs ? kHalfVec : 1];
        auto take_turns = [&] {
            if constexpr (kCsRegs)
#pragma unroll
                for (int j = 0; j < kHalfVec; ++j) cs[j] = turns[j << turn_shift];
        };
        take_turns();
        auto turn = [&](Pairs& p) {
            if (place.rot == 0) return;
            const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
            for (int j = 0; j < kHalfVec; ++j) {
                const float4 q = kCsRegs ? cs[kCsRegs ? j : 0] : turns[j << turn_shift];
                const float2 c = make_float2(q.x, q.y), s = make_float2(q.z, q.w);
                const float2 u = fma2(mul2(p.y[j], s), minus, mul2(p.x[j], c)), v = fma2(p.x[j], s, mul2(p.y[j], c));
                if ((MODE == kRotate && sizeof(T) == 2) || place.rot == 0xffu) {  // the former stores the others as it read them
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
        while (to_store > 0) {
            --to_store;
            const bool there = on && head < heads;
            copies_wait<D - 1>();
            if constexpr (!R::kOwn) __syncwarp();
            const RowRaw<T, LAYOUT> raw = R::read(ring + slot, place);
            Pairs p = pairs_of<T, LAYOUT>(raw), g;
            if constexpr (MODE == kNormBwd) g = pairs_of<T, LAYOUT>(R::read(ring + slot + R::kSlotBytes, place));
            if constexpr (R::kOwn) load();
            if constexpr (MODE != kRotate) {
                float2 q = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < kHalfVec; ++j) q = fma2(p.x[j], p.x[j], fma2(p.y[j], p.y[j], q));
                // a lane's part of the mean, and not of the sum, which leaves FP32 before the mean does
                const float r = rsqrtf(group_sum<LPR>((q.x + q.y) * a.inv_dim) + a.eps);
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
            R::store(ring + slot, py, p, raw, there, MODE == kRotate, skip_rest, 2 * a.pairs, place);
            if constexpr (!R::kOwn) load();
            slot = slot + kRow == D * kRow ? 0 : slot + kRow;
            head += head_step;
            py += head_step * vy.hs;
            if (--store_i == 0 && to_store > 0) {
                store_i = iters;
                head = head0;
                t += 1 << shift;
                open_store();
                turns += LPR << shift;
                take_turns();
            }
        }
    }
    if constexpr (MODE == kNormBwd) {
        if (!a.partial) return;
        // the groups' sums, in the row's order, added in the groups' order
        __syncthreads();  // the rings are free
        float* const sums = reinterpret_cast<float*>(smem);
        float* mine = sums + (warp * GW + group) * a.dim;
        float u[kVec], v[kVec];
        chunks_of<LAYOUT>(sum, u, v);
#pragma unroll
        for (int j = 0; j < RowRaw<T, LAYOUT>::J; ++j) {
            constexpr int W = RowRaw<T, LAYOUT>::W;
            bool ta, tb;
            const int ea = place.first(j, ta), eb = place.second(j, tb);
#pragma unroll
            for (int k = 0; k < W; ++k) {
                if (ta) mine[ea + k] = u[j * W + k];
                if (tb) mine[eb + k] = v[j * W + k];
            }
        }
        __syncthreads();
        for (int j = threadIdx.x; j < a.dim; j += kHeadsThreads) {
            float total = 0.f;
            for (int k = 0; k < G; ++k) total += sums[k * a.dim + j];
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
#pragma unroll 10
        for (int k = begin; k < end; ++k) sum += partial[static_cast<int64_t>(first + k) * dim + j];
    part[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y == 0 && j < dim) {
        for (int k = 1; k < 32; ++k) sum += part[k][threadIdx.x];
        dw[j] = from_f32<T>(sum);
    }
}

template <typename T, int LAYOUT, int LPR, int MODE>
cudaError_t launch_kernel(const HeadsArgs& a, int ctas, cudaStream_t s) {
    static int done[kMaxDevices];
    const cudaError_t e = allow_max_dynamic_smem(heads_kernel<T, LAYOUT, LPR, MODE>, done);
    if (e != cudaSuccess) return e;
    const int tokens = 1 << std::max(a.tok_shift[0] + a.sub_shift[0], a.tok_shift[1] + a.sub_shift[1]);
    const size_t row = Ring<T, LAYOUT, LPR>::kSlotBytes * (MODE == kNormBwd ? 2 : 1);
    const size_t smem = kHeadsWarps * (ring_slots<T, MODE>() * row + static_cast<size_t>(tokens) * LPR * kVec * 8);
    return launch_pdl(heads_kernel<T, LAYOUT, LPR, MODE>, dim3(static_cast<unsigned>(ctas)), dim3(kHeadsThreads), smem, s, a);
}

template <typename T, int LAYOUT, int LPR>
cudaError_t launch_mode(const HeadsArgs& a, const HeadsCall& c, int ctas, cudaStream_t s) {
    if (!c.norm) return launch_kernel<T, LAYOUT, LPR, kRotate>(a, ctas, s);
    if (!c.backward) return launch_kernel<T, LAYOUT, LPR, kNormFwd>(a, ctas, s);
    return launch_kernel<T, LAYOUT, LPR, kNormBwd>(a, ctas, s);
}

template <typename T, int LAYOUT>
cudaError_t launch_width(int lpr, const HeadsArgs& a, const HeadsCall& c, int ctas, cudaStream_t s) {
    if (lpr == 1) return launch_mode<T, LAYOUT, 1>(a, c, ctas, s);
    if (lpr == 2) return launch_mode<T, LAYOUT, 2>(a, c, ctas, s);
    if (lpr == 4) return launch_mode<T, LAYOUT, 4>(a, c, ctas, s);
    if (lpr == 8) return launch_mode<T, LAYOUT, 8>(a, c, ctas, s);
    if (lpr == 16) return launch_mode<T, LAYOUT, 16>(a, c, ctas, s);
    return launch_mode<T, LAYOUT, 32>(a, c, ctas, s);
}

template <typename T> cudaError_t launch_halves(int width, int lpr, const HeadsArgs& a, const HeadsCall& c, int ctas, cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (width == 8) return launch_width<T, 8>(lpr, a, c, ctas, s);
    return launch_width<T, 4>(lpr, a, c, ctas, s);
}

HeadsView view_of(const ls_head_view* v) {
    return v ? HeadsView{v->data, v->batch_stride, v->seq_stride, v->head_stride} : HeadsView{nullptr, 0, 0, 0};
}

// A unit's tokens, and the units that share their heads.  The groups that share a token go through its heads
// side by side: few of them leave each more heads to use its cosines on, many end sooner; heads that are few leave
// room for more tokens one after the other.  Counted in rounds of the warps that the GPU holds (`slots` of them are
// this tensor's): a unit takes as long as three rows, a row counting 2, and what its rows and its angles take.
void plan_units(HeadsArgs& a, int which, int log_groups, uint32_t slots) {
    int64_t best = INT64_MAX;
    for (int split = 0; split <= 5; ++split)
        for (int shift = 0; shift <= log_groups; ++shift)
            for (int sub = 0; sub <= kMostSub; ++sub) {
                const int steps = log_groups - shift + split;  // log2 of the heads that are side by side
                if (split > 0 && (sub > 0 || 1 << steps >= 2 * a.heads[which])) continue;
                const int64_t iters = (a.heads[which] + (1 << steps) - 1) >> steps;
                const int64_t units = ((static_cast<int64_t>(a.tokens) + (1 << (shift + sub)) - 1) >> (shift + sub)) << split;
                const int64_t angles = ((static_cast<int64_t>(a.pairs) << (shift + sub)) + 31) / 32;
                if (units > int64_t{1} << 30) continue;
                // 32 bits: a division for each candidate is what this costs the host
                const int64_t rounds = (static_cast<uint32_t>(units) + slots - 1) / slots;
                const int64_t t = rounds * (2 * (iters << sub) + angles + 3);
                if (t > best || (t == best && split > a.split_shift[which])) continue;
                best = t;
                a.tok_shift[which] = shift;
                a.sub_shift[which] = sub;
                a.split_shift[which] = split;
                a.iters[which] = static_cast<int>(iters);
                a.units[which] = static_cast<uint32_t>(units);
            }
}

}  // namespace

template <typename T> cudaError_t launch_heads(const HeadsCall& c, cudaStream_t s) {
    HeadsArgs a = {};
    a.tokens = static_cast<int>(c.batch * c.seq);
    a.by_seq = make_fastdiv(static_cast<uint32_t>(std::max<int64_t>(c.seq, 1)));
    a.dim = static_cast<int>(c.dim);
    a.eps = c.eps;
    a.inv_dim = 1.f / static_cast<float>(a.dim);
    a.sign = c.backward ? -1.f : 1.f;
    a.scale = 1.f;
    if (const ls_rotation* r = c.rotation) {
        a.pairs = static_cast<int>(r->rotary_dim / 2);
        a.turns = r->turns;
        a.positions = r->positions;
        a.first = static_cast<int32_t>(r->first_position);
        a.scale = r->scale;
    }
    a.by_pairs = make_fastdiv(static_cast<uint32_t>(std::max(a.pairs, 1)));
    int layout = 16 / sizeof(T);
    if (c.rotation && c.rotation->interleaved) layout = kInterleaved;
    while (layout > 1 && a.pairs % layout) layout /= 2;
    int lpr = 1, log_groups = 5;  // log2 of a warp's groups
    for (; 2 * kVec * lpr < a.dim; --log_groups) lpr *= 2;
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
        plan_units(a, k, log_groups, static_cast<uint32_t>(std::max<int64_t>(1, 152 * 16 * rows[k] / (rows[0] + rows[1]))));
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
        e = layout == kInterleaved ? launch_width<T, kInterleaved>(lpr, a, c, all, s)
            : layout >= 4          ? launch_halves<T>(layout, lpr, a, c, all, s)
            : layout == 2          ? launch_width<T, 2>(lpr, a, c, all, s)
                                   : launch_width<T, 1>(lpr, a, c, all, s);
    }
    if (e != cudaSuccess || !partial) return e;
    // zeros for a tensor without rows
    return launch_pdl(heads_dweight_kernel<T>, dim3(static_cast<unsigned>((c.dim + 31) / 32), 2), dim3(32, 32), 0, s,
                      static_cast<T*>(c.dweight[0]), static_cast<T*>(c.dweight[1]), static_cast<const float*>(a.partial), a.dim,
                      a.ctas0, all);
}

}  // namespace ls
