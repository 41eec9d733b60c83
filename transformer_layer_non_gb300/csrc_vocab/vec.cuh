// vec.cuh -- BF16 instances of the 8-element vectors of ls_device.cuh.
#pragma once

#include <cuda_bf16.h>

#include "../csrc/ls_device.cuh"

namespace ls {

using bf16 = __nv_bfloat16;

template <> struct Raw8<bf16> { uint4 v; };

template <> __device__ __forceinline__ Raw8<bf16> load8<bf16>(const bf16* p) {
    return Raw8<bf16>{ld16(p)};
}
template <> __device__ __forceinline__ void store8<bf16>(bf16* p, const Raw8<bf16>& r) {
    st16(p, r.v);
}
// A BF16 value is the upper half of the FP32 value: widening is a shift.
__device__ __forceinline__ float2 b2f(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ uint32_t f2b(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);  // round to nearest even
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void unpack(const Raw8<bf16>& r, float (&f)[8]) {
    float2 t;
    t = b2f(r.v.x); f[0] = t.x; f[1] = t.y;
    t = b2f(r.v.y); f[2] = t.x; f[3] = t.y;
    t = b2f(r.v.z); f[4] = t.x; f[5] = t.y;
    t = b2f(r.v.w); f[6] = t.x; f[7] = t.y;
}
template <> __device__ __forceinline__ Raw8<bf16> pack<bf16>(const float (&f)[8]) {
    return Raw8<bf16>{make_uint4(f2b(f[0], f[1]), f2b(f[2], f[3]), f2b(f[4], f[5]),
                                 f2b(f[6], f[7]))};
}
template <> __device__ __forceinline__ Raw8<bf16> zero8<bf16>() {
    return Raw8<bf16>{make_uint4(0, 0, 0, 0)};
}
// Element-wise maximum of two vectors.
__device__ __forceinline__ uint32_t hmax2u(uint32_t a, uint32_t b) {
    const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t bmax2u(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m =
        __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ Raw8<__half> vmax(const Raw8<__half>& a, const Raw8<__half>& b) {
    return Raw8<__half>{make_uint4(hmax2u(a.v.x, b.v.x), hmax2u(a.v.y, b.v.y),
                                   hmax2u(a.v.z, b.v.z), hmax2u(a.v.w, b.v.w))};
}
__device__ __forceinline__ Raw8<bf16> vmax(const Raw8<bf16>& a, const Raw8<bf16>& b) {
    return Raw8<bf16>{make_uint4(bmax2u(a.v.x, b.v.x), bmax2u(a.v.y, b.v.y),
                                 bmax2u(a.v.z, b.v.z), bmax2u(a.v.w, b.v.w))};
}
__device__ __forceinline__ Raw8<float> vmax(const Raw8<float>& a, const Raw8<float>& b) {
    return Raw8<float>{make_float4(fmaxf(a.a.x, b.a.x), fmaxf(a.a.y, b.a.y), fmaxf(a.a.z, b.a.z),
                                   fmaxf(a.a.w, b.a.w)),
                       make_float4(fmaxf(a.b.x, b.b.x), fmaxf(a.b.y, b.b.y), fmaxf(a.b.z, b.b.z),
                                   fmaxf(a.b.w, b.b.w))};
}
__device__ __forceinline__ float vmax8(const Raw8<bf16>& r) {
    const float2 m = b2f(bmax2u(bmax2u(r.v.x, r.v.y), bmax2u(r.v.z, r.v.w)));
    return fmaxf(m.x, m.y);
}
// A vector of -inf.
template <typename T> __device__ __forceinline__ Raw8<T> lowest8();
template <> __device__ __forceinline__ Raw8<__half> lowest8<__half>() {
    return Raw8<__half>{make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u)};
}
template <> __device__ __forceinline__ Raw8<bf16> lowest8<bf16>() {
    return Raw8<bf16>{make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)};
}
template <> __device__ __forceinline__ Raw8<float> lowest8<float>() {
    const float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    return Raw8<float>{f, f};
}

// launch_pdl with thread-block clusters of `cluster` CTAs along x.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_cluster(void (*kernel)(KArgs...), dim3 grid, int cluster, dim3 block, size_t smem,
                                  cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
}
// Address, in the cluster's shared-memory window, of CTA `rank`'s copy of a variable.
__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// Two values to one 32-bit word of the 16-bit storage type.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) { return f2h(a, b); }
template <> __device__ __forceinline__ uint32_t pack2<bf16>(float a, float b) { return f2b(a, b); }

// One value of the storage type.
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace ls
