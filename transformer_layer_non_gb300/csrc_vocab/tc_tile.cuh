// tc_tile.cuh -- what the kernels that multiply in tiles of a pair of CTAs
// share: bounded waits, the way from accumulators to store boxes, and, on the
// host, tensor maps.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "tc.cuh"

namespace ls {
namespace {

// Bounded wait of a converged warp; false (and the failure flagged for the CTA
// and the host) when it runs out.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead,
                                         uint32_t polls = kWaitPolls) {
    for (uint32_t i = 0; i < polls; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((i & 63) == 63 && __any_sync(0xffffffffu, *dead)) return false;
    }
    flag_device_error(kDevErrWaitTimeout);
    *dead = 1;
    return false;
}

// 16 bytes `c` of a lane's 128-byte row in a swizzled store box.
__device__ __forceinline__ void put16(unsigned char* box, int lane, int c, uint4 v) {
    st16(box + lane * 128 + ((c ^ (lane & 7)) << 4), v);
}

template <typename T> __device__ __forceinline__ uint4 pack8(const float (&z)[32], int j, float sc) {
    return make_uint4(pack2<T>(z[j] * sc, z[j + 1] * sc), pack2<T>(z[j + 2] * sc, z[j + 3] * sc),
                      pack2<T>(z[j + 4] * sc, z[j + 5] * sc), pack2<T>(z[j + 6] * sc, z[j + 7] * sc));
}

// f(c, z) for the warp's four groups of 32 accumulator columns, the next group
// on its way while f works; release() once all of them are in registers.
template <typename R, typename F>
__device__ __forceinline__ void sweep(uint32_t cols, R&& release, F&& f) {
    float za[32], zb[32];
    tmem_ld32(za, cols);
    tmem_ld_wait(za);
    tmem_ld32(zb, cols + 32);
    f(0, za);
    tmem_ld_wait(zb);
    tmem_ld32(za, cols + 64);
    f(1, zb);
    tmem_ld_wait(za);
    tmem_ld32(zb, cols + 96);
    f(2, za);
    tmem_ld_wait(zb);
    release();
    f(3, zb);
}

// --- host ----------------------------------------------------------------------
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t n) { return (n + 255) / 256 * 256; }

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                               cudaEnableDefault, &r);
        return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeFn>(p) : nullptr;
    }();
    return fn;
}

// A row-major [depth][outer][inner] tensor in boxes of [1][box_outer][128 bytes].
template <typename E>
cudaError_t make_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int64_t ld, int box_outer,
                     int64_t depth = 0) {
    const EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const CUtensorMapDataType type = std::is_same<E, float>::value  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : std::is_same<E, bf16>::value ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const cuuint64_t size = sizeof(E);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer),
                                static_cast<cuuint64_t>(depth)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * size,
                                   static_cast<cuuint64_t>(ld) * static_cast<cuuint64_t>(outer) * size};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), static_cast<cuuint32_t>(box_outer), 1};
    const cuuint32_t one[3] = {1, 1, 1};
    const CUresult r = fn(map, type, depth ? 3 : 2, const_cast<void*>(base), dims, strides, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

#define LS_CUDA(expr)                        \
    do {                                     \
        const cudaError_t _e = (expr);       \
        if (_e != cudaSuccess) return _e;    \
    } while (0)

}  // namespace
}  // namespace ls
