// block_internal.h -- launchers behind the C ABI of ls_block.h.  Arguments
// reaching them have been validated by block_api.cu; grids, workspace layouts
// and the order of every sum depend on the shapes alone.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ls_block.h"

namespace ls {

constexpr int64_t kMaxHeadDim = 512;
constexpr int64_t kMaxGatedRows = int64_t{1} << 24;
constexpr int64_t kMaxGatedCols = 65536;

// Rotation and norm of up to two tensors of heads (heads.cuh).
struct HeadsCall {
    const ls_head_view* x[2];  // forward: the inputs; norm's backward: the forward's inputs
    const ls_head_view* g[2];  // norm's backward: the outputs' gradients
    const ls_head_view* y[2];  // outputs
    const void* weight[2];
    void* dweight[2];
    bool norm, backward;
    int64_t batch, seq, dim;
    const ls_rotation* rotation;  // nullable
    float eps;
    void* workspace;
};
constexpr int kPartialCtas = 608;  // CTAs that hold sums of the weights' gradients: four on each of 152 SMs
inline size_t heads_workspace_bytes(int64_t dim) { return static_cast<size_t>(kPartialCtas * dim) * sizeof(float); }
template <typename T> cudaError_t launch_heads(const HeadsCall& c, cudaStream_t s);
cudaError_t launch_heads_dtype(ls_dtype dt, const HeadsCall& c, cudaStream_t s);

// Many gradients (clip.cu).
size_t grad_norm_workspace_bytes();
cudaError_t launch_grad_norm(float* norm, float* factor, const ls_tensor* grads, int64_t count,
                             float max_norm, float grad_scale, void* workspace, cudaStream_t s);
cudaError_t launch_scale_gradients(const ls_tensor* out, const ls_tensor* in, int64_t count,
                                   const float* factor, cudaStream_t s);
struct AdamScaled {
    float lr, beta1, beta2, eps, weight_decay;
    int64_t step;
    const float* factor;
    const float* norm;  // nullable
};
cudaError_t launch_adam_scaled(ls_dtype dt, void* param, const void* grad, float* m, float* v,
                               int64_t n, const AdamScaled& h, cudaStream_t s);

// The gated block (gated.cu).
struct GatedShape {
    int64_t rows, hidden, ffn;
    ls_activation act;
};
// How the gradients' sums are cut, and the workspace's layout; made once for a call.
struct GatedPlan {
    int64_t width;                     // of dx's and dW's tiles
    int64_t slices, slice_blocks;      // of dx's K
    int64_t w_slices, w_slice_blocks;  // of the rows, for dW
    int64_t x_len;                     // what a unit of dx takes
    bool w_first;
    bool pairs;                        // dg and du as two numbers each
    size_t du, partial, w_partial, bytes;
};
GatedPlan gated_plan(int64_t rows, int64_t hidden, int64_t ffn);
cudaError_t launch_gated_fwd(ls_dtype dt, void* h, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, cudaStream_t s);
cudaError_t launch_gated_bwd(ls_dtype dt, void* dx, void* dwg, void* dwu, bool f32_dweight,
                             const void* dh, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, const GatedPlan& plan, void* workspace, cudaStream_t s);
// Few rows (gated_few.cu): whether these sizes are its own; h, or with dh dg (in h's place) and du, with the rest of
// their rounding in dg_low and du_low unless these are NULL.
bool gated_few_rows(int64_t rows, int64_t hidden, int64_t ffn);
cudaError_t launch_gated_few(ls_dtype dt, void* h, void* du, const void* dh, const void* x, const void* wg, const void* wu,
                             const GatedShape& sh, void* dg_low, void* du_low, cudaStream_t s);
cudaError_t launch_block_wait_selftest(uint32_t polls, cudaStream_t s);
cudaError_t gated_take_device_error(unsigned int* flags);

}  // namespace ls
