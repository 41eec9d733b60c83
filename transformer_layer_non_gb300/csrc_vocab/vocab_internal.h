// vocab_internal.h -- launchers behind the C ABI of ls_vocab.h.  Arguments
// reaching them have been validated by vocab_api.cu; workspace layouts and
// piece sizes depend on the shapes alone.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ls_vocab.h"

namespace ls {

constexpr int64_t kMaxHeadRows = int64_t{1} << 24;
constexpr int64_t kMaxHeadHidden = 65536;
constexpr int64_t kMaxVocab = int64_t{1} << 30;
constexpr int64_t kMaxLookupTokens = int64_t{1} << 30;
constexpr int64_t kMaxTeacherEntries = 1024;

struct HeadShape {
    int64_t rows, hidden, vocab;
    float eps;
    int32_t ignore_index;
};
size_t linear_ce_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab);
size_t linear_ce_fwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab);
cudaError_t launch_linear_ce_fwd(ls_dtype dt, float* loss, float* lse, const void* x,
                                 const void* weight, const int32_t* target, const HeadShape& sh,
                                 void* workspace, cudaStream_t s);
// f32_dweight: dweight is FP32 and added to; otherwise it has the storage dtype and is written.
cudaError_t launch_linear_ce_bwd(ls_dtype dt, void* dx, void* dweight, bool f32_dweight,
                                 const void* x, const void* weight, const int32_t* target,
                                 const float* lse, const float* dloss, const HeadShape& sh,
                                 void* workspace, cudaStream_t s);
cudaError_t launch_vocab_wait_selftest(uint32_t polls, cudaStream_t s);
cudaError_t linear_ce_take_device_error(unsigned int* flags);

struct DistillShape {
    int64_t rows, vocab;
    int k;
    float tau;
};
cudaError_t launch_distill_fwd(ls_dtype dt, float* loss, float* lse, const void* logits,
                               const int32_t* index, const void* teacher, const float* teacher_lse,
                               const DistillShape& sh, cudaStream_t s);
cudaError_t launch_distill_bwd(ls_dtype dt, void* dlogits, const void* logits,
                               const int32_t* index, const void* teacher, const float* lse,
                               const float* teacher_lse, const float* dloss,
                               const DistillShape& sh, cudaStream_t s);

size_t embedding_lookup_workspace_bytes(int64_t tokens, int64_t hidden, int64_t vocab);
cudaError_t launch_embedding_lookup_fwd(ls_dtype dt, void* y, const int32_t* tokens,
                                        const void* table, int64_t n, int64_t hidden,
                                        int64_t vocab, float scale, cudaStream_t s);
cudaError_t launch_embedding_lookup_bwd(ls_dtype dt, float* d_table, const void* dy,
                                        const int32_t* tokens, int64_t n, int64_t hidden,
                                        int64_t vocab, float scale, int32_t padding_id,
                                        bool accumulate, void* workspace, cudaStream_t s);

}  // namespace ls
