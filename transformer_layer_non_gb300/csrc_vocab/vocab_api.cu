// vocab_api.cu -- the C ABI declared in include/ls_vocab.h: every entry point
// checks its arguments on the host, before anything is enqueued, and hands
// the call to a launcher of vocab_internal.h.  Nothing here allocates,
// synchronises (ls_vocab_check_device_errors apart) or keeps state but the
// per-thread message of the last error.
#include <math.h>

#include "host_check.h"
#include "vocab_internal.h"

namespace {

ls_status check_head(const char* fn, ls_dtype dt, int64_t rows, int64_t hidden, int64_t vocab,
                     float eps) {
    LS_TRY(check_storage(fn, dt, false));
    LS_TRY(check_size(fn, "rows", rows, 0, ls::kMaxHeadRows));
    LS_TRY(check_size(fn, "hidden", hidden, 1, ls::kMaxHeadHidden));
    LS_TRY(check_multiple_of_8(fn, "hidden", hidden));
    LS_TRY(check_size(fn, "vocab", vocab, 1, ls::kMaxVocab));
    if (rows * vocab > (int64_t{1} << 46) || vocab * hidden > (int64_t{1} << 40))
        return fail(LS_ERR_UNSUPPORTED_SHAPE, "%s: %lld rows of %lld logits too large", fn,
                    (long long)rows, (long long)vocab);
    if (!(eps >= 0.f && eps < 1.f))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: label_smoothing = %g is not in [0, 1)", fn,
                    static_cast<double>(eps));
    return LS_OK;
}

ls_status check_distill(const char* fn, ls_dtype dt, int64_t rows, int64_t vocab, int64_t k,
                        float tau) {
    LS_TRY(check_storage(fn, dt, true));
    LS_TRY(check_size(fn, "rows", rows, 0, int64_t{INT32_MAX}));
    LS_TRY(check_size(fn, "vocab", vocab, 1, ls::kMaxVocab));
    LS_TRY(check_multiple_of_8(fn, "vocab", vocab));
    LS_TRY(check_size(fn, "k", k, 1, ls::kMaxTeacherEntries));
    if (!(tau >= 0x1p-60f && tau <= 0x1p60f))  // 1/tau and tau^2 are FP32 factors
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: temperature = %g is not in [2^-60, 2^60]", fn,
                    static_cast<double>(tau));
    return LS_OK;
}

ls_status check_lookup(const char* fn, ls_dtype dt, int64_t n, int64_t hidden, int64_t vocab,
                       float scale) {
    LS_TRY(check_storage(fn, dt, true));
    LS_TRY(check_size(fn, "tokens_count", n, 0, ls::kMaxLookupTokens));
    LS_TRY(check_size(fn, "hidden", hidden, 1, ls::kMaxHeadHidden));
    LS_TRY(check_multiple_of_8(fn, "hidden", hidden));
    LS_TRY(check_size(fn, "vocab", vocab, 0, ls::kMaxVocab));
    if (n * hidden > (int64_t{1} << 40) || vocab * hidden > (int64_t{1} << 40))
        return fail(LS_ERR_UNSUPPORTED_SHAPE, "%s: too many elements", fn);
    if (!isfinite(scale)) return fail(LS_ERR_INVALID_ARGUMENT, "%s: scale is not finite", fn);
    return LS_OK;
}

}  // namespace

#pragma GCC visibility push(default)
extern "C" {

const char* ls_vocab_last_error(void) { return g_last_error; }

ls_status ls_vocab_check_device_errors(uint32_t* flags) {
    if (!flags) return fail(LS_ERR_INVALID_ARGUMENT, "flags is NULL");
    *flags = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return from_cuda(e, "ls_vocab_check_device_errors: synchronise");
    unsigned int v = 0;
    e = ls::linear_ce_take_device_error(&v);
    if (e != cudaSuccess) return from_cuda(e, "ls_vocab_check_device_errors: read flags");
    *flags = v;
    return ok();
}

ls_status ls_vocab_selftest_wait_timeout(uint32_t polls, void* stream) {
    if (polls == 0 || polls > (1u << 19))
        return fail(LS_ERR_INVALID_ARGUMENT, "polls = %u is not in [1, 2^19]", polls);
    return from_cuda(ls::launch_vocab_wait_selftest(polls, as_stream(stream)),
                     "ls_vocab_selftest_wait_timeout");
}

static bool head_sizes(int64_t rows, int64_t hidden, int64_t vocab) {
    return rows > 0 && rows <= ls::kMaxHeadRows && hidden > 0 && hidden <= ls::kMaxHeadHidden &&
           hidden % 8 == 0 && vocab > 0 && vocab <= ls::kMaxVocab;
}

size_t ls_linear_cross_entropy_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab) {
    return head_sizes(rows, hidden, vocab) ? ls::linear_ce_workspace_bytes(rows, hidden, vocab) : 0;
}

size_t ls_linear_cross_entropy_fwd_workspace_bytes(int64_t rows, int64_t hidden, int64_t vocab) {
    return head_sizes(rows, hidden, vocab) ? ls::linear_ce_fwd_workspace_bytes(rows, hidden, vocab)
                                           : 0;
}

ls_status ls_linear_cross_entropy_fwd(ls_dtype dtype, float* loss, float* lse, const void* x,
                                      const void* weight, const int32_t* target, int64_t rows,
                                      int64_t hidden, int64_t vocab, float label_smoothing,
                                      int32_t ignore_index, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    const char* fn = "ls_linear_cross_entropy_fwd";
    LS_TRY(check_head(fn, dtype, rows, hidden, vocab, label_smoothing));
    if (rows == 0) return ok();
    LS_TRY(check_ptr4(loss, "loss", true));
    LS_TRY(check_ptr4(lse, "lse", false));
    LS_TRY(check_ptr(x, "x", true));
    LS_TRY(check_ptr(weight, "weight", true));
    LS_TRY(check_ptr4(target, "target", true));
    const size_t need = ls::linear_ce_fwd_workspace_bytes(rows, hidden, vocab);
    LS_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    const size_t rb = static_cast<size_t>(rows) * 4;
    const Span outs[] = {{"loss", loss, rb}, {"lse", lse, rb}, {"workspace", workspace, need}};
    const Span ins[] = {{"x", x, static_cast<size_t>(rows * hidden) * 2},
                        {"weight", weight, static_cast<size_t>(vocab * hidden) * 2},
                        {"target", target, rb}};
    LS_TRY(check_disjoint(outs, 3, ins, 3));
    const ls::HeadShape sh{rows, hidden, vocab, label_smoothing, ignore_index};
    return from_cuda(ls::launch_linear_ce_fwd(dtype, loss, lse, x, weight, target, sh, workspace,
                                              as_stream(stream)),
                     fn);
}

ls_status ls_linear_cross_entropy_bwd(ls_dtype dtype, void* dx, void* dweight,
                                      ls_dtype dweight_dtype, const void* x, const void* weight,
                                      const int32_t* target, const float* lse, const float* dloss,
                                      int64_t rows, int64_t hidden, int64_t vocab,
                                      float label_smoothing, int32_t ignore_index,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "ls_linear_cross_entropy_bwd";
    LS_TRY(check_head(fn, dtype, rows, hidden, vocab, label_smoothing));
    const bool f32 = dweight_dtype == LS_F32;
    if (!f32 && dweight_dtype != dtype)
        return fail(LS_ERR_INVALID_ARGUMENT,
                    "%s: dweight_dtype = %d is neither the storage dtype nor LS_F32", fn,
                    static_cast<int>(dweight_dtype));
    LS_TRY(check_ptr(dx, "dx", false));
    LS_TRY(check_ptr(dweight, "dweight", false));
    if (rows > 0 && !dx && !dweight)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: dx and dweight are both NULL", fn);
    const size_t wb = static_cast<size_t>(vocab * hidden) * elem_size(dweight_dtype);
    if (rows == 0) {
        if (!dweight || f32) return ok();
        return from_cuda(cudaMemsetAsync(dweight, 0, wb, as_stream(stream)), fn);
    }
    LS_TRY(check_ptr(x, "x", true));
    LS_TRY(check_ptr(weight, "weight", true));
    LS_TRY(check_ptr4(target, "target", true));
    LS_TRY(check_ptr4(lse, "lse", true));
    LS_TRY(check_ptr4(dloss, "dloss", false));
    const size_t need = ls::linear_ce_workspace_bytes(rows, hidden, vocab);
    LS_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    const size_t rb = static_cast<size_t>(rows) * 4, xb = static_cast<size_t>(rows * hidden) * 2;
    const Span outs[] = {{"dx", dx, xb}, {"dweight", dweight, wb}, {"workspace", workspace, need}};
    const Span ins[] = {{"x", x, xb},
                        {"weight", weight, static_cast<size_t>(vocab * hidden) * 2},
                        {"target", target, rb},
                        {"lse", lse, rb},
                        {"dloss", dloss, rb}};
    LS_TRY(check_disjoint(outs, 3, ins, 5));
    const ls::HeadShape sh{rows, hidden, vocab, label_smoothing, ignore_index};
    return from_cuda(ls::launch_linear_ce_bwd(dtype, dx, dweight, f32, x, weight, target, lse,
                                              dloss, sh, workspace, as_stream(stream)),
                     fn);
}

ls_status ls_distill_topk_fwd(ls_dtype dtype, float* loss, float* lse, const void* logits,
                              const int32_t* teacher_index, const void* teacher_logits,
                              const float* teacher_lse, int64_t rows, int64_t vocab, int64_t k,
                              float temperature, void* stream) {
    const char* fn = "ls_distill_topk_fwd";
    LS_TRY(check_distill(fn, dtype, rows, vocab, k, temperature));
    if (rows == 0) return ok();
    LS_TRY(check_ptr4(loss, "loss", true));
    LS_TRY(check_ptr4(lse, "lse", false));
    LS_TRY(check_ptr(logits, "logits", true));
    LS_TRY(check_ptr4(teacher_index, "teacher_index", true));
    LS_TRY(check_ptr_n(teacher_logits, "teacher_logits", true, elem_size(dtype)));
    LS_TRY(check_ptr4(teacher_lse, "teacher_lse", false));
    const size_t rb = static_cast<size_t>(rows) * 4, es = elem_size(dtype);
    const Span outs[] = {{"loss", loss, rb}, {"lse", lse, rb}};
    const Span ins[] = {{"logits", logits, static_cast<size_t>(rows * vocab) * es},
                        {"teacher_index", teacher_index, static_cast<size_t>(rows * k) * 4},
                        {"teacher_logits", teacher_logits, static_cast<size_t>(rows * k) * es},
                        {"teacher_lse", teacher_lse, rb}};
    LS_TRY(check_disjoint(outs, 2, ins, 4));
    const ls::DistillShape sh{rows, vocab, static_cast<int>(k), temperature};
    return from_cuda(ls::launch_distill_fwd(dtype, loss, lse, logits, teacher_index,
                                            teacher_logits, teacher_lse, sh, as_stream(stream)),
                     fn);
}

ls_status ls_distill_topk_bwd(ls_dtype dtype, void* dlogits, const void* logits,
                              const int32_t* teacher_index, const void* teacher_logits,
                              const float* lse, const float* teacher_lse, const float* dloss,
                              int64_t rows, int64_t vocab, int64_t k, float temperature,
                              void* stream) {
    const char* fn = "ls_distill_topk_bwd";
    LS_TRY(check_distill(fn, dtype, rows, vocab, k, temperature));
    if (rows == 0) return ok();
    LS_TRY(check_ptr(dlogits, "dlogits", true));
    LS_TRY(check_ptr(logits, "logits", true));
    LS_TRY(check_ptr4(teacher_index, "teacher_index", true));
    LS_TRY(check_ptr_n(teacher_logits, "teacher_logits", true, elem_size(dtype)));
    LS_TRY(check_ptr4(lse, "lse", true));
    LS_TRY(check_ptr4(teacher_lse, "teacher_lse", false));
    LS_TRY(check_ptr4(dloss, "dloss", false));
    const size_t rb = static_cast<size_t>(rows) * 4, es = elem_size(dtype);
    const size_t zb = static_cast<size_t>(rows * vocab) * es;
    const Span outs[] = {{"dlogits", dlogits, zb}};
    // logits themselves may be dlogits; anything else may not overlap it.
    const Span ins[] = {{"logits", dlogits == logits ? nullptr : logits, zb},
                        {"teacher_index", teacher_index, static_cast<size_t>(rows * k) * 4},
                        {"teacher_logits", teacher_logits, static_cast<size_t>(rows * k) * es},
                        {"lse", lse, rb},
                        {"teacher_lse", teacher_lse, rb},
                        {"dloss", dloss, rb}};
    LS_TRY(check_disjoint(outs, 1, ins, 6));
    const ls::DistillShape sh{rows, vocab, static_cast<int>(k), temperature};
    return from_cuda(ls::launch_distill_bwd(dtype, dlogits, logits, teacher_index, teacher_logits,
                                            lse, teacher_lse, dloss, sh, as_stream(stream)),
                     fn);
}

ls_status ls_embedding_lookup_fwd(ls_dtype dtype, void* y, const int32_t* tokens,
                                  const void* table, int64_t tokens_count, int64_t hidden,
                                  int64_t vocab, float scale, void* stream) {
    const char* fn = "ls_embedding_lookup_fwd";
    LS_TRY(check_lookup(fn, dtype, tokens_count, hidden, vocab, scale));
    if (tokens_count == 0) return ok();
    LS_TRY(check_ptr(y, "y", true));
    LS_TRY(check_ptr4(tokens, "tokens", true));
    LS_TRY(check_ptr(table, "table", vocab > 0));
    const size_t es = elem_size(dtype);
    const Span outs[] = {{"y", y, static_cast<size_t>(tokens_count * hidden) * es}};
    const Span ins[] = {{"tokens", tokens, static_cast<size_t>(tokens_count) * 4},
                        {"table", table, static_cast<size_t>(vocab * hidden) * es}};
    LS_TRY(check_disjoint(outs, 1, ins, 2));
    return from_cuda(ls::launch_embedding_lookup_fwd(dtype, y, tokens, table, tokens_count, hidden,
                                                     vocab, scale, as_stream(stream)),
                     fn);
}

size_t ls_embedding_lookup_workspace_bytes(int64_t tokens_count, int64_t hidden, int64_t vocab) {
    if (tokens_count <= 0 || tokens_count > ls::kMaxLookupTokens || hidden <= 0 ||
        hidden > ls::kMaxHeadHidden || hidden % 8 != 0 || vocab <= 0 || vocab > ls::kMaxVocab)
        return 0;
    return ls::embedding_lookup_workspace_bytes(tokens_count, hidden, vocab);
}

ls_status ls_embedding_lookup_bwd(ls_dtype dtype, float* d_table, const void* dy,
                                  const int32_t* tokens, int64_t tokens_count, int64_t hidden,
                                  int64_t vocab, float scale, int32_t padding_id, int accumulate,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "ls_embedding_lookup_bwd";
    LS_TRY(check_lookup(fn, dtype, tokens_count, hidden, vocab, scale));
    if (vocab == 0) return ok();
    LS_TRY(check_ptr(d_table, "d_table", !(tokens_count == 0 && accumulate)));
    const size_t tb = static_cast<size_t>(vocab * hidden) * 4;
    if (tokens_count == 0) {
        if (accumulate) return ok();
        return from_cuda(cudaMemsetAsync(d_table, 0, tb, as_stream(stream)), fn);
    }
    LS_TRY(check_ptr(dy, "dy", true));
    LS_TRY(check_ptr4(tokens, "tokens", true));
    const size_t need = ls::embedding_lookup_workspace_bytes(tokens_count, hidden, vocab);
    LS_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    const Span outs[] = {{"d_table", d_table, tb}, {"workspace", workspace, need}};
    const Span ins[] = {{"dy", dy, static_cast<size_t>(tokens_count * hidden) * elem_size(dtype)},
                        {"tokens", tokens, static_cast<size_t>(tokens_count) * 4}};
    LS_TRY(check_disjoint(outs, 2, ins, 2));
    return from_cuda(ls::launch_embedding_lookup_bwd(dtype, d_table, dy, tokens, tokens_count,
                                                     hidden, vocab, scale, padding_id,
                                                     accumulate != 0, workspace,
                                                     as_stream(stream)),
                     fn);
}

}  // extern "C"
#pragma GCC visibility pop
