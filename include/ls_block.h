/*
 * ls_block.h -- C ABI of the decoder block's operators for NVIDIA GB300
 * (sm_103a), libls_block.so: what a training or decoding step of a gated
 * decoder runs between its matrix products, and between its backward pass and
 * its update.  They stand next to the reshape of Q, K and V, the bias + ReLU +
 * dropout and the trainer update of ls_ops.h:
 *  - rotary positions of queries and keys, forward and backward;
 *  - norms of queries and keys for each head with the rotation in the same
 *    pass, forward and backward;
 *  - the gated feed-forward block: both projections, the activation and the
 *    product in one kernel, and its gradients;
 *  - the global norm of many gradients, gradients scaled by a factor on the
 *    device, and the trainer update with such a factor.
 *
 * Conventions are those of ls_ops.h (status codes, storage types with FP32
 * arithmetic, device buffers owned by the caller, nothing allocated, nothing
 * synchronised, all work enqueued on `stream`, argument errors returned before
 * anything is enqueued), and:
 *  - Storage may also be BF16 (LS_BF16).
 *  - Descriptors (ls_head_view, ls_rotation, ls_tensor) are read during the
 *    call and may be changed or freed after it.
 *  - No output may overlap an input, another output or the workspace, except
 *    where an entry point says so.
 *  - A workspace is scratch: it needs no initialisation and holds nothing
 *    between calls, so calls ordered on one stream (or graphs whose replays
 *    are ordered) may share one.  Calls that can run at the same time on the
 *    GPU must not.
 *  - Results do not depend on the run: every sum is added in an order that
 *    the shapes fix, without floating-point atomics.
 */
#ifndef LS_BLOCK_H
#define LS_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "ls_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Message of this library's last failing call on this host thread ("" if none). */
const char* ls_block_last_error(void);

/* ls_check_device_errors for this library's kernels: waits for all work on
 * the current device, returns the OR of the failure flags raised since the
 * previous call (LS_DEVERR_WAIT_TIMEOUT: a bounded wait for a bulk copy or a
 * tensor-core product ran out, and that call's outputs are incomplete) and
 * clears them. */
ls_status ls_block_check_device_errors(uint32_t* flags);

/* Self-test of that failure path, as ls_selftest_wait_timeout: enqueues two
 * warps that wait on a barrier which nothing completes, for `polls` polls
 * (1 .. 2^19, each up to about 2 us); LS_DEVERR_WAIT_TIMEOUT is recorded and
 * they exit. */
ls_status ls_block_selftest_wait_timeout(uint32_t polls, void* stream);

/* --- Queries and keys -------------------------------------------------------
 * A [batch, seq, heads, head_dim] view in the storage dtype: element
 * (b, l, h, j) is data[b * batch_stride + l * seq_stride + h * head_stride + j],
 * strides in elements.  Head-major memory ([batch, heads, seq, head_dim], as
 * ls_bias_reshape_qkv_fwd writes it) and the rows of a packed projection are
 * both such views.  data must be 16-byte aligned, the strides (of sizes above
 * 1) non-negative multiples of 8, head_dim a multiple of 8 up to 512, and
 * batch * seq at most 2^30.  The elements of an output must be distinct (each
 * stride at least what the smaller ones span); an input may repeat them
 * (stride 0). */
typedef struct {
    void* data;
    int64_t heads;
    int64_t batch_stride, seq_stride, head_stride;
} ls_head_view;

/* A rotation of the first rotary_dim elements of each head (even, at most
 * head_dim), the others left as they are.  Pair i is the elements (2i, 2i + 1)
 * (interleaved != 0) or (i, i + rotary_dim / 2), and turns by
 * turns[i] * position * 2^-64 of a full circle: fixed-point numbers, so that
 * the angle of a far position is as exact as that of a near one.
 *   (a, b) -> scale * (a cos - b sin, a sin + b cos)
 * turns: device memory, [rotary_dim / 2], 8-byte aligned, made once from
 * ls_rotary_frequencies or ls_rotary_turns.  positions: int32 [batch * seq]
 * on the device (any value, negative ones too), or NULL: element l of a
 * sequence is at first_position + l, both ends of which are int32. */
typedef struct {
    const uint64_t* turns;
    int64_t rotary_dim;
    int32_t interleaved;
    float scale;
    const int32_t* positions;
    int64_t first_position;
} ls_rotation;

/* How positions beyond the trained ones are brought into its range. */
typedef enum {
    LS_ROTARY_PLAIN = 0,   /* w_i = base^(-2i / rotary_dim) */
    LS_ROTARY_LINEAR = 1,  /* w_i / factor */
    LS_ROTARY_NTK = 2,     /* base * factor^(rotary_dim / (rotary_dim - 2)) in place of base, so that
                              the slowest pair is slowed by factor and the fastest stays */
    LS_ROTARY_YARN = 3     /* by parts (Peng et al., "YaRN", ICLR 2024): pairs that turn more than 32
                              times in original_positions stay, those that turn less than once are
                              slowed by factor, linearly in i between them (from the floor of the one
                              border to the ceiling of the other); scale = 0.1 ln(factor) + 1 */
} ls_rotary_scaling;

/* The frequencies of a rotation: turns (HOST memory, [rotary_dim / 2]) and
 * scale (host, nullable; 1 but for LS_ROTARY_YARN).  rotary_dim is even, 2 to
 * 512; base is at least 1 (above 1 for LS_ROTARY_YARN) and finite; factor is
 * at least 1 (1 for LS_ROTARY_PLAIN); original_positions at least 1 for
 * LS_ROTARY_YARN, ignored otherwise. */
ls_status ls_rotary_frequencies(uint64_t* turns, float* scale, int64_t rotary_dim, double base,
                                ls_rotary_scaling scaling, double factor,
                                int64_t original_positions);

/* turns of frequencies of the program's own: radians per position (host, any
 * finite values), n of them. */
ls_status ls_rotary_turns(uint64_t* turns, const double* radians, int64_t n);

/* q_out = the rotation of q, k_out that of k.  k and k_out may both be NULL
 * (one tensor).  An output may be its own input (the same view): elements
 * behind rotary_dim are then not touched. */
ls_status ls_rotary_fwd(ls_dtype dtype, const ls_head_view* q_out, const ls_head_view* k_out,
                        const ls_head_view* q, const ls_head_view* k, int64_t batch, int64_t seq,
                        int64_t head_dim, const ls_rotation* rotation, void* stream);

/* Backward of the above: dq = the transposed rotation of dq_out (the gradient
 * of q_out), dk likewise.  dq may be dq_out and dk dk_out. */
ls_status ls_rotary_bwd(ls_dtype dtype, const ls_head_view* dq, const ls_head_view* dk,
                        const ls_head_view* dq_out, const ls_head_view* dk_out, int64_t batch,
                        int64_t seq, int64_t head_dim, const ls_rotation* rotation, void* stream);

/* Norm of each head's row, and the rotation:
 *   u = x / sqrt(mean_j x_j^2 + eps),  y = rotation(weight * u)
 * for q with q_weight and for k with k_weight ([head_dim] in the storage
 * dtype, shared by the heads, 16-byte aligned; NULL: ones).  rotation may be
 * NULL (no rotation); k with its output and weight may be NULL.  The mean of
 * squares is an FP32 number: BF16 and FP32 values up to 2^60 are within its
 * range, and squares below 2^-126 vanish, so that a row whose values are all
 * below 2^-60 needs an eps above 2^-120.  An output may be its own input (the
 * same view). */
ls_status ls_qk_norm_rotary_fwd(ls_dtype dtype, const ls_head_view* q_out,
                                const ls_head_view* k_out, const ls_head_view* q,
                                const ls_head_view* k, const void* q_weight, const void* k_weight,
                                float eps, int64_t batch, int64_t seq, int64_t head_dim,
                                const ls_rotation* rotation, void* stream);

/* Backward of the above from its inputs (nothing else is kept), with
 * g = the transposed rotation of the output's gradient:
 *   dweight = sum over batch, seq and heads of g u      (storage dtype, written, or NULL)
 *   dx      = (weight g - u mean_j(weight g u)) / sqrt(mean_j x_j^2 + eps)
 * dq may be dq_out or q (the same view), dk likewise.  workspace: at least
 * ls_qk_norm_rotary_workspace_bytes(head_dim) bytes where a dweight is wanted. */
ls_status ls_qk_norm_rotary_bwd(ls_dtype dtype, const ls_head_view* dq, const ls_head_view* dk,
                                void* dq_weight, void* dk_weight, const ls_head_view* dq_out,
                                const ls_head_view* dk_out, const ls_head_view* q,
                                const ls_head_view* k, const void* q_weight, const void* k_weight,
                                float eps, int64_t batch, int64_t seq, int64_t head_dim,
                                const ls_rotation* rotation, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Workspace bytes of ls_qk_norm_rotary_bwd, for any number of rows; 0 for an
 * invalid head_dim. */
size_t ls_qk_norm_rotary_workspace_bytes(int64_t head_dim);

/* --- The gated feed-forward block -------------------------------------------
 * Activations: x sigmoid(x); x Phi(x) with the normal distribution's Phi; its
 * form 0.5 x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))); max(x, 0) with slope 0
 * at 0.  They are off by a few 1e-6 of themselves at most, where they all but
 * vanish by 2e-5, which is far below a rounding to storage. */
typedef enum {
    LS_ACT_SILU = 0,
    LS_ACT_GELU = 1,
    LS_ACT_GELU_TANH = 2,
    LS_ACT_RELU = 3
} ls_activation;

/* Both projections of a gated block, the activation and the product in one
 * kernel.  x: [rows, hidden], gate_weight and up_weight: [ffn, hidden], h:
 * [rows, ffn], row-major and contiguous, LS_F16 or LS_BF16:
 *   h[i,f] = act(sum_c x[i,c] gate_weight[f,c]) * sum_c x[i,c] up_weight[f,c]
 * Both sums stay in FP32; h is rounded once.  They run in the tensor cores'
 * accumulators, which drop low bits, over at most 32768 columns (2e-4 of a sum
 * of terms of one sign), and in FP32 from there on.  hidden and ffn are
 * multiples of 8, at most 65536; rows at most 2^24. */
ls_status ls_gated_linear_fwd(ls_dtype dtype, void* h, const void* x, const void* gate_weight,
                              const void* up_weight, int64_t rows, int64_t hidden, int64_t ffn,
                              ls_activation activation, void* stream);

/* Backward of the above, from its inputs (g and u, the two sums, are computed
 * again; the forward keeps nothing):
 *   dg = dh u act'(g),  du = dh act(g)                    (rounded once to the storage dtype; of up
 *                                to 32 rows and 16384 elements to two numbers of it each)
 *   dx = dg gate_weight + du up_weight,  dgate_weight = dg^T x,  dup_weight = du^T x
 * That rounding adds as much error as the gradients' own: sqrt(2) of a rounding
 * as a whole.  In LS_F16 it also has the type's range: a dg or du beyond 65504
 * is infinite, and the gradients that it is part of are infinite or NaNs, and
 * one below 2^-25 is zero, even where the gradients themselves are in range.  A
 * loss scale has to keep dg and du in range as it has to keep the gradients;
 * LS_BF16 has FP32's range.  dx: [rows, hidden] in the storage dtype, written, or NULL.  dgate_weight and
 * dup_weight: [ffn, hidden], both or neither NULL; with dweight_dtype == dtype
 * they are written; with dweight_dtype == LS_F32 the gradients are ADDED to
 * them.  rows == 0 writes zeros to weight gradients in the storage dtype.  The
 * sums run in the tensor cores' accumulators as the forward's do, over at most
 * 16384 rows or 32768 columns (9e-5 and 2e-4 of a sum of terms of one sign),
 * and in FP32 from there on.  workspace: at least
 * ls_gated_linear_workspace_bytes bytes. */
ls_status ls_gated_linear_bwd(ls_dtype dtype, void* dx, void* dgate_weight, void* dup_weight,
                              ls_dtype dweight_dtype, const void* dh, const void* x,
                              const void* gate_weight, const void* up_weight, int64_t rows,
                              int64_t hidden, int64_t ffn, ls_activation activation,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of ls_gated_linear_bwd: dg and du (of few elements twice), up to 16 FP32 copies of
 * dx, and FP32 sums of the weights' gradients (one of each beyond 16384 rows, up
 * to 8 of small weights).  0 for invalid sizes.  The forward needs none. */
size_t ls_gated_linear_workspace_bytes(int64_t rows, int64_t hidden, int64_t ffn);

/* --- The norm of many gradients, clipping, and the update ---------------------
 * One of many tensors: n contiguous elements (0 is allowed) of `dtype`, data
 * aligned to its element. */
typedef struct {
    void* data;
    int64_t n;
    int64_t dtype; /* an ls_dtype */
} ls_tensor;

/* The global norm of `count` gradients times grad_scale (1 / loss scale), and
 * the factor that brings them to a norm of at most max_norm:
 *   norm[0]   = |grad_scale| * sqrt(sum over all tensors and elements of g^2)
 *   factor[0] = grad_scale * min(1, max_norm / (norm + 1e-6))
 * norm and factor: FP32 on the device, 4-byte aligned, either may be NULL.
 * grads: host array; the types may differ.  The sum neither overflows nor
 * underflows as long as the norm is an FP32 number.  A NaN among the gradients
 * gives a NaN for both, an infinite one the norm inf and, for a finite
 * max_norm, the factor 0 (of which an infinity makes a NaN: a step to be left
 * out, as ls_adam_update_clipped does).  max_norm: at least 0, inf for none; grad_scale:
 * finite.  workspace: at least ls_grad_norm_workspace_bytes() bytes. */
ls_status ls_grad_norm(float* norm, float* factor, const ls_tensor* grads, int64_t count,
                       float max_norm, float grad_scale, void* workspace, size_t workspace_bytes,
                       void* stream);

size_t ls_grad_norm_workspace_bytes(void);

/* out[t] = factor[0] * in[t], rounded once, for each of `count` pairs of
 * tensors of one size and type; out[t] may be in[t] (the same data).  factor:
 * FP32 on the device.  In place a factor of 1 reads and writes nothing.
 * Outputs may not overlap other tensors of the call; of that only each pair is
 * checked. */
ls_status ls_scale_gradients(const ls_tensor* out, const ls_tensor* in, int64_t count,
                             const float* factor, void* stream);

/* ls_adam_update with the gradient's factor in device memory (such as
 * ls_grad_norm leaves it), so that clipping needs neither a pass over the
 * gradients nor the host; LS_F32, LS_F16 or LS_BF16. */
ls_status ls_adam_update_scaled(ls_dtype dtype, void* param, const void* grad, float* exp_avg,
                                float* exp_avg_sq, int64_t n, float lr, float beta1, float beta2,
                                float eps, float weight_decay, int64_t step, const float* factor,
                                void* stream);

/* The same for a step that may have overflowed, as one of a scaled loss may:
 * where norm[0] (FP32 on the device, such as ls_grad_norm leaves it) is
 * infinite or a NaN, nothing is written.  What takes a factor without its norm
 * has no such guard: infinite or NaN gradients reach its outputs. */
ls_status ls_adam_update_clipped(ls_dtype dtype, void* param, const void* grad, float* exp_avg,
                                 float* exp_avg_sq, int64_t n, float lr, float beta1, float beta2,
                                 float eps, float weight_decay, int64_t step, const float* norm,
                                 const float* factor, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LS_BLOCK_H */
