// block_api.cu -- the C ABI declared in include/ls_block.h: every entry point
// checks its arguments on the host, before anything is enqueued, and hands
// the call to a launcher of block_internal.h.  Nothing here allocates,
// synchronises (ls_block_check_device_errors apart) or keeps state but the
// per-thread message of the last error.
#include <math.h>

#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../csrc_vocab/host_check.h"
#include "block_internal.h"

namespace {

constexpr int64_t kMaxTokens = int64_t{1} << 30;
constexpr int64_t kMaxHeads = 65536;
constexpr int64_t kMostElements = int64_t{1} << 46;  // from a view's first element to its last

// --- views of heads -------------------------------------------------------------
// Elements i0 stride0 + i1 stride1 + i2 stride2 + [0, run) from `at` on.
struct Lattice {
    int64_t at;  // in elements
    int64_t size[3], stride[3];
    int64_t run;
    int64_t extent() const {
        int64_t n = run;
        for (int k = 0; k < 3; ++k) n += (size[k] - 1) * stride[k];
        return n;
    }
};

Lattice lattice_of(const ls_head_view& v, int64_t batch, int64_t seq, int64_t dim, size_t es) {
    return Lattice{static_cast<int64_t>(reinterpret_cast<uintptr_t>(v.data) / es),
                   {batch, seq, v.heads},
                   {v.batch_stride, v.seq_stride, v.head_stride},
                   dim};
}

bool is_empty(const Lattice& a) { return a.size[0] == 0 || a.size[1] == 0 || a.size[2] == 0; }

bool same(const Lattice& a, const Lattice& b) {
    if (a.at != b.at) return false;
    for (int k = 0; k < 3; ++k)
        if (a.size[k] != b.size[k] || (a.size[k] > 1 && a.stride[k] != b.stride[k])) return false;
    return true;
}

// Whether two sets of elements surely have none in common: their extents do
// not overlap, or they repeat with one outermost period, in which both find
// room, and have none in common within a period.
bool apart(Lattice a, Lattice b) {
    if (is_empty(a) || is_empty(b)) return true;
    for (;;) {
        const int64_t ea = a.extent(), eb = b.extent();
        if (a.at + ea <= b.at || b.at + eb <= a.at) return true;
        int k = -1;
        for (int i = 0; i < 3; ++i)
            if (std::max(a.size[i], b.size[i]) > 1 && (k < 0 || a.stride[i] > a.stride[k])) k = i;
        if (k < 0 || a.stride[k] != b.stride[k] || a.stride[k] == 0) return false;
        const int64_t period = a.stride[k];
        a.size[k] = b.size[k] = 1;
        const int64_t ra = a.extent(), rb = b.extent();
        int64_t off = (b.at - a.at) % period;  // either side of 0
        bool fits = false;
        for (const int64_t o : {off, off > 0 ? off - period : off + period})
            if (std::max(ra, o + rb) - std::min<int64_t>(0, o) <= period) {
                fits = true;
                off = o;
                break;
            }
        if (!fits) return false;
        a.at = std::max<int64_t>(0, -off);
        b.at = a.at + off;
    }
}

ls_status check_view(const char* fn, const char* name, const ls_head_view* v, int64_t batch,
                     int64_t seq, int64_t dim, bool output) {
    if (!v) return fail(LS_ERR_INVALID_ARGUMENT, "%s: %s is NULL", fn, name);
    LS_TRY(check_size(fn, "heads", v->heads, 0, kMaxHeads));
    const int64_t size[3] = {batch, seq, v->heads};
    const int64_t stride[3] = {v->batch_stride, v->seq_stride, v->head_stride};
    if (batch * seq == 0 || v->heads == 0) return LS_OK;
    LS_TRY(check_ptr(v->data, name, true));
    for (int k = 0; k < 3; ++k) {
        if (size[k] <= 1) continue;
        if (stride[k] < 0)
            return fail(LS_ERR_INVALID_ARGUMENT, "%s: %s has a negative stride", fn, name);
        if (stride[k] % 8 != 0)
            return fail(LS_ERR_MISALIGNED, "%s: %s has a stride that is no multiple of 8", fn, name);
        if (stride[k] > kMostElements / size[k])
            return fail(LS_ERR_UNSUPPORTED_SHAPE, "%s: %s spans too many elements", fn, name);
    }
    if (!output) return LS_OK;
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return stride[a] < stride[b]; });
    int64_t extent = dim;
    for (const int k : order) {
        if (size[k] <= 1) continue;
        if (stride[k] < extent)
            return fail(LS_ERR_INVALID_ARGUMENT, "%s: elements of the output %s overlap", fn, name);
        extent += (size[k] - 1) * stride[k];
    }
    return LS_OK;
}

// Views with sizes of 1 in the place of strides that nothing uses.
ls_head_view tidy(const ls_head_view& v, int64_t batch, int64_t seq) {
    ls_head_view t = v;
    if (batch <= 1) t.batch_stride = 0;
    if (seq <= 1) t.seq_stride = 0;
    if (v.heads <= 1) t.head_stride = 0;
    return t;
}

ls_status check_rotation(const char* fn, const ls_rotation* r, int64_t batch, int64_t seq,
                         int64_t dim) {
    if (r->rotary_dim < 2 || r->rotary_dim % 2 != 0)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: rotary_dim = %lld is not an even number from 2 on",
                    fn, (long long)r->rotary_dim);
    if (r->rotary_dim > dim)
        return fail(LS_ERR_UNSUPPORTED_SHAPE, "%s: rotary_dim = %lld exceeds head_dim = %lld", fn,
                    (long long)r->rotary_dim, (long long)dim);
    if (!isfinite(r->scale)) return fail(LS_ERR_INVALID_ARGUMENT, "%s: scale is not finite", fn);
    if (batch * seq == 0) return LS_OK;
    LS_TRY(check_ptr_n(r->turns, "turns", true, 8));
    LS_TRY(check_ptr4(r->positions, "positions", false));
    if (!r->positions && (r->first_position < INT32_MIN || r->first_position > INT32_MAX ||
                          r->first_position + seq - 1 > INT32_MAX))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: positions from %lld on are not int32", fn,
                    (long long)r->first_position);
    return LS_OK;
}

ls_status check_heads_sizes(const char* fn, ls_dtype dt, int64_t batch, int64_t seq, int64_t dim) {
    LS_TRY(check_storage(fn, dt, true));
    LS_TRY(check_size(fn, "batch", batch, 0, kMaxTokens));
    LS_TRY(check_size(fn, "seq", seq, 0, kMaxTokens));
    LS_TRY(check_size(fn, "batch * seq", batch * seq, 0, kMaxTokens));
    LS_TRY(check_size(fn, "head_dim", dim, 1, ls::kMaxHeadDim));
    return check_multiple_of_8(fn, "head_dim", dim);
}

// One of a call's two tensors: its views and their names.
struct HeadsTensor {
    const ls_head_view *x, *g, *y;  // g: the backward's second input, or NULL
    const char *xn, *gn, *yn;
    const void* w;
    void* dw;
    const char *wn, *dwn;
};

ls_status run_heads(const char* fn, ls_dtype dt, HeadsTensor (&t)[2], bool norm, bool backward,
                    int64_t batch, int64_t seq, int64_t dim, const ls_rotation* rot, float eps,
                    void* workspace, size_t workspace_bytes, void* stream) {
    LS_TRY(check_heads_sizes(fn, dt, batch, seq, dim));
    if (rot) LS_TRY(check_rotation(fn, rot, batch, seq, dim));
    if (norm && !(eps >= 0.f && eps < INFINITY))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: eps = %g is not a finite number from 0 on", fn,
                    static_cast<double>(eps));
    const bool two = t[1].x || t[1].y || t[1].g;
    if (!two && (t[1].w || t[1].dw))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: a weight of k without k", fn);
    const size_t es = elem_size(dt), wb = static_cast<size_t>(dim) * es;
    bool dweights = false;
    Lattice y[2], in[4];
    const char* in_name[4];
    ls_head_view view[2][3];
    int n_in = 0;
    ls::HeadsCall c = {};
    for (int k = 0; k < (two ? 2 : 1); ++k) {
        HeadsTensor& q = t[k];
        LS_TRY(check_view(fn, q.xn, q.x, batch, seq, dim, false));
        LS_TRY(check_view(fn, q.yn, q.y, batch, seq, dim, true));
        if (q.gn) LS_TRY(check_view(fn, q.gn, q.g, batch, seq, dim, false));
        if (q.y->heads != q.x->heads || (q.gn && q.g->heads != q.x->heads))
            return fail(LS_ERR_INVALID_ARGUMENT, "%s: %s and %s have different numbers of heads", fn,
                        q.xn, q.yn);
        if (norm) {
            LS_TRY(check_ptr(q.w, q.wn, false));
            if (q.dwn) LS_TRY(check_ptr(q.dw, q.dwn, false));
            if (q.dw && !q.w)
                return fail(LS_ERR_INVALID_ARGUMENT, "%s: %s without %s", fn, q.dwn, q.wn);
            dweights = dweights || q.dw;
        }
        view[k][0] = tidy(*q.x, batch, seq);
        view[k][1] = tidy(*q.y, batch, seq);
        if (q.gn) view[k][2] = tidy(*q.g, batch, seq);
        y[k] = lattice_of(view[k][1], batch, seq, dim, es);
        in_name[n_in] = q.xn;
        in[n_in++] = lattice_of(view[k][0], batch, seq, dim, es);
        if (q.gn) {
            in_name[n_in] = q.gn;
            in[n_in++] = lattice_of(view[k][2], batch, seq, dim, es);
        }
        c.x[k] = &view[k][0];
        c.y[k] = &view[k][1];
        c.g[k] = q.gn ? &view[k][2] : nullptr;
        c.weight[k] = q.w;
        c.dweight[k] = q.dw;
    }
    const size_t need = dweights ? ls::heads_workspace_bytes(dim) : 0;
    LS_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    const int per = n_in / (two ? 2 : 1);
    if (two && !apart(y[0], y[1]))
        return fail(LS_ERR_INVALID_ARGUMENT, "outputs %s and %s overlap", t[0].yn, t[1].yn);
    for (int k = 0; k < (two ? 2 : 1); ++k)
        for (int i = 0; i < n_in; ++i)
            if (!apart(y[k], in[i]) && !(i / per == k && same(y[k], in[i])))
                return fail(LS_ERR_INVALID_ARGUMENT, "output %s overlaps input %s", t[k].yn,
                            in_name[i]);
    // Contiguous buffers, against the outputs' extents and one another.
    const size_t pb = rot && rot->positions ? static_cast<size_t>(batch * seq) * 4 : 0;
    const Span ins[] = {{"turns", rot ? rot->turns : nullptr,
                         rot ? static_cast<size_t>(rot->rotary_dim) * 4 : 0},
                        {"positions", rot ? rot->positions : nullptr, pb},
                        {"q_weight", t[0].w, wb},
                        {"k_weight", t[1].w, wb}};
    const Span small[] = {{t[0].dwn, t[0].dw, wb},
                          {t[1].dwn, t[1].dw, wb},
                          {"workspace", need ? workspace : nullptr, need}};
    LS_TRY(check_disjoint(small, 3, ins, 4));
    auto span_of = [&](const Lattice& l, const char* name) {
        return Span{name, is_empty(l) ? nullptr : reinterpret_cast<const void*>(static_cast<uintptr_t>(l.at) * es),
                    is_empty(l) ? 0 : static_cast<size_t>(l.extent()) * es};
    };
    for (int k = 0; k < (two ? 2 : 1); ++k) {
        const Span out[] = {span_of(y[k], t[k].yn)};
        LS_TRY(check_disjoint(out, 1, ins, 4));
        LS_TRY(check_disjoint(out, 1, small, 3));
    }
    for (int i = 0; i < n_in; ++i) {
        const Span input[] = {span_of(in[i], in_name[i])};
        LS_TRY(check_disjoint(small, 3, input, 1));
    }
    c.norm = norm;
    c.backward = backward;
    c.batch = batch;
    c.seq = seq;
    c.dim = dim;
    c.rotation = rot;
    c.eps = eps;
    c.workspace = workspace;
    if (batch * seq == 0 && !dweights) return ok();
    return from_cuda(ls::launch_heads_dtype(dt, c, as_stream(stream)), fn);
}

// --- gated, clip ------------------------------------------------------------------
ls_status check_gated(const char* fn, ls_dtype dt, int64_t rows, int64_t hidden, int64_t ffn,
                      ls_activation act) {
    LS_TRY(check_storage(fn, dt, false));
    LS_TRY(check_size(fn, "rows", rows, 0, ls::kMaxGatedRows));
    LS_TRY(check_size(fn, "hidden", hidden, 1, ls::kMaxGatedCols));
    LS_TRY(check_multiple_of_8(fn, "hidden", hidden));
    LS_TRY(check_size(fn, "ffn", ffn, 1, ls::kMaxGatedCols));
    LS_TRY(check_multiple_of_8(fn, "ffn", ffn));
    if (static_cast<int>(act) < 0 || act > LS_ACT_RELU)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: unknown activation %d", fn, static_cast<int>(act));
    return LS_OK;
}

ls_status check_tensors(const char* fn, const char* name, const ls_tensor* t, int64_t count) {
    if (count > 0 && !t) return fail(LS_ERR_INVALID_ARGUMENT, "%s: %s is NULL", fn, name);
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].dtype != LS_F32 && t[i].dtype != LS_F16 && t[i].dtype != LS_BF16)
            return fail(LS_ERR_INVALID_ARGUMENT, "%s: %s[%lld] has the unknown dtype %lld", fn, name,
                        (long long)i, (long long)t[i].dtype);
        if (t[i].n < 0 || t[i].n > (int64_t{1} << 44))
            return fail(t[i].n < 0 ? LS_ERR_INVALID_ARGUMENT : LS_ERR_UNSUPPORTED_SHAPE,
                        "%s: %s[%lld] has %lld elements", fn, name, (long long)i, (long long)t[i].n);
        if (t[i].n == 0) continue;
        if (!t[i].data)
            return fail(LS_ERR_INVALID_ARGUMENT, "%s: %s[%lld] is NULL", fn, name, (long long)i);
        if (reinterpret_cast<uintptr_t>(t[i].data) % elem_size(static_cast<ls_dtype>(t[i].dtype)))
            return fail(LS_ERR_MISALIGNED, "%s: %s[%lld] is not aligned to its elements", fn, name,
                        (long long)i);
    }
    return LS_OK;
}

ls_status run_adam(const char* fn, ls_dtype dtype, void* param, const void* grad, float* exp_avg,
                   float* exp_avg_sq, int64_t n, const ls::AdamScaled& h, void* stream) {
    LS_TRY(check_storage(fn, dtype, true));
    LS_TRY(check_size(fn, "n", n, 0, int64_t{1} << 44));
    LS_TRY(check_size(fn, "step", h.step, 1, INT64_MAX));
    if (!(h.beta1 >= 0.f && h.beta1 < 1.f && h.beta2 >= 0.f && h.beta2 < 1.f))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: betas %g, %g are not in [0, 1)", fn,
                    static_cast<double>(h.beta1), static_cast<double>(h.beta2));
    for (const float v : {h.lr, h.eps, h.weight_decay})
        if (!(v >= 0.f && v < INFINITY))
            return fail(LS_ERR_INVALID_ARGUMENT, "%s: lr, eps or weight_decay is not a finite number from 0 on", fn);
    if (n == 0) return ok();
    LS_TRY(check_ptr(param, "param", true));
    LS_TRY(check_ptr(grad, "grad", true));
    LS_TRY(check_ptr(exp_avg, "exp_avg", true));
    LS_TRY(check_ptr(exp_avg_sq, "exp_avg_sq", true));
    LS_TRY(check_ptr4(h.factor, "factor", true));
    const size_t b = static_cast<size_t>(n) * elem_size(dtype), f = static_cast<size_t>(n) * 4;
    const Span outs[] = {{"param", param, b}, {"exp_avg", exp_avg, f}, {"exp_avg_sq", exp_avg_sq, f}};
    const Span ins[] = {{"grad", grad, b}, {"factor", h.factor, 4}, {"norm", h.norm, 4}};
    LS_TRY(check_disjoint(outs, 3, ins, 3));
    return from_cuda(ls::launch_adam_scaled(dtype, param, grad, exp_avg, exp_avg_sq, n, h, as_stream(stream)),
                     fn);
}

size_t bytes_of(const ls_tensor& t) {
    return static_cast<size_t>(t.n) * elem_size(static_cast<ls_dtype>(t.dtype));
}

}  // namespace

namespace ls {
cudaError_t launch_heads_dtype(ls_dtype dt, const HeadsCall& c, cudaStream_t s) {
    if (dt == LS_F16) return launch_heads<__half>(c, s);
    if (dt == LS_BF16) return launch_heads<__nv_bfloat16>(c, s);
    return launch_heads<float>(c, s);
}
}  // namespace ls

#pragma GCC visibility push(default)
extern "C" {

const char* ls_block_last_error(void) { return g_last_error; }

ls_status ls_block_check_device_errors(uint32_t* flags) {
    if (!flags) return fail(LS_ERR_INVALID_ARGUMENT, "flags is NULL");
    *flags = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return from_cuda(e, "ls_block_check_device_errors: synchronise");
    unsigned int v = 0;
    e = ls::gated_take_device_error(&v);
    if (e != cudaSuccess) return from_cuda(e, "ls_block_check_device_errors: read flags");
    *flags = v;
    return ok();
}

ls_status ls_block_selftest_wait_timeout(uint32_t polls, void* stream) {
    if (polls == 0 || polls > (1u << 19))
        return fail(LS_ERR_INVALID_ARGUMENT, "polls = %u is not in [1, 2^19]", polls);
    return from_cuda(ls::launch_block_wait_selftest(polls, as_stream(stream)),
                     "ls_block_selftest_wait_timeout");
}

ls_status ls_rotary_turns(uint64_t* turns, const double* radians, int64_t n) {
    const char* fn = "ls_rotary_turns";
    LS_TRY(check_size(fn, "n", n, 0, ls::kMaxHeadDim / 2));
    if (n > 0 && (!turns || !radians))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: turns or radians is NULL", fn);
    for (int64_t i = 0; i < n; ++i)
        if (!isfinite(radians[i]))
            return fail(LS_ERR_INVALID_ARGUMENT, "%s: radians[%lld] is not finite", fn, (long long)i);
    for (int64_t i = 0; i < n; ++i) {
        const double t = radians[i] / 6.283185307179586;
        const double part = t - floor(t);  // [0, 1]: 1 where t is a negative number next to 0
        turns[i] = part < 1.0 ? static_cast<uint64_t>(part * 0x1p64) : 0;
    }
    return ok();
}

ls_status ls_rotary_frequencies(uint64_t* turns, float* scale, int64_t rotary_dim, double base,
                                ls_rotary_scaling scaling, double factor,
                                int64_t original_positions) {
    const char* fn = "ls_rotary_frequencies";
    LS_TRY(check_size(fn, "rotary_dim", rotary_dim, 2, ls::kMaxHeadDim));
    if (rotary_dim % 2 != 0)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: rotary_dim = %lld is odd", fn, (long long)rotary_dim);
    if (static_cast<int>(scaling) < 0 || scaling > LS_ROTARY_YARN)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: unknown scaling %d", fn, static_cast<int>(scaling));
    const bool yarn = scaling == LS_ROTARY_YARN;
    if (!(base >= 1.0 && base < INFINITY) || (yarn && base == 1.0))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: base = %g is out of range", fn, base);
    if (!(factor >= 1.0 && factor < INFINITY) || (scaling == LS_ROTARY_PLAIN && factor != 1.0))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: factor = %g is out of range", fn, factor);
    if (yarn && original_positions < 1)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: original_positions = %lld < 1", fn,
                    (long long)original_positions);
    if (!turns) return fail(LS_ERR_INVALID_ARGUMENT, "%s: turns is NULL", fn);
    const double rd = static_cast<double>(rotary_dim);
    const int n = static_cast<int>(rotary_dim / 2);
    if (scaling == LS_ROTARY_NTK) base *= pow(factor, rd / std::max(rd - 2.0, 1.0));
    double low = 0.0, high = 0.0;
    if (yarn) {
        // the pair that turns so often in the original positions
        auto pair = [&](double often) {
            return rd * log(static_cast<double>(original_positions) / (6.283185307179586 * often)) /
                   (2.0 * log(base));
        };
        low = std::max(floor(pair(32.0)), 0.0);
        high = std::min(ceil(pair(1.0)), rd - 1.0);
    }
    double w[ls::kMaxHeadDim / 2];
    for (int i = 0; i < n; ++i) {
        w[i] = pow(base, -2.0 * i / rd);
        if (scaling == LS_ROTARY_LINEAR) w[i] /= factor;
        if (yarn) {
            const double slow = std::min(std::max((i - low) / std::max(high - low, 0.001), 0.0), 1.0);
            w[i] = w[i] * (1.0 - slow) + w[i] / factor * slow;
        }
    }
    if (scale) *scale = yarn ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
    return ls_rotary_turns(turns, w, n);
}

ls_status ls_rotary_fwd(ls_dtype dtype, const ls_head_view* q_out, const ls_head_view* k_out,
                        const ls_head_view* q, const ls_head_view* k, int64_t batch, int64_t seq,
                        int64_t head_dim, const ls_rotation* rotation, void* stream) {
    const char* fn = "ls_rotary_fwd";
    if (!rotation) return fail(LS_ERR_INVALID_ARGUMENT, "%s: rotation is NULL", fn);
    HeadsTensor t[2] = {{q, nullptr, q_out, "q", nullptr, "q_out", nullptr, nullptr, nullptr, nullptr},
                        {k, nullptr, k_out, "k", nullptr, "k_out", nullptr, nullptr, nullptr, nullptr}};
    return run_heads(fn, dtype, t, false, false, batch, seq, head_dim, rotation, 0.f, nullptr, 0, stream);
}

ls_status ls_rotary_bwd(ls_dtype dtype, const ls_head_view* dq, const ls_head_view* dk,
                        const ls_head_view* dq_out, const ls_head_view* dk_out, int64_t batch,
                        int64_t seq, int64_t head_dim, const ls_rotation* rotation, void* stream) {
    const char* fn = "ls_rotary_bwd";
    if (!rotation) return fail(LS_ERR_INVALID_ARGUMENT, "%s: rotation is NULL", fn);
    HeadsTensor t[2] = {{dq_out, nullptr, dq, "dq_out", nullptr, "dq", nullptr, nullptr, nullptr, nullptr},
                        {dk_out, nullptr, dk, "dk_out", nullptr, "dk", nullptr, nullptr, nullptr, nullptr}};
    return run_heads(fn, dtype, t, false, true, batch, seq, head_dim, rotation, 0.f, nullptr, 0, stream);
}

ls_status ls_qk_norm_rotary_fwd(ls_dtype dtype, const ls_head_view* q_out,
                                const ls_head_view* k_out, const ls_head_view* q,
                                const ls_head_view* k, const void* q_weight, const void* k_weight,
                                float eps, int64_t batch, int64_t seq, int64_t head_dim,
                                const ls_rotation* rotation, void* stream) {
    HeadsTensor t[2] = {{q, nullptr, q_out, "q", nullptr, "q_out", q_weight, nullptr, "q_weight", nullptr},
                        {k, nullptr, k_out, "k", nullptr, "k_out", k_weight, nullptr, "k_weight", nullptr}};
    return run_heads("ls_qk_norm_rotary_fwd", dtype, t, true, false, batch, seq, head_dim, rotation, eps,
                     nullptr, 0, stream);
}

ls_status ls_qk_norm_rotary_bwd(ls_dtype dtype, const ls_head_view* dq, const ls_head_view* dk,
                                void* dq_weight, void* dk_weight, const ls_head_view* dq_out,
                                const ls_head_view* dk_out, const ls_head_view* q,
                                const ls_head_view* k, const void* q_weight, const void* k_weight,
                                float eps, int64_t batch, int64_t seq, int64_t head_dim,
                                const ls_rotation* rotation, void* workspace,
                                size_t workspace_bytes, void* stream) {
    HeadsTensor t[2] = {
        {q, dq_out, dq, "q", "dq_out", "dq", q_weight, dq_weight, "q_weight", "dq_weight"},
        {k, dk_out, dk, "k", "dk_out", "dk", k_weight, dk_weight, "k_weight", "dk_weight"}};
    return run_heads("ls_qk_norm_rotary_bwd", dtype, t, true, true, batch, seq, head_dim, rotation, eps,
                     workspace, workspace_bytes, stream);
}

size_t ls_qk_norm_rotary_workspace_bytes(int64_t head_dim) {
    return head_dim > 0 && head_dim <= ls::kMaxHeadDim && head_dim % 8 == 0
               ? ls::heads_workspace_bytes(head_dim)
               : 0;
}

size_t ls_gated_linear_workspace_bytes(int64_t rows, int64_t hidden, int64_t ffn) {
    if (rows <= 0 || rows > ls::kMaxGatedRows || hidden <= 0 || hidden > ls::kMaxGatedCols ||
        hidden % 8 != 0 || ffn <= 0 || ffn > ls::kMaxGatedCols || ffn % 8 != 0)
        return 0;
    return ls::gated_plan(rows, hidden, ffn).bytes;
}

ls_status ls_gated_linear_fwd(ls_dtype dtype, void* h, const void* x, const void* gate_weight,
                              const void* up_weight, int64_t rows, int64_t hidden, int64_t ffn,
                              ls_activation activation, void* stream) {
    const char* fn = "ls_gated_linear_fwd";
    LS_TRY(check_gated(fn, dtype, rows, hidden, ffn, activation));
    if (rows == 0) return ok();
    LS_TRY(check_ptr(h, "h", true));
    LS_TRY(check_ptr(x, "x", true));
    LS_TRY(check_ptr(gate_weight, "gate_weight", true));
    LS_TRY(check_ptr(up_weight, "up_weight", true));
    const size_t wb = static_cast<size_t>(ffn * hidden) * 2;
    const Span outs[] = {{"h", h, static_cast<size_t>(rows * ffn) * 2}};
    const Span ins[] = {{"x", x, static_cast<size_t>(rows * hidden) * 2},
                        {"gate_weight", gate_weight, wb},
                        {"up_weight", up_weight, wb}};
    LS_TRY(check_disjoint(outs, 1, ins, 3));
    const ls::GatedShape sh{rows, hidden, ffn, activation};
    return from_cuda(ls::launch_gated_fwd(dtype, h, x, gate_weight, up_weight, sh, as_stream(stream)), fn);
}

ls_status ls_gated_linear_bwd(ls_dtype dtype, void* dx, void* dgate_weight, void* dup_weight,
                              ls_dtype dweight_dtype, const void* dh, const void* x,
                              const void* gate_weight, const void* up_weight, int64_t rows,
                              int64_t hidden, int64_t ffn, ls_activation activation,
                              void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "ls_gated_linear_bwd";
    LS_TRY(check_gated(fn, dtype, rows, hidden, ffn, activation));
    const bool f32 = dweight_dtype == LS_F32;
    if (!f32 && dweight_dtype != dtype)
        return fail(LS_ERR_INVALID_ARGUMENT,
                    "%s: dweight_dtype = %d is neither the storage dtype nor LS_F32", fn,
                    static_cast<int>(dweight_dtype));
    LS_TRY(check_ptr(dx, "dx", false));
    LS_TRY(check_ptr(dgate_weight, "dgate_weight", dup_weight != nullptr));
    LS_TRY(check_ptr(dup_weight, "dup_weight", dgate_weight != nullptr));
    if (rows > 0 && !dx && !dgate_weight)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: dx and the weights' gradients are all NULL", fn);
    const size_t wb = static_cast<size_t>(ffn * hidden) * 2, gb = wb / 2 * elem_size(dweight_dtype);
    if (rows == 0) {
        if (!dgate_weight || f32) return ok();
        const Span both[] = {{"dgate_weight", dgate_weight, gb}, {"dup_weight", dup_weight, gb}};
        LS_TRY(check_disjoint(both, 2, nullptr, 0));
        const cudaError_t e = cudaMemsetAsync(dgate_weight, 0, gb, as_stream(stream));
        if (e != cudaSuccess) return from_cuda(e, fn);
        return from_cuda(cudaMemsetAsync(dup_weight, 0, gb, as_stream(stream)), fn);
    }
    LS_TRY(check_ptr(dh, "dh", true));
    LS_TRY(check_ptr(x, "x", true));
    LS_TRY(check_ptr(gate_weight, "gate_weight", true));
    LS_TRY(check_ptr(up_weight, "up_weight", true));
    const ls::GatedPlan plan = ls::gated_plan(rows, hidden, ffn);
    const size_t need = plan.bytes;
    LS_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    const size_t xb = static_cast<size_t>(rows * hidden) * 2;
    const Span outs[] = {{"dx", dx, xb},
                         {"dgate_weight", dgate_weight, gb},
                         {"dup_weight", dup_weight, gb},
                         {"workspace", workspace, need}};
    const Span ins[] = {{"dh", dh, static_cast<size_t>(rows * ffn) * 2},
                        {"x", x, xb},
                        {"gate_weight", gate_weight, wb},
                        {"up_weight", up_weight, wb}};
    LS_TRY(check_disjoint(outs, 4, ins, 4));
    const ls::GatedShape sh{rows, hidden, ffn, activation};
    return from_cuda(ls::launch_gated_bwd(dtype, dx, dgate_weight, dup_weight, f32, dh, x, gate_weight,
                                          up_weight, sh, plan, workspace, as_stream(stream)),
                     fn);
}

size_t ls_grad_norm_workspace_bytes(void) { return ls::grad_norm_workspace_bytes(); }

ls_status ls_grad_norm(float* norm, float* factor, const ls_tensor* grads, int64_t count,
                       float max_norm, float grad_scale, void* workspace, size_t workspace_bytes,
                       void* stream) {
    const char* fn = "ls_grad_norm";
    LS_TRY(check_size(fn, "count", count, 0, int64_t{1} << 24));
    if (!norm && !factor)
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: norm and factor are both NULL", fn);
    LS_TRY(check_ptr4(norm, "norm", false));
    LS_TRY(check_ptr4(factor, "factor", false));
    if (!(max_norm >= 0.f))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: max_norm = %g is not a number from 0 on", fn,
                    static_cast<double>(max_norm));
    if (!isfinite(grad_scale))
        return fail(LS_ERR_INVALID_ARGUMENT, "%s: grad_scale is not finite", fn);
    LS_TRY(check_tensors(fn, "grads", grads, count));
    const size_t need = ls::grad_norm_workspace_bytes();
    LS_TRY(check_workspace(fn, workspace, workspace_bytes, need));
    const Span outs[] = {{"norm", norm, 4}, {"factor", factor, 4}, {"workspace", workspace, need}};
    LS_TRY(check_disjoint(outs, 3, nullptr, 0));
    for (int64_t i = 0; i < count; ++i) {
        const Span in[] = {{"grads", grads[i].data, bytes_of(grads[i])}};
        LS_TRY(check_disjoint(outs, 3, in, 1));
    }
    return from_cuda(ls::launch_grad_norm(norm, factor, grads, count, max_norm, grad_scale, workspace,
                                          as_stream(stream)),
                     fn);
}

ls_status ls_scale_gradients(const ls_tensor* out, const ls_tensor* in, int64_t count,
                             const float* factor, void* stream) {
    const char* fn = "ls_scale_gradients";
    LS_TRY(check_size(fn, "count", count, 0, int64_t{1} << 24));
    LS_TRY(check_ptr4(factor, "factor", true));
    LS_TRY(check_tensors(fn, "out", out, count));
    LS_TRY(check_tensors(fn, "in", in, count));
    for (int64_t i = 0; i < count; ++i) {
        if (out[i].n != in[i].n || out[i].dtype != in[i].dtype)
            return fail(LS_ERR_INVALID_ARGUMENT, "%s: out[%lld] and in[%lld] differ in size or type", fn,
                        (long long)i, (long long)i);
        const Span o[] = {{"out", out[i].data, bytes_of(out[i])}};
        const Span n[] = {{"in", out[i].data == in[i].data ? nullptr : in[i].data, bytes_of(in[i])},
                          {"factor", factor, 4}};
        LS_TRY(check_disjoint(o, 1, n, 2));
    }
    return from_cuda(ls::launch_scale_gradients(out, in, count, factor, as_stream(stream)), fn);
}

ls_status ls_adam_update_scaled(ls_dtype dtype, void* param, const void* grad, float* exp_avg,
                                float* exp_avg_sq, int64_t n, float lr, float beta1, float beta2,
                                float eps, float weight_decay, int64_t step, const float* factor,
                                void* stream) {
    return run_adam("ls_adam_update_scaled", dtype, param, grad, exp_avg, exp_avg_sq, n,
                    {lr, beta1, beta2, eps, weight_decay, step, factor, nullptr}, stream);
}

ls_status ls_adam_update_clipped(ls_dtype dtype, void* param, const void* grad, float* exp_avg,
                                 float* exp_avg_sq, int64_t n, float lr, float beta1, float beta2,
                                 float eps, float weight_decay, int64_t step, const float* norm,
                                 const float* factor, void* stream) {
    LS_TRY(check_ptr4(norm, "norm", n > 0));
    return run_adam("ls_adam_update_clipped", dtype, param, grad, exp_avg, exp_avg_sq, n,
                    {lr, beta1, beta2, eps, weight_decay, step, factor, norm}, stream);
}

}  // extern "C"
#pragma GCC visibility pop
