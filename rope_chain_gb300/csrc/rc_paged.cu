// C ABI of the operators around the drafted tokens' step (declared in
// include/rope_chain.h): head norms with their rotation.  Arguments are checked on
// the host, then the kernels go on the caller's stream; nothing here allocates
// device memory or synchronises.
#include "rope_chain.h"
#include "rc_checks.cuh"
#include "rc_paged.cuh"

#include <algorithm>
#include <cmath>

using namespace rc;

namespace {

// The checks that both directions of the head norm share.  `views`: x, out and
// (gradient) dy; out is the one written.
rc_status check_head_norm(const char *fn, int32_t dtype, int64_t T, int32_t heads, int32_t head_dim,
                          const rc_head_norm_params *params, const int64_t *positions, const void *cos_sin,
                          int32_t table_dtype, int64_t max_position, int32_t rot_dim, int32_t layout,
                          std::initializer_list<const void *> tensors, std::initializer_list<int64_t> strides,
                          const int32_t *err)
{
    if ((dtype != RC_BF16 && dtype != RC_F32) || (table_dtype != RC_BF16 && table_dtype != RC_F32))
        return fail(RC_ERR_INVALID_ARG, "%s: unknown dtype %d or table dtype %d", fn, dtype, table_dtype);
    if (layout != RC_ROPE_PAIRS && layout != RC_ROPE_HALVES)
        return fail(RC_ERR_INVALID_ARG, "%s: unknown layout %d", fn, layout);
    if (T < 0 || heads < 1 || T > 0x7FFFFFFFLL || T * heads > 0x7FFFFFFFLL)
        return fail(RC_ERR_INVALID_ARG, "%s: need T >= 0, heads >= 1 and T*heads < 2^31", fn);
    if (head_dim < 2 || head_dim > kMaxNormDim || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > head_dim)
        return fail(RC_ERR_UNSUPPORTED, "%s: head_dim=%d, rot_dim=%d: need a head_dim in [2, %d] and an even rot_dim in "
                    "[2, head_dim]", fn, head_dim, rot_dim, kMaxNormDim);
    if (layout == RC_ROPE_PAIRS && head_dim % 2 != 0)
        return fail(RC_ERR_UNSUPPORTED, "%s: the pairs layout needs an even head_dim, not %d", fn, head_dim);
    if (!params || params->q_heads < 0 || params->q_heads > heads)
        return fail(RC_ERR_INVALID_ARG, "%s: params must not be NULL and q_heads in [0, heads]", fn);
    if (!(params->eps >= 0.0f) || !std::isfinite(params->eps))
        return fail(RC_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    if (params->q_weight || params->k_weight) {
        if (params->weight_dtype != RC_BF16 && params->weight_dtype != RC_F32)
            return fail(RC_ERR_INVALID_ARG, "%s: unknown weight dtype %d", fn, params->weight_dtype);
        const int size = size_of(params->weight_dtype);
        if (!aligned(params->q_weight, size) || !aligned(params->k_weight, size))
            return fail(RC_ERR_INVALID_ARG, "%s: weights must be aligned to their element", fn);
    }
    for (const int64_t s : strides)
        if (s < 0 || s > kMaxStride)
            return fail(RC_ERR_INVALID_ARG, "%s: strides outside [0, 2^40]", fn);
    for (const void *p : tensors)           // (an empty tensor may have no address)
        if ((T > 0 && !p) || !aligned(p, size_of(dtype)))
            return fail(RC_ERR_INVALID_ARG, "%s: x, out and gradients must be pointers aligned to their element", fn);
    if ((T > 0 && !positions) || !aligned(positions, 8))
        return fail(RC_ERR_INVALID_ARG, "%s: positions must be an 8-byte aligned pointer", fn);
    if (!cos_sin || !aligned(cos_sin, size_of(table_dtype)) || max_position < 1)
        return fail(RC_ERR_INVALID_ARG, "%s: cos_sin must be an aligned pointer with max_position >= 1", fn);
    if (!aligned(err, 4))
        return fail(RC_ERR_INVALID_ARG, "%s: err must be 4-byte aligned", fn);
    return RC_OK;
}

// What both directions read beside x (and dy).
struct NormReads {
    Span positions, table, q_weight, k_weight, err;
};

NormReads norm_reads(int64_t T, int32_t head_dim, const rc_head_norm_params &p, const int64_t *positions,
                     const void *cos_sin, int32_t table_dtype, int64_t max_position, int32_t rot_dim, const int32_t *err) {
    const size_t weight = (size_t)head_dim * size_of(p.weight_dtype);
    return {{positions, (size_t)T * 8}, {cos_sin, (size_t)max_position * rot_dim * size_of(table_dtype)},
            {p.q_weight, weight}, {p.k_weight, weight}, {err, 4}};
}

bool over(const Span &written, const NormReads &r) {
    return overlap(written, {r.positions, r.table, r.q_weight, r.k_weight, r.err});
}

// Whether `a` over `b` is the same view.
bool same_view(const void *a, const HeadsView &va, const void *b, const HeadsView &vb) {
    return a == b && va.row_stride == vb.row_stride && va.head_stride == vb.head_stride;
}

HeadNormLaunch norm_launch(int64_t T, int32_t heads, int32_t head_dim, const rc_head_norm_params &p,
                           const int64_t *positions, const void *cos_sin, int32_t table_dtype, int64_t max_position,
                           int32_t rot_dim, int32_t *err) {
    HeadNormLaunch a{};
    a.weight[0] = p.q_weight;
    a.weight[1] = p.k_weight;
    a.weight_f32 = p.weight_dtype == RC_F32;
    a.positions = positions;
    a.table = cos_sin;
    a.table_f32 = table_dtype == RC_F32;
    a.max_position = max_position;
    a.T = T;
    a.heads = heads;
    a.q_heads = p.q_heads;
    a.width = head_dim;
    a.rot = rot_dim;
    a.eps = p.eps;
    a.err = err;
    return a;
}

// 16-byte accesses: every pointer, and what leads from one access to the next.
bool norm_wide(int32_t dtype, int32_t head_dim, int32_t rot_dim, int32_t layout, const rc_head_norm_params &p,
               const void *cos_sin, std::initializer_list<const void *> tensors, std::initializer_list<HeadsView> views) {
    const int vec = 16 / size_of(dtype);
    bool wide = aligned(cos_sin, 16) && aligned(p.q_weight, 16) && aligned(p.k_weight, 16) && head_dim % vec == 0 &&
                rot_dim % (layout == RC_ROPE_HALVES ? 2 * vec : vec) == 0;
    for (const void *t : tensors)
        wide = wide && aligned(t, 16);
    for (const HeadsView &v : views)
        wide = wide && (v.row_stride | v.head_stride) % vec == 0;
    return wide;
}

}  // namespace

extern "C" {

rc_status rc_head_norm_rope(const void *x, int32_t dtype, int64_t x_row_stride, int64_t x_head_stride,
                            int64_t T, int32_t heads, int32_t head_dim, const rc_head_norm_params *params,
                            const int64_t *positions, const void *cos_sin, int32_t table_dtype,
                            int64_t max_position, int32_t rot_dim, int32_t layout, void *out,
                            int64_t out_row_stride, int64_t out_head_stride, int32_t *err,
                            cudaStream_t stream)
{
    const char *fn = "rc_head_norm_rope";
    const rc_status s = check_head_norm(fn, dtype, T, heads, head_dim, params, positions, cos_sin, table_dtype, max_position,
                                        rot_dim, layout, {x, out},
                                        {x_row_stride, x_head_stride, out_row_stride, out_head_stride}, err);
    if (s != RC_OK)
        return s;
    if (T == 0)
        return ok();
    const int size = size_of(dtype);
    const HeadsView vx = heads_view(T, x_row_stride, x_head_stride, heads, head_dim);
    const HeadsView vo = heads_view(T, out_row_stride, out_head_stride, heads, head_dim);
    if (!vo.distinct())
        return fail(RC_ERR_INVALID_ARG, "%s: elements of out overlap one another", fn);
    const Span xs = {x, (size_t)vx.elements() * size}, os = {out, (size_t)vo.elements() * size};
    if (!same_view(x, vx, out, vo) && overlap(os, {xs}))
        return fail(RC_ERR_INVALID_ARG, "%s: out overlaps x and is not x itself", fn);
    if (over(os, norm_reads(T, head_dim, *params, positions, cos_sin, table_dtype, max_position, rot_dim, err)))
        return fail(RC_ERR_INVALID_ARG, "%s: out overlaps positions, cos_sin, a weight or err", fn);
    HeadNormLaunch a = norm_launch(T, heads, head_dim, *params, positions, cos_sin, table_dtype, max_position, rot_dim, err);
    a.x = x;
    a.x_row_stride = vx.row_stride;
    a.x_head_stride = vx.head_stride;
    a.out = out;
    a.out_row_stride = vo.row_stride;
    a.out_head_stride = vo.head_stride;
    const int sms = num_sms_current();
    if (sms <= 0)
        return fail(RC_ERR_CUDA, "%s: no current CUDA device", fn);
    const cudaError_t e = launch_head_norm_rope(a, dtype == RC_F32, layout == RC_ROPE_HALVES,
                                                norm_wide(dtype, head_dim, rot_dim, layout, *params, cos_sin, {x, out}, {vx, vo}),
                                                sms, stream);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rc_head_norm_rope launch");
}

size_t rc_head_norm_rope_grad_workspace_size(int32_t head_dim)
{
    if (head_dim < 2 || head_dim > kMaxNormDim)
        return 0;
    const int sms = num_sms_current();
    return sms > 0 ? head_norm_grad_workspace(head_dim, sms) : 0;
}

rc_status rc_head_norm_rope_grad(const void *dy, int64_t dy_row_stride, int64_t dy_head_stride,
                                 const void *x, int32_t dtype, int64_t x_row_stride,
                                 int64_t x_head_stride, int64_t T, int32_t heads, int32_t head_dim,
                                 const rc_head_norm_params *params, const int64_t *positions,
                                 const void *cos_sin, int32_t table_dtype, int64_t max_position,
                                 int32_t rot_dim, int32_t layout, void *dx, int64_t dx_row_stride,
                                 int64_t dx_head_stride, float *dq_weight, float *dk_weight,
                                 void *workspace, size_t workspace_bytes, int32_t *err,
                                 cudaStream_t stream)
{
    const char *fn = "rc_head_norm_rope_grad";
    const rc_status s = check_head_norm(fn, dtype, T, heads, head_dim, params, positions, cos_sin, table_dtype, max_position,
                                        rot_dim, layout, {dy, x, dx},
                                        {dy_row_stride, dy_head_stride, x_row_stride, x_head_stride, dx_row_stride,
                                         dx_head_stride}, err);
    if (s != RC_OK)
        return s;
    const bool weights = dq_weight || dk_weight;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || (workspace && !aligned(workspace, 16)))
        return fail(RC_ERR_INVALID_ARG, "%s: gradients of weights must be 4-byte and the workspace 16-byte aligned", fn);
    if (weights && !workspace)
        return fail(RC_ERR_INVALID_ARG, "%s: gradients of weights need a workspace", fn);
    if (T == 0 && !weights)
        return ok();
    const int size = size_of(dtype);
    const HeadsView vd = heads_view(T, dy_row_stride, dy_head_stride, heads, head_dim);
    const HeadsView vx = heads_view(T, x_row_stride, x_head_stride, heads, head_dim);
    const HeadsView vo = heads_view(T, dx_row_stride, dx_head_stride, heads, head_dim);
    if (T > 0 && !vo.distinct())
        return fail(RC_ERR_INVALID_ARG, "%s: elements of dx overlap one another", fn);
    auto span = [&](const void *p, const HeadsView &v) { return Span{p, T > 0 ? (size_t)v.elements() * size : (size_t)0}; };
    const Span ds = span(dy, vd), xs = span(x, vx), os = span(dx, vo);
    const NormReads reads = norm_reads(T, head_dim, *params, positions, cos_sin, table_dtype, max_position, rot_dim, err);
    if ((!same_view(x, vx, dx, vo) && overlap(os, {xs})) || (!same_view(dy, vd, dx, vo) && overlap(os, {ds})) || over(os, reads))
        return fail(RC_ERR_INVALID_ARG, "%s: dx overlaps an operand and is not dy or x itself", fn);
    const Span dq = {dq_weight, (size_t)head_dim * 4}, dk = {dk_weight, (size_t)head_dim * 4};
    for (const Span &w : {dq, dk})
        if (overlap(w, {ds, xs, os}) || over(w, reads))
            return fail(RC_ERR_INVALID_ARG, "%s: a weight's gradient overlaps another operand", fn);
    if (overlap(dq, {dk}))
        return fail(RC_ERR_INVALID_ARG, "%s: the weights' gradients overlap", fn);
    const int sms = num_sms_current();
    if (sms <= 0)
        return fail(RC_ERR_CUDA, "%s: no current CUDA device", fn);
    if (weights) {
        const size_t need = head_norm_grad_workspace(head_dim, sms);
        if (workspace_bytes < need)
            return fail(RC_ERR_INVALID_ARG, "%s: the workspace holds %zu bytes, these sizes take %zu", fn, workspace_bytes, need);
        const Span ws = {workspace, need};
        if (overlap(ws, {ds, xs, os, dq, dk}) || over(ws, reads))
            return fail(RC_ERR_INVALID_ARG, "%s: the workspace overlaps an operand", fn);
    }
    HeadNormLaunch a = norm_launch(T, heads, head_dim, *params, positions, cos_sin, table_dtype, max_position, rot_dim, err);
    // (with T == 0 nothing but the weights' gradients is looked at)
    a.dy = dy ? dy : workspace;
    a.x = x;
    a.out = dx;
    a.dy_row_stride = vd.row_stride;
    a.dy_head_stride = vd.head_stride;
    a.x_row_stride = vx.row_stride;
    a.x_head_stride = vx.head_stride;
    a.out_row_stride = vo.row_stride;
    a.out_head_stride = vo.head_stride;
    a.dweight[0] = dq_weight;
    a.dweight[1] = dk_weight;
    a.partial = static_cast<float *>(workspace);
    const cudaError_t e = launch_head_norm_rope(a, dtype == RC_F32, layout == RC_ROPE_HALVES,
                                                norm_wide(dtype, head_dim, rot_dim, layout, *params, cos_sin, {dy, x, dx},
                                                          {vd, vx, vo}), sms, stream);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rc_head_norm_rope_grad launch");
}

}  // extern "C"
