// C ABI of the operators around the drafted tokens' step (declared in
// include/rope_chain.h): head norms with their rotation, rows of a cache in 4 bits,
// accepted rows moved.  Arguments are checked on the host, then the kernels go on the
// caller's stream; nothing here allocates device memory or synchronises.
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

// A cache in 4 bits: sizes and addresses.
static rc_status check_kv4(const char *fn, int64_t T, int32_t heads, const int64_t *slots, const uint8_t *cache4,
                           const uint16_t *scales, int32_t num_blocks, int32_t block_size, const int32_t *err)
{
    if (heads < 1 || T < 0 || T > 0x7FFFFFFFLL || T * heads > 0x7FFFFFFFLL)
        return fail(RC_ERR_INVALID_ARG, "%s: need T >= 0, num_kv_heads >= 1 and T*num_kv_heads < 2^31", fn);
    if (num_blocks < 1 || block_size < 1 || (int64_t)num_blocks * block_size >= (1LL << 31))
        return fail(RC_ERR_INVALID_ARG, "%s: need num_blocks, block_size >= 1 and num_blocks*block_size < 2^31", fn);
    if ((T > 0 && !slots) || !aligned(slots, 8))
        return fail(RC_ERR_INVALID_ARG, "%s: slots must be an 8-byte aligned pointer", fn);
    if (!cache4 || !aligned(cache4, 16) || !scales || !aligned(scales, 8))
        return fail(RC_ERR_INVALID_ARG, "%s: cache4 must be a 16-byte and scales an 8-byte aligned pointer", fn);
    if (!aligned(err, 4))
        return fail(RC_ERR_INVALID_ARG, "%s: err must be 4-byte aligned", fn);
    return RC_OK;
}

static Span kv4_span(const void *p, int32_t num_blocks, int32_t heads, int32_t block_size, size_t row) {
    return {p, (size_t)num_blocks * heads * block_size * row};
}

rc_status rc_kv4_store(const uint16_t *k, int64_t k_row_stride, int64_t k_head_stride, const uint16_t *v,
                       int64_t v_row_stride, int64_t v_head_stride, int64_t T, int32_t num_kv_heads,
                       const int64_t *slots, uint8_t *cache4, uint16_t *scales, int32_t num_blocks,
                       int32_t block_size, int32_t *err, cudaStream_t stream)
{
    const char *fn = "rc_kv4_store";
    const rc_status s = check_kv4(fn, T, num_kv_heads, slots, cache4, scales, num_blocks, block_size, err);
    if (s != RC_OK)
        return s;
    const HeadsView vk = heads_view(std::max<int64_t>(T, 1), k_row_stride, k_head_stride, num_kv_heads, kHeadDim);
    const HeadsView vv = heads_view(std::max<int64_t>(T, 1), v_row_stride, v_head_stride, num_kv_heads, kHeadDim);
    for (const int64_t x : {vk.row_stride, vk.head_stride, vv.row_stride, vv.head_stride})
        if (x < 0 || x > kMaxStride || x % 8 != 0)
            return fail(RC_ERR_INVALID_ARG, "%s: strides of k and v must be multiples of 8 in [0, 2^40]", fn);
    if ((T > 0 && (!k || !v)) || !aligned(k, 16) || !aligned(v, 16))
        return fail(RC_ERR_INVALID_ARG, "%s: k and v must be 16-byte aligned pointers", fn);
    if (T == 0)
        return ok();
    const Span cs = kv4_span(cache4, num_blocks, num_kv_heads, block_size, 64), ss = kv4_span(scales, num_blocks, num_kv_heads, block_size, 8);
    const Span ks = {k, (size_t)vk.elements() * 2}, vs = {v, (size_t)vv.elements() * 2}, at = {slots, (size_t)T * 8}, es = {err, 4};
    if (overlap(cs, {ss, ks, vs, at, es}) || overlap(ss, {ks, vs, at, es}))
        return fail(RC_ERR_INVALID_ARG, "%s: cache4 or scales overlaps another operand", fn);
    Kv4StoreLaunch a{};
    a.k = k;
    a.v = v;
    a.k_row_stride = vk.row_stride;
    a.k_head_stride = vk.head_stride;
    a.v_row_stride = vv.row_stride;
    a.v_head_stride = vv.head_stride;
    a.T = T;
    a.slots = slots;
    a.cache4 = cache4;
    a.scales = scales;
    a.capacity = (int64_t)num_blocks * block_size;
    a.heads = num_kv_heads;
    a.block_size = block_size;
    a.err = err;
    const cudaError_t e = launch_kv4_store(a, stream);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rc_kv4_store launch");
}

rc_status rc_kv4_load(const int64_t *slots, int64_t T, int32_t num_kv_heads, const uint8_t *cache4,
                      const uint16_t *scales, int32_t num_blocks, int32_t block_size, uint16_t *out,
                      int32_t *err, cudaStream_t stream)
{
    const char *fn = "rc_kv4_load";
    const rc_status s = check_kv4(fn, T, num_kv_heads, slots, cache4, scales, num_blocks, block_size, err);
    if (s != RC_OK)
        return s;
    if ((T > 0 && !out) || !aligned(out, 16))
        return fail(RC_ERR_INVALID_ARG, "%s: out must be a 16-byte aligned pointer", fn);
    if (T == 0)
        return ok();
    if (overlap({out, (size_t)T * num_kv_heads * 256},
                {kv4_span(cache4, num_blocks, num_kv_heads, block_size, 64),
                 kv4_span(scales, num_blocks, num_kv_heads, block_size, 8), {slots, (size_t)T * 8}, {err, 4}}))
        return fail(RC_ERR_INVALID_ARG, "%s: out overlaps another operand", fn);
    const Kv4LoadLaunch a = {slots, T, cache4, scales, (int64_t)num_blocks * block_size, num_kv_heads, block_size, out, err};
    const int sms = num_sms_current();
    if (sms <= 0)
        return fail(RC_ERR_CUDA, "%s: no current CUDA device", fn);
    const cudaError_t e = launch_kv4_load(a, sms, stream);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rc_kv4_load launch");
}

rc_status rc_kv_compact(void *const *caches, const int32_t *row_bytes, int32_t count, int32_t num_blocks,
                        int32_t num_kv_heads, int32_t block_size, const int32_t *block_table,
                        int64_t table_stride, int32_t table_width, const int32_t *context_len,
                        const int32_t *row_start, int32_t seqs, int64_t rows, const int32_t *path,
                        int64_t path_stride, int32_t path_width, const int32_t *path_len, int32_t *new_len,
                        int32_t *err, cudaStream_t stream)
{
    const char *fn = "rc_kv_compact";
    if (count < 1 || count > kMaxCompactCaches || !caches || !row_bytes)
        return fail(RC_ERR_INVALID_ARG, "%s: need 1 to %d caches with their row_bytes, not %d", fn, kMaxCompactCaches, count);
    if (num_kv_heads < 1 || num_kv_heads > 65536 || num_blocks < 1 || block_size < 1 ||
        (int64_t)num_blocks * block_size >= (1LL << 31))
        return fail(RC_ERR_INVALID_ARG, "%s: need num_kv_heads in [1, 65536], num_blocks, block_size >= 1 and "
                    "num_blocks*block_size < 2^31", fn);
    if (seqs < 1 || seqs >= (1 << 24) || rows < 0 || rows > 0x7FFFFFFFLL)
        return fail(RC_ERR_INVALID_ARG, "%s: need 1 <= seqs < 2^24 and 0 <= rows < 2^31", fn);
    if (table_width < 0 || table_stride < 0 || table_stride > kMaxStride || (int64_t)table_width * block_size >= (1LL << 31) ||
        path_width < 0 || path_stride < 0 || path_stride > kMaxStride)
        return fail(RC_ERR_INVALID_ARG, "%s: need table_width, table_stride, path_width, path_stride >= 0 and "
                    "table_width*block_size < 2^31", fn);
    if (!row_start || !context_len || !path_len || (path_width > 0 && !path) || (table_width > 0 && !block_table) ||
        !aligned(row_start, 4) || !aligned(context_len, 4) || !aligned(path_len, 4) || !aligned(path, 4) ||
        !aligned(block_table, 4) || !aligned(new_len, 4) || !aligned(err, 4))
        return fail(RC_ERR_INVALID_ARG, "%s: row_start, context_len, block_table, path and path_len must be 4-byte aligned "
                    "pointers, new_len and err 4-byte aligned", fn);
    CompactLaunch a{};
    Span spans[kMaxCompactCaches];
    for (int i = 0; i < count; ++i) {
        const int32_t n = row_bytes[i];
        if (n < 8 || n % 8 != 0 || n > 4096)
            return fail(RC_ERR_INVALID_ARG, "%s: row_bytes[%d]=%d is not a multiple of 8 in [8, 4096]", fn, i, n);
        if (!caches[i] || !aligned(caches[i], n % 16 == 0 ? 16 : 8))
            return fail(RC_ERR_INVALID_ARG, "%s: caches[%d] must be a 16-byte aligned pointer (8 where its row_bytes are no "
                        "multiple of 16)", fn, i);
        spans[i] = {caches[i], (size_t)num_blocks * num_kv_heads * block_size * n};
        a.caches[i] = caches[i];
        a.row_bytes[i] = n;
    }
    const Span table_span = {block_table, table_width > 0 ? (size_t)((seqs - 1) * table_stride + table_width) * 4 : (size_t)0};
    const Span path_span = {path, path_width > 0 ? (size_t)((seqs - 1) * path_stride + path_width) * 4 : (size_t)0};
    const Span start_span = {row_start, ((size_t)seqs + 1) * 4}, len_span = {context_len, (size_t)seqs * 4};
    const Span count_span = {path_len, (size_t)seqs * 4}, new_span = {new_len, (size_t)seqs * 4}, err_span = {err, 4};
    for (int i = 0; i < count; ++i) {
        if (overlap(spans[i], {table_span, path_span, start_span, len_span, count_span, new_span, err_span}))
            return fail(RC_ERR_INVALID_ARG, "%s: caches[%d] overlaps another operand", fn, i);
        for (int j = 0; j < i; ++j)
            if (overlap(spans[i], {spans[j]}))
                return fail(RC_ERR_INVALID_ARG, "%s: caches[%d] and caches[%d] overlap", fn, j, i);
    }
    if (overlap(new_span, {table_span, path_span, start_span, len_span, count_span, err_span}))
        return fail(RC_ERR_INVALID_ARG, "%s: new_len overlaps an operand that is read, or err", fn);
    a.count = count;
    a.num_blocks = num_blocks;
    a.heads = num_kv_heads;
    a.block_size = block_size;
    a.seqs = seqs;
    a.block_table = block_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.context_len = context_len;
    a.row_start = row_start;
    a.rows = rows;
    a.path = path;
    a.path_stride = path_stride;
    a.path_width = path_width;
    a.path_len = path_len;
    a.new_len = new_len;
    a.err = err;
    const cudaError_t e = launch_kv_compact(a, stream);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rc_kv_compact launch");
}

}  // extern "C"
