// C ABI of the drafted tokens' operators (declared in include/rope_chain.h):
// rotary positions, attention over the paged caches, logits adjustment.
// Arguments are checked on the host, then the kernels go on the caller's
// stream; nothing here allocates device memory or synchronises.
#include "rope_chain.h"
#include "rc_draft.cuh"
#include "rc_checks.cuh"

#include <algorithm>
#include <cmath>

using namespace rc;

namespace {

// Rows times heads of an attention: a row's index is 32 bits, that of the last
// row tile's end (up to 256 rows) included.
constexpr int64_t kMaxAttentionRows = 0x7FFFFFFFLL - 256;

// The attention calls: `a` as the entry points fill it in (group and partial apart).
rc_status attend(const char *fn, TreeAttentionLaunch a, int32_t num_heads, void *workspace, size_t workspace_bytes,
                 cudaStream_t stream)
{
    const bool four = a.cache4 != nullptr;
    if (a.kv_heads < 1 || num_heads < a.kv_heads || num_heads % a.kv_heads != 0)
        return fail(RC_ERR_INVALID_ARG, "%s: num_heads=%d is not a positive multiple of num_kv_heads=%d",
                    fn, num_heads, a.kv_heads);
    if (a.rows < 0 || a.rows > kMaxAttentionRows / num_heads)
        return fail(RC_ERR_INVALID_ARG, "%s: need rows >= 0 and rows*num_heads < 2^31 - 256", fn);
    if (a.seqs < 1 || a.seqs >= (1 << 24))
        return fail(RC_ERR_INVALID_ARG, "%s: seqs=%d outside [1, 2^24)", fn, a.seqs);
    if (a.num_blocks < 1 || a.block_size < 1 || (int64_t)a.num_blocks * a.block_size >= (1LL << 31))
        return fail(RC_ERR_INVALID_ARG,
                    "%s: need num_blocks, block_size >= 1 and num_blocks*block_size < 2^31", fn);
    // a logical key is a 32-bit index, a tile's end included
    if (a.table_width < 0 || a.table_stride < 0 || a.table_stride > kMaxStride ||
        (int64_t)a.table_width * a.block_size >= (1LL << 31) - 4096)
        return fail(RC_ERR_INVALID_ARG, "%s: need table_width, table_stride >= 0 and table_width*block_size "
                    "< 2^31 - 4096", fn);
    if (!(a.scale > 0.0f) || !std::isfinite(a.scale))
        return fail(RC_ERR_INVALID_ARG, "%s: scale must be positive and finite", fn);
    const void *cache = four ? static_cast<const void *>(a.cache4) : a.cache;
    if ((a.rows > 0 && (!a.q || !a.out)) || !cache || !aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(cache, 16))
        return fail(RC_ERR_INVALID_ARG, "%s: q, out and the cache must be 16-byte aligned pointers", fn);
    if (four && (!a.scales || !aligned(a.scales, 8)))
        return fail(RC_ERR_INVALID_ARG, "%s: scales must be an 8-byte aligned pointer", fn);
    if (!a.row_start || !a.context_len || !aligned(a.row_start, 4) || !aligned(a.context_len, 4) ||
        (a.table_width > 0 && (!a.block_table || !aligned(a.block_table, 4))))
        return fail(RC_ERR_INVALID_ARG, "%s: row_start, context_len and block_table must be 4-byte "
                    "aligned pointers", fn);
    if (a.tree_mask && (!aligned(a.tree_mask, 8) || a.mask_words < 1))
        return fail(RC_ERR_INVALID_ARG, "%s: tree_mask must be 8-byte aligned with mask_words >= 1", fn);
    const int64_t width = 64LL * num_heads;
    if (a.rows <= 1)                    // the stride of an axis of length one is never used
        a.q_row_stride = a.out_row_stride = 0;
    if (a.q_row_stride % 8 != 0 || a.out_row_stride % 8 != 0 || a.q_row_stride < 0 || a.q_row_stride > kMaxStride ||
        a.out_row_stride > kMaxStride || (a.rows > 1 && a.out_row_stride < width) || a.out_row_stride < 0)
        return fail(RC_ERR_INVALID_ARG, "%s: row strides must be non-negative multiples of 8, and out's "
                    "at least 64*num_heads", fn);
    if ((a.lse && !aligned(a.lse, 4)) || (workspace && !aligned(workspace, 16)))
        return fail(RC_ERR_INVALID_ARG, "%s: lse must be 4-byte and the workspace 16-byte aligned", fn);
    if (a.rows == 0)
        return ok();
    const size_t out_bytes = ((a.rows - 1) * a.out_row_stride + width) * 2;
    const Span out_span = {a.out, out_bytes}, lse_span = {a.lse, (size_t)a.rows * num_heads * 4};
    const Span q_span = {a.q, (size_t)((a.rows - 1) * a.q_row_stride + width) * 2};
    const size_t keys = (size_t)a.num_blocks * a.kv_heads * a.block_size;
    const Span cache_span = {cache, keys * (four ? 64 : 256)}, scales_span = {a.scales, keys * 8};
    const Span start_span = {a.row_start, ((size_t)a.seqs + 1) * 4}, len_span = {a.context_len, (size_t)a.seqs * 4};
    const Span table_span = {a.block_table,
                             a.table_width > 0 ? (size_t)((a.seqs - 1) * a.table_stride + a.table_width) * 4 : (size_t)0};
    const Span mask_span = {a.tree_mask, (size_t)a.rows * a.mask_words * 8}, err_span = {a.err, 4};
    auto reads = [&](const Span &written) {
        return overlap(written, {q_span, cache_span, scales_span, start_span, len_span, table_span, mask_span, err_span});
    };
    if (reads(out_span) || reads(lse_span) || overlap(lse_span, {out_span}) || !aligned(a.err, 4))
        return fail(RC_ERR_INVALID_ARG, "%s: out or lse overlaps another operand, or err is not 4-byte aligned", fn);
    const int sms = num_sms_current();
    if (sms <= 0)
        return fail(RC_ERR_CUDA, "%s: no current CUDA device", fn);
    a.group = num_heads / a.kv_heads;
    if (workspace) {
        const size_t need = four ? kv4_attention_workspace(a.rows, a.seqs, a.group, sms)
                                 : tree_attention_workspace(a.rows, a.seqs, a.group, sms);
        if (workspace_bytes < need)
            return fail(RC_ERR_INVALID_ARG, "%s: the workspace holds %zu bytes, these sizes take %zu", fn,
                        workspace_bytes, need);
        if (reads({workspace, need}) || overlap({workspace, need}, {out_span, lse_span}))
            return fail(RC_ERR_INVALID_ARG, "%s: the workspace overlaps an operand", fn);
    }
    a.partial = static_cast<float *>(workspace);
    const char *why = "launch";
    const cudaError_t e = four ? launch_kv4_attention(a, sms, stream, &why) : launch_tree_attention(a, sms, stream, &why);
    return e == cudaSuccess ? ok() : cuda_fail(e, why);
}

// The operands that the attention calls have in common.
TreeAttentionLaunch attention_launch(const uint16_t *q, int64_t q_row_stride, int64_t rows, int32_t num_kv_heads,
                                     const int32_t *row_start, int32_t seqs, const int32_t *context_len,
                                     const int32_t *block_table, int64_t table_stride, int32_t table_width,
                                     const uint64_t *tree_mask, int32_t mask_words, int32_t num_blocks,
                                     int32_t block_size, float scale, uint16_t *out, int64_t out_row_stride, float *lse,
                                     int32_t *err)
{
    TreeAttentionLaunch a{};
    a.q = q;
    a.q_row_stride = q_row_stride;
    a.rows = rows;
    a.kv_heads = num_kv_heads;
    a.seqs = seqs;
    a.row_start = row_start;
    a.context_len = context_len;
    a.block_table = block_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.tree_mask = tree_mask;
    a.mask_words = mask_words;
    a.num_blocks = num_blocks;
    a.block_size = block_size;
    a.scale = scale;
    a.out = out;
    a.out_row_stride = out_row_stride;
    a.lse = lse;
    a.err = err;
    return a;
}

// Sizes for which an attention has a workspace.
bool attention_sizes(int64_t rows, int32_t seqs, int32_t num_heads, int32_t num_kv_heads) {
    return rows >= 1 && seqs >= 1 && num_kv_heads >= 1 && num_heads >= num_kv_heads && num_heads % num_kv_heads == 0 &&
           rows <= kMaxAttentionRows / num_heads;
}

}  // namespace

extern "C" {

rc_status rc_rope_table(void *out, int32_t dtype, int64_t max_position, int32_t rot_dim,
                        double theta, const rc_rope_scaling *scaling, cudaStream_t stream)
{
    const char *fn = "rc_rope_table";
    if (dtype != RC_BF16 && dtype != RC_F32)
        return fail(RC_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
    if (max_position < 0 || max_position > 0x7FFFFFFFLL)
        return fail(RC_ERR_INVALID_ARG, "%s: max_position=%lld outside [0, 2^31)", fn,
                    (long long)max_position);
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > rc::kMaxRotDim)
        return fail(RC_ERR_UNSUPPORTED, "%s: rot_dim=%d is not even in [2, %d]", fn, rot_dim,
                    rc::kMaxRotDim);
    if (!(theta > 1.0) || !std::isfinite(theta))
        return fail(RC_ERR_INVALID_ARG, "%s: theta must be finite and above 1", fn);
    const rc_rope_scaling none = {RC_ROPE_SCALE_NONE, 1.0, 1.0, 32.0, 1.0, 1.0};
    const rc_rope_scaling &sc = scaling ? *scaling : none;
    if (sc.kind < RC_ROPE_SCALE_NONE || sc.kind > RC_ROPE_SCALE_PARTS)
        return fail(RC_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, sc.kind);
    if (sc.kind != RC_ROPE_SCALE_NONE && (!(sc.factor > 0.0) || !std::isfinite(sc.factor)))
        return fail(RC_ERR_INVALID_ARG, "%s: factor must be positive and finite", fn);
    if (!std::isfinite(sc.attention_factor))
        return fail(RC_ERR_INVALID_ARG, "%s: attention_factor must be finite", fn);
    if (sc.kind == RC_ROPE_SCALE_BASE && rot_dim < 4)
        return fail(RC_ERR_UNSUPPORTED, "%s: base scaling needs rot_dim >= 4", fn);
    if (sc.kind == RC_ROPE_SCALE_PARTS &&
        (!(sc.original_max_position > 0.0) || !std::isfinite(sc.original_max_position) ||
         !(sc.beta_slow > 0.0) || !(sc.beta_fast > sc.beta_slow) || !std::isfinite(sc.beta_fast)))
        return fail(RC_ERR_INVALID_ARG, "%s: scaling by parts needs original_max_position > 0 and "
                    "beta_fast > beta_slow > 0", fn);
    if ((max_position > 0 && !out) || !aligned(out, 16))
        return fail(RC_ERR_INVALID_ARG, "%s: out must be a 16-byte aligned pointer", fn);
    if (max_position == 0)
        return ok();

    double inv[rc::kMaxRotDim / 2];
    const double base = sc.kind == RC_ROPE_SCALE_BASE
                            ? theta * std::pow(sc.factor, rot_dim / (rot_dim - 2.0)) : theta;
    if (!(base > 0.0) || !std::isfinite(base))
        return fail(RC_ERR_INVALID_ARG, "%s: the scaled theta is not positive and finite", fn);
    double lo = 0.0, hi = 0.0;
    if (sc.kind == RC_ROPE_SCALE_PARTS) {
        const double two_pi = 6.283185307179586476925;
        auto column = [&](double beta) {
            return rot_dim * std::log(sc.original_max_position / (beta * two_pi)) / (2.0 * std::log(theta));
        };
        lo = std::max(std::floor(column(sc.beta_fast)), 0.0);
        hi = std::min(std::ceil(column(sc.beta_slow)), rot_dim - 1.0);
    }
    for (int j = 0; j < rot_dim / 2; ++j) {
        inv[j] = std::pow(base, -2.0 * j / rot_dim);
        if (sc.kind == RC_ROPE_SCALE_LINEAR)
            inv[j] /= sc.factor;
        if (sc.kind == RC_ROPE_SCALE_PARTS) {
            const double ramp = std::min(1.0, std::max(0.0, (j - lo) / std::max(hi - lo, 1e-3)));
            inv[j] = inv[j] * (1.0 - ramp) + inv[j] / sc.factor * ramp;
        }
        if (!std::isfinite(inv[j]))
            return fail(RC_ERR_INVALID_ARG, "%s: a frequency is not finite", fn);
    }
    const int sms = num_sms_current();
    if (sms <= 0)
        return fail(RC_ERR_CUDA, "%s: no current CUDA device", fn);
    const cudaError_t e = rc::launch_rope_table(out, dtype == RC_F32, max_position, rot_dim, inv,
                                                (float)sc.attention_factor, sms, stream);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rc_rope_table launch");
}

rc_status rc_rope_apply(const void *x, int32_t dtype, int64_t x_row_stride, int64_t x_head_stride,
                        int64_t T, int32_t heads, int32_t head_dim, const int64_t *positions,
                        const void *cos_sin, int32_t table_dtype, int64_t max_position,
                        int32_t rot_dim, int32_t layout, int32_t inverse, void *out,
                        int64_t out_row_stride, int64_t out_head_stride, int32_t *err,
                        cudaStream_t stream)
{
    const char *fn = "rc_rope_apply";
    if ((dtype != RC_BF16 && dtype != RC_F32) || (table_dtype != RC_BF16 && table_dtype != RC_F32))
        return fail(RC_ERR_INVALID_ARG, "%s: unknown dtype %d or table dtype %d", fn, dtype, table_dtype);
    if (layout != RC_ROPE_PAIRS && layout != RC_ROPE_HALVES)
        return fail(RC_ERR_INVALID_ARG, "%s: unknown layout %d", fn, layout);
    if (T < 0 || heads < 1 || T > 0x7FFFFFFFLL || T * heads > 0x7FFFFFFFLL)
        return fail(RC_ERR_INVALID_ARG, "%s: need T >= 0, heads >= 1 and T*heads < 2^31", fn);
    if (head_dim < 2 || head_dim > 65536 || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > head_dim ||
        rot_dim > rc::kMaxRotDim)
        return fail(RC_ERR_UNSUPPORTED, "%s: head_dim=%d, rot_dim=%d: need an even rot_dim in [2, "
                    "min(head_dim, %d)]", fn, head_dim, rot_dim, rc::kMaxRotDim);
    if (layout == RC_ROPE_PAIRS && head_dim % 2 != 0)
        return fail(RC_ERR_UNSUPPORTED, "%s: the pairs layout needs an even head_dim, not %d", fn, head_dim);
    if (x_row_stride < 0 || x_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0 ||
        std::max(std::max(x_row_stride, x_head_stride), std::max(out_row_stride, out_head_stride)) > kMaxStride)
        return fail(RC_ERR_INVALID_ARG, "%s: strides outside [0, 2^40]", fn);
    const int size = size_of(dtype), table_size = size_of(table_dtype);
    // (an empty tensor may have no address)
    if ((T > 0 && (!x || !out)) || !aligned(x, size) || !aligned(out, size))
        return fail(RC_ERR_INVALID_ARG, "%s: x and out must be pointers aligned to their element", fn);
    if ((T > 0 && !positions) || !aligned(positions, 8))
        return fail(RC_ERR_INVALID_ARG, "%s: positions must be an 8-byte aligned pointer", fn);
    if (!cos_sin || !aligned(cos_sin, table_size) || max_position < 1)
        return fail(RC_ERR_INVALID_ARG, "%s: cos_sin must be an aligned pointer with max_position >= 1", fn);
    if (T == 0)
        return ok();
    // strides of an axis of length one are never used
    if (T == 1)
        x_row_stride = out_row_stride = 0;
    if (heads == 1)
        x_head_stride = out_head_stride = 0;
    const int64_t out_heads = (heads - 1) * out_head_stride + head_dim;
    const int64_t out_tokens = (T - 1) * out_row_stride + head_dim;
    const bool tokens_outer = (heads == 1 || out_head_stride >= head_dim) && (T == 1 || out_row_stride >= out_heads);
    const bool heads_outer = (T == 1 || out_row_stride >= head_dim) && (heads == 1 || out_head_stride >= out_tokens);
    if (!tokens_outer && !heads_outer)
        return fail(RC_ERR_INVALID_ARG, "%s: elements of out overlap one another", fn);
    const size_t x_span = ((T - 1) * x_row_stride + (heads - 1) * x_head_stride + head_dim) * (size_t)size;
    const size_t out_span = ((T - 1) * out_row_stride + (heads - 1) * out_head_stride + head_dim) * (size_t)size;
    const bool in_place = x == out && x_row_stride == out_row_stride && x_head_stride == out_head_stride;
    if (!in_place && overlap(x, x_span, out, out_span))
        return fail(RC_ERR_INVALID_ARG, "%s: out overlaps x and is not x itself", fn);
    if (!aligned(err, 4) ||
        overlap({out, out_span}, {{positions, (size_t)T * 8}, {cos_sin, (size_t)max_position * rot_dim * table_size},
                                  {err, 4}}))
        return fail(RC_ERR_INVALID_ARG, "%s: out overlaps positions, cos_sin or err, or err is not 4-byte aligned", fn);
    const int vec = 16 / size;
    const bool wide = aligned(x, 16) && aligned(out, 16) && aligned(cos_sin, 16) &&
                      (x_row_stride | x_head_stride | out_row_stride | out_head_stride | (int64_t)head_dim) % vec == 0 &&
                      rot_dim % (layout == RC_ROPE_HALVES ? 2 * vec : vec) == 0;
    rc::RopeLaunch a{};
    a.x = x;
    a.out = out;
    a.x_row_stride = x_row_stride;
    a.x_head_stride = x_head_stride;
    a.out_row_stride = out_row_stride;
    a.out_head_stride = out_head_stride;
    a.positions = positions;
    a.table = cos_sin;
    a.max_position = max_position;
    a.T = T;
    a.heads = heads;
    a.width = head_dim;
    a.rot = rot_dim;
    a.err = err;
    const int sms = num_sms_current();
    if (sms <= 0)
        return fail(RC_ERR_CUDA, "%s: no current CUDA device", fn);
    const cudaError_t e = rc::launch_rope_apply(a, dtype == RC_F32, table_dtype == RC_F32,
                                                layout == RC_ROPE_HALVES, inverse != 0, wide, sms, stream);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rc_rope_apply launch");
}

size_t rc_tree_attention_workspace_size(int64_t rows, int32_t seqs, int32_t num_heads,
                                        int32_t num_kv_heads)
{
    if (!attention_sizes(rows, seqs, num_heads, num_kv_heads))
        return 0;
    const int sms = num_sms_current();
    return sms > 0 ? tree_attention_workspace(rows, seqs, num_heads / num_kv_heads, sms) : 0;
}

rc_status rc_tree_attention(const uint16_t *q, int64_t q_row_stride, int64_t rows, int32_t num_heads,
                            int32_t num_kv_heads, const int32_t *row_start, int32_t seqs,
                            const int32_t *context_len, const int32_t *block_table,
                            int64_t table_stride, int32_t table_width, const uint64_t *tree_mask,
                            int32_t mask_words, const uint16_t *cache, int32_t num_blocks,
                            int32_t block_size, float scale, uint16_t *out, int64_t out_row_stride,
                            float *lse, int32_t *err, void *workspace, size_t workspace_bytes,
                            cudaStream_t stream)
{
    TreeAttentionLaunch a = attention_launch(q, q_row_stride, rows, num_kv_heads, row_start, seqs, context_len, block_table,
                                             table_stride, table_width, tree_mask, mask_words, num_blocks, block_size, scale,
                                             out, out_row_stride, lse, err);
    a.cache = cache;
    return attend("rc_tree_attention", a, num_heads, workspace, workspace_bytes, stream);
}

rc_status rc_window_attention(const uint16_t *q, int64_t q_row_stride, int64_t rows, int32_t num_heads,
                              int32_t num_kv_heads, const int32_t *row_start, int32_t seqs,
                              const int32_t *context_len, const int32_t *block_table,
                              int64_t table_stride, int32_t table_width, const uint64_t *tree_mask,
                              int32_t mask_words, const uint16_t *cache, int32_t num_blocks,
                              int32_t block_size, int32_t window, int32_t sinks, float scale,
                              uint16_t *out, int64_t out_row_stride, float *lse, int32_t *err,
                              void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const char *fn = "rc_window_attention";
    if (window < 1 || sinks < 0)
        return fail(RC_ERR_INVALID_ARG, "%s: need window >= 1 and sinks >= 0", fn);
    TreeAttentionLaunch a = attention_launch(q, q_row_stride, rows, num_kv_heads, row_start, seqs, context_len, block_table,
                                             table_stride, table_width, tree_mask, mask_words, num_blocks, block_size, scale,
                                             out, out_row_stride, lse, err);
    a.cache = cache;
    a.window = window;
    a.sinks = sinks;
    return attend(fn, a, num_heads, workspace, workspace_bytes, stream);
}

size_t rc_kv4_attention_workspace_size(int64_t rows, int32_t seqs, int32_t num_heads, int32_t num_kv_heads)
{
    if (!attention_sizes(rows, seqs, num_heads, num_kv_heads))
        return 0;
    const int sms = num_sms_current();
    return sms > 0 ? kv4_attention_workspace(rows, seqs, num_heads / num_kv_heads, sms) : 0;
}

rc_status rc_kv4_attention(const uint16_t *q, int64_t q_row_stride, int64_t rows, int32_t num_heads,
                           int32_t num_kv_heads, const int32_t *row_start, int32_t seqs,
                           const int32_t *context_len, const int32_t *block_table, int64_t table_stride,
                           int32_t table_width, const uint64_t *tree_mask, int32_t mask_words,
                           const uint8_t *cache4, const uint16_t *scales, int32_t num_blocks,
                           int32_t block_size, int32_t window, int32_t sinks, float scale,
                           uint16_t *out, int64_t out_row_stride, float *lse, int32_t *err,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const char *fn = "rc_kv4_attention";
    if (window < 0 || sinks < 0 || (window == 0 && sinks > 0))
        return fail(RC_ERR_INVALID_ARG, "%s: need window >= 0 (0: none) and sinks >= 0 (0 without a window)", fn);
    if (!cache4)
        return fail(RC_ERR_INVALID_ARG, "%s: cache4 must not be NULL", fn);
    TreeAttentionLaunch a = attention_launch(q, q_row_stride, rows, num_kv_heads, row_start, seqs, context_len, block_table,
                                             table_stride, table_width, tree_mask, mask_words, num_blocks, block_size, scale,
                                             out, out_row_stride, lse, err);
    a.cache4 = cache4;
    a.scales = scales;
    a.window = window;
    a.sinks = sinks;
    return attend(fn, a, num_heads, workspace, workspace_bytes, stream);
}

rc_status rc_logits_adjust(const void *logits, int32_t dtype, int64_t row_stride, int64_t rows,
                           int32_t vocab, const int32_t *row_start, int32_t seqs,
                           const rc_logits_params *params, void *out, int64_t out_row_stride,
                           int32_t *err, cudaStream_t stream)
{
    const char *fn = "rc_logits_adjust";
    if (dtype != RC_BF16 && dtype != RC_F32)
        return fail(RC_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
    if (rows < 0 || rows > (1LL << 30) || vocab < 1 || vocab > (1 << 30))
        return fail(RC_ERR_INVALID_ARG, "%s: rows=%lld outside [0, 2^30] or vocab=%d outside [1, 2^30]", fn,
                    (long long)rows, vocab);
    if (seqs < 1 || seqs > 65535)
        return fail(RC_ERR_INVALID_ARG, "%s: seqs=%d outside [1, 65535]", fn, seqs);
    const int size = size_of(dtype);
    if ((rows > 0 && (!logits || !out)) || !row_start || !params)
        return fail(RC_ERR_INVALID_ARG, "%s: logits, out, row_start and params must not be NULL", fn);
    if (!aligned(logits, size) || !aligned(out, size) || !aligned(row_start, 4))
        return fail(RC_ERR_INVALID_ARG, "%s: logits, out and row_start must be aligned to their element", fn);
    if (row_stride < 0 || out_row_stride < 0 || row_stride > kMaxStride || out_row_stride > kMaxStride ||
        (rows > 1 && out_row_stride < vocab))
        return fail(RC_ERR_INVALID_ARG, "%s: row strides must be non-negative and out's at least vocab", fn);
    const rc_logits_params &p = *params;
    if (p.history && (!p.history_start || p.history_size < 0 || p.history_size >= (1 << 28) ||
                      !aligned(p.history, 4) || !aligned(p.history_start, 8)))
        return fail(RC_ERR_INVALID_ARG, "%s: a history needs history_start, its size below 2^28 and "
                    "aligned pointers", fn);
    if (p.bias_start && (!p.bias_tokens || !p.bias_values || p.bias_size < 0 || p.bias_size > 0x7FFFFFFFLL ||
                         !aligned(p.bias_start, 4) || !aligned(p.bias_tokens, 4) || !aligned(p.bias_values, 4)))
        return fail(RC_ERR_INVALID_ARG, "%s: biases need bias_tokens, bias_values, a size below 2^31 and "
                    "aligned pointers", fn);
    if (!p.bias_start && (p.bias_tokens || p.bias_values))
        return fail(RC_ERR_INVALID_ARG, "%s: biases without bias_start", fn);
    if (p.tree_mask && (!aligned(p.tree_mask, 8) || p.mask_words < 1))
        return fail(RC_ERR_INVALID_ARG, "%s: tree_mask must be 8-byte aligned with mask_words >= 1", fn);
    if (!aligned(p.prompt_len, 4) || !aligned(p.draft_tokens, 4) || !aligned(p.repetition, 4) ||
        !aligned(p.frequency, 4) || !aligned(p.presence, 4) || !aligned(p.allowed, 4))
        return fail(RC_ERR_INVALID_ARG, "%s: per-sequence and per-row arrays must be 4-byte aligned", fn);
    if (p.allowed && (p.allowed_stride < 0 || p.allowed_stride > kMaxStride ||
                      (rows > 1 && p.allowed_stride < (vocab + 31) / 32)))
        return fail(RC_ERR_INVALID_ARG, "%s: allowed needs rows of at least ceil(vocab/32) words", fn);
    if (rows == 0)
        return ok();
    const size_t in_bytes = ((rows - 1) * row_stride + vocab) * (size_t)size;
    const size_t out_bytes = ((rows - 1) * out_row_stride + vocab) * (size_t)size;
    const bool in_place = logits == out && (rows == 1 || row_stride == out_row_stride);
    if (!in_place && overlap(logits, in_bytes, out, out_bytes))
        return fail(RC_ERR_INVALID_ARG, "%s: out overlaps logits and is not logits itself", fn);
    // (what other CTAs still read while one writes)
    const size_t per_seq = (size_t)seqs * 4, starts = ((size_t)seqs + 1) * 4;
    if (!aligned(err, 4) ||
        overlap({out, out_bytes},
                {{row_start, starts}, {p.history, p.history ? (size_t)p.history_size * 4 : (size_t)0},
                 {p.history ? p.history_start : nullptr, 2 * starts}, {p.prompt_len, per_seq},
                 {p.draft_tokens, (size_t)rows * 4}, {p.tree_mask, (size_t)rows * p.mask_words * 8},
                 {p.repetition, per_seq}, {p.frequency, per_seq}, {p.presence, per_seq},
                 {p.bias_start, starts}, {p.bias_tokens, (size_t)p.bias_size * 4},
                 {p.bias_values, (size_t)p.bias_size * 4},
                 {p.allowed, (size_t)((rows - 1) * p.allowed_stride + (vocab + 31) / 32) * 4}, {err, 4}}))
        return fail(RC_ERR_INVALID_ARG, "%s: out overlaps a history, a mask or another operand that is read, or err "
                    "is not 4-byte aligned", fn);
    const int sms = num_sms_current();
    if (sms <= 0)
        return fail(RC_ERR_CUDA, "%s: no current CUDA device", fn);
    rc::LogitsLaunch a{};
    a.logits = logits;
    a.out = out;
    a.row_stride = row_stride;
    a.out_row_stride = out_row_stride;
    a.rows = rows;
    a.V = vocab;
    a.seqs = seqs;
    a.row_start = row_start;
    a.history = p.history;
    a.history_size = p.history_size;
    a.history_start = p.history_start;
    a.prompt_len = p.prompt_len;
    a.draft_tokens = p.draft_tokens;
    a.tree_mask = p.tree_mask;
    a.mask_words = p.mask_words;
    a.repetition = p.repetition;
    a.frequency = p.frequency;
    a.presence = p.presence;
    a.bias_start = p.bias_start;
    a.bias_tokens = p.bias_tokens;
    a.bias_values = p.bias_values;
    a.bias_size = p.bias_size;
    a.allowed = p.allowed;
    a.allowed_stride = p.allowed_stride;
    a.err = err;
    const cudaError_t e = rc::launch_logits_adjust(a, dtype == RC_F32, sms, stream);
    return e == cudaSuccess ? ok() : cuda_fail(e, "rc_logits_adjust launch");
}

}  // extern "C"
