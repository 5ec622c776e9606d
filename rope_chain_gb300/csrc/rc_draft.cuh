// The drafted tokens' operators: what their kernels' files (k5, k6, k7) offer
// to the C ABI (rc_draft.cu, and rc_api.cu for the fault bits).  Apart from
// rc_internal.cuh, so that a change here leaves the chain's sources as they are.
#pragma once
#include "rc_internal.cuh"

namespace rc {

constexpr int kMaxRotDim = 512;

// Rotary application over T tokens of `heads` heads (strides in elements,
// any order of token and head).
struct RopeLaunch {
    const void *x;
    void *out;
    int64_t x_row_stride, x_head_stride, out_row_stride, out_head_stride;
    const int64_t *positions;        // [T]
    const void *table;               // [max_position, rot]: cos, then sin
    int64_t max_position;
    int64_t T;
    int32_t heads, width, rot;       // T * heads < 2^31
    int32_t *err;
};

// `wide`: 16-byte accesses (pointers, strides, width and rot allow them).
cudaError_t launch_rope_apply(const RopeLaunch &a, bool x_f32, bool table_f32, bool halves, bool inverse,
                              bool wide, int num_sms, cudaStream_t stream);

// The table of `positions` rows from the rot / 2 angular frequencies inv.
cudaError_t launch_rope_table(void *out, bool f32, int64_t positions, int32_t rot, const double *inv,
                              float gain, int num_sms, cudaStream_t stream);

// Logits adjustment: row r of sequence b (row_start) gets the repetition,
// frequency and presence penalties, the biases and the mask.
struct LogitsLaunch {
    const void *logits;
    void *out;
    int64_t row_stride, out_row_stride;      // elements
    int64_t rows;
    int32_t V, seqs;
    const int32_t *row_start;                // [seqs + 1]
    const int32_t *history;                  // or NULL
    int64_t history_size;
    const int64_t *history_start;            // [seqs + 1]
    const int32_t *prompt_len;               // [seqs] or NULL
    const int32_t *draft_tokens;             // [rows] or NULL
    const uint64_t *tree_mask;               // [rows, mask_words] or NULL (chain)
    int32_t mask_words;
    const float *repetition, *frequency, *presence;   // [seqs] or NULL
    const int32_t *bias_start, *bias_tokens;          // [seqs + 1], [bias_size], or NULL
    const float *bias_values;
    int64_t bias_size;
    const uint32_t *allowed;                 // [rows, allowed_stride] bit words, or NULL
    int64_t allowed_stride;
    int32_t *err;
};

cudaError_t launch_logits_adjust(const LogitsLaunch &a, bool f32, int num_sms, cudaStream_t stream);

// Tree attention over the paged cache.
struct TreeAttentionLaunch {
    const uint16_t *q;                       // bf16 [rows, heads, 64], head stride 64
    int64_t q_row_stride;
    int64_t rows;
    int32_t kv_heads, group, seqs;
    const int32_t *row_start;                // [seqs + 1]
    const int32_t *context_len;              // [seqs]
    const int32_t *block_table;              // [seqs, table_width], row stride table_stride
    int64_t table_stride;
    int32_t table_width;
    const uint64_t *tree_mask;               // [rows, mask_words] or NULL (chain)
    int32_t mask_words;
    const uint16_t *cache;                   // bf16 [num_blocks, kv_heads, block_size, 128]
    const uint8_t *cache4;                   // or in 4 bits, [num_blocks, kv_heads, block_size, 64]
    const uint16_t *scales;                  // with its scales, bf16 [num_blocks, kv_heads, block_size, 4]
    int32_t num_blocks, block_size;
    float scale;
    uint16_t *out;                           // bf16 [rows, heads, 64], head stride 64
    int64_t out_row_stride;
    float *lse;                              // [rows, heads] or NULL
    int32_t *err;
    float *partial;                          // workspace, or NULL: no split
    int32_t window, sinks;                   // keys that count, the last and the first (window 0: all)
};

// Workspace bytes with which the keys are split over the GPU.
size_t tree_attention_workspace(int64_t rows, int32_t seqs, int32_t group, int num_sms);

cudaError_t launch_tree_attention(const TreeAttentionLaunch &a, int num_sms, cudaStream_t stream,
                                  const char **why);

// The same over a cache in 4 bits.
size_t kv4_attention_workspace(int64_t rows, int32_t seqs, int32_t group, int num_sms);
cudaError_t launch_kv4_attention(const TreeAttentionLaunch &a, int num_sms, cudaStream_t stream, const char **why);

// Its tiles of 128 rows (two: 256) on tcgen05, and their workspace.
size_t kv4_wide_workspace(bool two, int num_sms);
cudaError_t launch_kv4_wide(const TreeAttentionLaunch &a, bool two, int num_sms, cudaStream_t stream, const char **why);

// Sticky device fault bits of the tree attention (current device).
cudaError_t read_attention_faults(uint32_t *flags, bool clear);

}  // namespace rc
