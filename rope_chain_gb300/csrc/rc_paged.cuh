// The operators around the drafted tokens' step: what their kernels' files (k8 to
// k11) offer to the C ABI (rc_paged.cu).
#pragma once
#include "rc_draft.cuh"

namespace rc {

// Dynamic shared memory of `bytes` allowed for a kernel, once per device.
template <typename Kernel> inline cudaError_t allow_smem(Kernel kernel, size_t bytes, bool (&configured)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && configured[dev]))
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64)
        configured[dev] = true;
    return e;
}

constexpr int kMaxNormDim = 512;

// Norm and rotation of T tokens of `heads` heads (strides in elements), and with
// dy its gradient (out is dx then).
struct HeadNormLaunch {
    const void *x, *dy;
    void *out;
    int64_t x_row_stride, x_head_stride, dy_row_stride, dy_head_stride, out_row_stride, out_head_stride;
    const void *weight[2];           // [width] of the first q_heads heads and of the others, or NULL
    float *dweight[2];               // FP32 [width], or NULL
    float *partial;                  // workspace, where a dweight is wanted
    const int64_t *positions;        // [T]
    const void *table;               // [max_position, rot]: cos, then sin
    int64_t max_position;
    int64_t T;
    int32_t heads, q_heads, width, rot;     // T * heads < 2^31
    float eps;
    int32_t weight_f32, table_f32;
    int32_t *err;
};

// `wide`: 16-byte accesses (pointers, strides, width and rot allow them).
cudaError_t launch_head_norm_rope(const HeadNormLaunch &a, bool f32, bool halves, bool wide, int num_sms,
                                  cudaStream_t stream);

// Workspace bytes of a gradient with weights.
size_t head_norm_grad_workspace(int32_t width, int num_sms);

// Rows into a cache in 4 bits (rc_kv4.cuh) and out of it.
struct Kv4StoreLaunch {
    const uint16_t *k, *v;           // bf16 [T, heads, 64], strides in elements
    int64_t k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    int64_t T;                       // T * heads < 2^31
    const int64_t *slots;            // [T]
    uint8_t *cache4;                 // [num_blocks, heads, block_size, 64]
    uint16_t *scales;                // bf16 [num_blocks, heads, block_size, 4]
    int64_t capacity;                // num_blocks * block_size
    int32_t heads, block_size;
    int32_t *err;
};
struct Kv4LoadLaunch {
    const int64_t *slots;
    int64_t T;
    const uint8_t *cache4;
    const uint16_t *scales;
    int64_t capacity;
    int32_t heads, block_size;
    uint16_t *out;                   // bf16 [T, heads, 128]
    int32_t *err;
};
cudaError_t launch_kv4_store(const Kv4StoreLaunch &a, cudaStream_t stream);
cudaError_t launch_kv4_load(const Kv4LoadLaunch &a, int num_sms, cudaStream_t stream);

// Accepted nodes' rows moved to follow the context.
constexpr int kMaxCompactCaches = 64;
struct CompactLaunch {
    void *caches[kMaxCompactCaches];
    int32_t row_bytes[kMaxCompactCaches];
    int32_t count, num_blocks, heads, block_size, seqs;
    const int32_t *block_table;      // [seqs, table_width], row stride table_stride
    int64_t table_stride;
    int32_t table_width;
    const int32_t *context_len;      // [seqs]
    const int32_t *row_start;        // [seqs + 1]
    int64_t rows;
    const int32_t *path;             // [seqs, path_width], row stride path_stride
    int64_t path_stride;
    int32_t path_width;
    const int32_t *path_len;         // [seqs]
    int32_t *new_len, *err;
};
cudaError_t launch_kv_compact(const CompactLaunch &a, cudaStream_t stream);

}  // namespace rc
