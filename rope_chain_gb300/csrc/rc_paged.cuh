// The operators around the drafted tokens' step: what their kernels' files (k8 to
// k11) offer to the C ABI (rc_paged.cu).
#pragma once
#include "rc_draft.cuh"

namespace rc {

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

}  // namespace rc
