/*
 * rope_chain.h -- C ABI of librope_chain.so: the speculative draft's context
 * K/V chain (MuseSparkDSparkModel.precompute_and_store_context_kv) on one
 * GB300 GPU (sm_103a).
 *
 * The chain, per context row t of width D = 8192 and draft layer l < L:
 *   1. hidden RMSNorm of x[t], rounded to bf16                 rc_context_norms
 *   2. layer l's input RMSNorm of that, stacked into [L, T, D]  rc_context_norms
 *   3. K/V projection [L, T, D] x [L, D, 2*H*64]                rc_kv_project
 *   4. weightless K-norm of every 64-wide key head, GPT-J RoPE,
 *      and the slot-mapped insert of K and V into paged caches  rc_kv_store
 *
 * Sources, cited by web page title and symbol:
 *   [ctx] "vllm.models.muse_spark.nvidia.specialized_decode.cutedsl.draft.context"
 *   [rt]  "vllm.models.muse_spark.nvidia.specialized_decode.runtime.draft"
 *   [bnd] "vllm.models.muse_spark.nvidia.specialized_decode.cutedsl.common.draft_boundary"
 *
 * Conventions for every call:
 *   - Tensor pointers are DEVICE pointers owned by the caller; the library
 *     never frees or retains them.  Pointer ARRAYS (slots, caches) are HOST
 *     arrays of device pointers, read during the call only.  A pointer
 *     to an INPUT may also be the device address of page-locked host memory
 *     (rc_device_address): the kernels then read it over the host link
 *     (NVLink-C2C on GB300) with no staging copy.  The host memory must
 *     stay allocated and unchanged until the stream has passed the call.
 *   - bf16 values travel as uint16_t bit patterns.
 *   - Work is enqueued on `stream`; calls do not synchronise and do not
 *     allocate device memory, so they can be issued inside CUDA graph
 *     capture.  Outputs are valid once the stream reaches that point.
 *   - Arguments are checked on the host before anything is launched; a
 *     rejected call returns RC_ERR_INVALID_ARG or RC_ERR_UNSUPPORTED, leaves
 *     every buffer untouched, and rc_last_error() says why.
 *   - Floating point: FP32 arithmetic with the rounding points of [ctx]
 *     (each product, sum and fma rounded to nearest even; nothing fused
 *     beyond the fma the pages write); 1/sqrt is the correctly rounded
 *     IEEE sqrt then divide (the pages use a hardware approximation).
 *     Subnormals are kept.
 */
#ifndef ROPE_CHAIN_H
#define ROPE_CHAIN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    RC_OK = 0,
    RC_ERR_INVALID_ARG = 1,   /* malformed argument: null, misaligned, out of range */
    RC_ERR_UNSUPPORTED = 2,   /* well-formed but outside what the kernels cover */
    RC_ERR_CUDA = 3           /* a CUDA runtime call or launch failed */
} rc_status;

/* Weight layouts accepted by rc_kv_project. */
typedef enum {
    RC_W_KN = 0,   /* W[L, D, N]: N contiguous (the projection as x @ W) */
    RC_W_NK = 1    /* W[L, N, D]: D contiguous (nn.Linear layout; [rt]
                      ContextKV._project multiplies by its transpose) */
} rc_weight_layout;

/* Message of the last failed call on this host thread ("" if none). */
const char *rc_last_error(void);

/* Library version, major*10000 + minor*100 + patch. */
int32_t rc_version(void);

/*
 * rc_context_norms -- steps 1 and 2.  [ctx] ContextNorms / _ContextNormsKernel,
 * [rt] ContextKV._project (the stack), [bnd] boundary_fragments (norm order).
 *
 *   z[t]      = bf16( hidden_norm(x[t]) )
 *   out[l, t] = bf16( pre_norm_l(z[t]) )         for l < L
 * with norm(v)_c = (v_c * r) * gamma_c (or v_c * r when the weight is NULL),
 * r = 1 / sqrt(fma(sum_c v_c^2, 1/D, eps)), the sum in a fixed documented
 * order (thread t of 256 holds columns 2048k + 8t + i; in-thread (k, i)
 * order; xor butterfly over each warp; the 8 warp sums left to right).
 *
 *   x         bf16 [T, D] row-major, contiguous, 16-byte aligned
 *   T         rows, 0 <= T < 2^31 (T == 0: nothing is launched)
 *   D         must be 8192 (the single-tile row norm); else RC_ERR_UNSUPPORTED
 *   hidden_w  bf16 [D] hidden-norm weight, 16-byte aligned, or NULL (weightless)
 *   pre_w     bf16 [L, D] layer input-norm weights, 16-byte aligned, or NULL
 *   L         layers, 1 <= L <= 64
 *   eps       shared by both norms
 *   out       bf16 [L, T, D] contiguous, 16-byte aligned; must not overlap x
 */
rc_status rc_context_norms(const uint16_t *x, int64_t T, int32_t D,
                           const uint16_t *hidden_w, const uint16_t *pre_w,
                           int32_t L, float eps, uint16_t *out,
                           cudaStream_t stream);

/*
 * rc_context_norms_ex -- steps 1 and 2 with every option of [ctx]
 * ContextNormConstants and ContextNorms: each norm's weight absent, bf16 or
 * FP32; the weight scaling the norm's input (before the sum of squares) or
 * its output; a gain center added to each weight element; and each norm's
 * own eps ([ctx] ContextNorms takes hidden_eps and pre_eps).
 *
 * For one norm with weight w, gamma_c = w_c + center (w_c itself when the
 * center is 0, so a -0.0 weight keeps its sign), and
 *   input scale:   u_c = gamma_c * v_c,  y_c = u_c * r(u)
 *   output scale:  y_c = (v_c * r(v)) * gamma_c
 *   no weight:     y_c = v_c * r(v)
 * with r(u) = 1 / sqrt(fma(sum_c u_c^2, 1/D, eps)) in the order of
 * rc_context_norms ([bnd] boundary_fragments writes both scale sides in this
 * order).  z = bf16(hidden norm of x); out[l, t] = bf16(layer l's norm of z),
 * an input-scale layer weight giving each layer its own r.
 *
 *   x, T, D, L, out   as rc_context_norms
 *   hidden, pre       HOST pointers to the two norms' parameters, read during
 *                     the call; hidden->weight is [D], pre->weight [L, D]
 *                     (device, 16-byte aligned, NULL exactly when
 *                     weight_dtype is RC_NORM_NONE; input_scale and
 *                     gain_center of a weightless norm are ignored)
 * Errors: RC_ERR_INVALID_ARG for a NULL or misaligned pointer, an unknown
 * weight_dtype or a weight/dtype mismatch; RC_ERR_UNSUPPORTED for D != 8192.
 */
typedef enum {
    RC_NORM_NONE = 0,   /* weightless norm */
    RC_NORM_BF16 = 1,   /* bf16 weight (uint16_t bit patterns) */
    RC_NORM_F32 = 2     /* FP32 weight */
} rc_norm_weight;

typedef struct {
    const void *weight;     /* device pointer, or NULL with RC_NORM_NONE */
    int32_t weight_dtype;   /* rc_norm_weight */
    int32_t input_scale;    /* non-zero: the weight scales the norm's input */
    float gain_center;      /* added to each weight element when non-zero */
    float eps;              /* this norm's eps */
} rc_norm_params;

rc_status rc_context_norms_ex(const uint16_t *x, int64_t T, int32_t D,
                              const rc_norm_params *hidden, const rc_norm_params *pre,
                              int32_t L, uint16_t *out, cudaStream_t stream);

/*
 * rc_kv_project -- step 3.  [rt] ContextKV._project
 * (torch.bmm(per_layer, stacked_kv_weight.transpose(1, 2))).
 *
 *   out[l, t, n] = bf16( sum_k normed[l, t, k] * W_l[k, n] )
 * BF16 inputs, FP32 accumulation on the tensor cores (tcgen05), one
 * rounding to bf16 at the end.  The summation order is the kernel's, so
 * results agree with an exact sum to within bf16 rounding plus FP32
 * accumulation error, not bit for bit.
 *
 *   normed     bf16 [L, T, D] contiguous, 16-byte aligned
 *   W          bf16 weights in `w_layout`, contiguous, 16-byte aligned
 *   w_layout   RC_W_KN or RC_W_NK
 *   out        bf16 [L, T, N] contiguous, 16-byte aligned
 *   L          1 <= L <= 4096;  T: 0 <= T <= 8388480 (T == 0: no launch)
 *   D          multiple of 64, >= 64;  N: multiple of 128, >= 128
 *   workspace  optional device scratch for split-K (16-byte aligned) and its
 *              size in bytes; NULL/0 runs without split-K.  For few output
 *              tiles the K dimension is split across CTAs and the FP32
 *              partial sums are added in split order by a second kernel
 *              (deterministic for a given workspace size).  With many
 *              tiles whose last round would leave most SMs idle, the last
 *              layer's final row blocks are split the same way in a launch
 *              of their own.  From eight rounds of tiles the persistent
 *              kernel's CTA pairs take their tiles in order from a 4-byte
 *              counter in the workspace (zeroed by the call), so the pairs
 *              that read the same rows of `normed` stay in step and share
 *              them in L2 (with a fixed tile order they drift apart and read
 *              them from DRAM again).  The tile order does not change the
 *              results.  The bytes that give all of this are
 *              rc_kv_project_workspace_size(); calls sharing one workspace
 *              must not overlap on the GPU.
 */
rc_status rc_kv_project(const uint16_t *normed, const uint16_t *W,
                        int32_t w_layout, uint16_t *out, int32_t L, int64_t T,
                        int32_t D, int32_t N, void *workspace,
                        size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes rc_kv_project uses at most for these sizes on the current
   device (0 when it would split nothing).  Host-only apart from one device
   attribute query; returns 0 for invalid sizes. */
size_t rc_kv_project_workspace_size(int32_t L, int64_t T, int32_t D, int32_t N);

/* The same figure for a GPU with num_sms streaming multiprocessors, with no
   device involved (plan allocations ahead of time, or for another GPU).
   Host-only; returns 0 for invalid sizes or num_sms < 1. */
size_t rc_kv_project_workspace_size_sms(int32_t L, int64_t T, int32_t D, int32_t N,
                                        int32_t num_sms);

/* How rc_kv_project (and rc_kv_project_store) run these sizes on a GPU with
   num_sms SMs given workspace_bytes of workspace.  Host-only.
     kernel          0: single CTAs (128-row tiles), 1: CTA pairs, one tile
                     each (256 x 256), 2: persistent CTA pairs walking the tiles
     splits          K splits of the main launch (1: none; > 1: FP32 partials
                     in the workspace, then a reduction launch)
     tail_splits     persistent plans: 0 without a tail launch; else the K
                     splits of the last layer's final row blocks, run as a
                     launch of their own (plus their reduction)
     tail_row0       the first of those rows (T without a tail launch)
     dynamic_tiles   persistent plans: 1 when the pairs take tiles in order
                     from a counter in the workspace (so pairs that share rows
                     of `normed` stay in step), 0 for a fixed tile sequence
     workspace_bytes the part of the workspace used
   T = 0 launches nothing: the plan reads single CTAs, 1 split, no
   workspace.  RC_ERR_INVALID_ARG / RC_ERR_UNSUPPORTED for sizes
   rc_kv_project refuses or num_sms < 1; *plan untouched then. */
typedef struct {
    int32_t kernel;
    int32_t splits;
    int32_t tail_splits;
    int32_t dynamic_tiles;
    int64_t tail_row0;
    size_t workspace_bytes;
} rc_project_plan;

rc_status rc_kv_project_plan(int32_t L, int64_t T, int32_t D, int32_t N, int32_t num_sms,
                             size_t workspace_bytes, rc_project_plan *plan);

/*
 * rc_kv_store -- step 4.  [ctx] ContextKvStore / _ContextKvStoreKernel,
 * _sum_squares_64, _rope; [rt] ContextKV.store.
 *
 * For every layer l < L whose slots[l] is not NULL and every row t < rows,
 * with s = slots[l][t]:
 *   s < 0                                      row skipped (nothing read or written)
 *   s >= num_blocks*block_size, or (cos_sin != NULL) positions[t] outside
 *   [0, max_position)                          row skipped and counted in *err
 *   otherwise, for each head h < H:
 *     key   = bf16(k_h * r), r = 1/sqrt(fma(sum k_h^2, 1/64, eps)),
 *             the sum folded as lane j holding the pair (2j, 2j+1): even and
 *             odd squares each by an xor butterfly, then even + odd;
 *     key   = GPT-J RoPE of each pair (2j, 2j+1) with c = cos_sin[pos, j],
 *             s = cos_sin[pos, 32 + j]: (fma(x, c, -(y*s)), fma(y, c, x*s)),
 *             rounded to bf16 (skipped when cos_sin is NULL);
 *     caches[l][s / block_size, h, s % block_size, 0:64]   = key
 *     caches[l][s / block_size, h, s % block_size, 64:128] = v[l, t, h, :]
 *   No other cache element is written.
 *
 *   k, v          bf16 views [L, >=rows, H, 64]: element (l, t, h, e) at
 *                 base + l*layer_stride + t*row_stride + h*64 + e; 4-byte
 *                 aligned, strides even and >= 0.  For a projection output
 *                 kv [L, T, 2*H*64]: k = kv, v = kv + 64*H, row stride
 *                 128*H, layer stride T*128*H.
 *   positions     int64 [rows] (read only with cos_sin), 8-byte aligned
 *   slots         host array of L device pointers to int64 [rows]; NULL
 *                 entries skip their layer
 *   cos_sin       bf16 [max_position, 64] (cos in 0..31, sin in 32..63) or NULL
 *   caches        host array of L device pointers to contiguous bf16
 *                 [num_blocks, H, block_size, 128], 4-byte aligned
 *   num_blocks, block_size   >= 1, num_blocks*block_size < 2^31
 *   H             KV heads: 1, 2, 4, 8, 16 or 32
 *   L             1 <= L <= 4096; layers go to the GPU 8 per launch
 *   rows          rows to insert, 0 <= rows < 2^31 (0: nothing launched)
 *   err           device int32 counter, incremented once per skipped
 *                 (row, layer) as above; may be NULL
 * Two non-negative slots of one layer that are equal write the same cache
 * entry in an unspecified order (a precondition violation).
 */
rc_status rc_kv_store(const uint16_t *k, const uint16_t *v,
                      int64_t k_layer_stride, int64_t k_row_stride,
                      int64_t v_layer_stride, int64_t v_row_stride,
                      const int64_t *positions, const int64_t *const *slots,
                      const uint16_t *cos_sin, int64_t max_position,
                      uint16_t *const *caches, int32_t num_blocks,
                      int32_t block_size, int32_t H, int32_t L, float eps,
                      int64_t rows, int32_t *err, cudaStream_t stream);

/*
 * rc_kv_store_rows -- rc_kv_store with a row count per layer ([rt]
 * _slot_groups: each layer's slot mapping has its own length and layer l
 * inserts its first len(slots[l]) rows; the pages issue one store call per
 * run of consecutive layers of equal length, here one launch takes up to 8
 * layers of any lengths).
 *
 *   layer_rows    HOST array of L row counts, each 0 <= layer_rows[l] < 2^31;
 *                 slots[l] and k, v hold at least layer_rows[l] rows
 *   other arguments as rc_kv_store (positions holds max_l layer_rows[l] rows)
 */
rc_status rc_kv_store_rows(const uint16_t *k, const uint16_t *v,
                           int64_t k_layer_stride, int64_t k_row_stride,
                           int64_t v_layer_stride, int64_t v_row_stride,
                           const int64_t *positions, const int64_t *const *slots,
                           const uint16_t *cos_sin, int64_t max_position,
                           uint16_t *const *caches, int32_t num_blocks,
                           int32_t block_size, int32_t H, int32_t L, float eps,
                           const int64_t *layer_rows, int32_t *err, cudaStream_t stream);

/*
 * rc_kv_project_store -- steps 3 and 4 fused (the projection and the store
 * of [rt] ContextKV.store in one pass; the scope's "store fused into the
 * GEMM epilogue").  The caches receive exactly the bits that
 *   rc_kv_project(normed, W, w_layout, kv, ...) followed by
 *   rc_kv_store(k = kv, v = kv + 64*H, row stride 128*H, layer stride
 *               T*128*H, positions, slots, cos_sin, caches, ..., rows, err)
 * would write with the same workspace, without the [L, T, 128*H] round trip:
 * the key is normed from the bf16-rounded projection exactly as
 * rc_kv_store norms it.  Where the projection is not split, CTA-pair tiles
 * store from the GEMM epilogue; split plans store from the pass that adds
 * the FP32 partials.
 *
 *   normed, W, w_layout, D        as rc_kv_project; N = 128*H
 *   L                             1 <= L <= 64 (one launch for all layers)
 *   T                             rows of the projection, as rc_kv_project
 *   positions, slots, cos_sin, max_position, caches, num_blocks,
 *   block_size, H, eps, err       as rc_kv_store (caches and cos_sin
 *                                 16-byte aligned)
 *   rows                          rows stored, 0 <= rows <= T
 *   kv_out                        optional bf16 [L, T, 128*H]: also write the
 *                                 projection; required when the plan neither
 *                                 splits nor uses CTA pairs (T <= 128 or
 *                                 N = 128, without a workspace)
 *   workspace                     as rc_kv_project
 */
rc_status rc_kv_project_store(const uint16_t *normed, const uint16_t *W,
                              int32_t w_layout, int32_t L, int64_t T, int32_t D,
                              int32_t H, const int64_t *positions,
                              const int64_t *const *slots,
                              const uint16_t *cos_sin, int64_t max_position,
                              uint16_t *const *caches, int32_t num_blocks,
                              int32_t block_size, float eps, int64_t rows,
                              int32_t *err, uint16_t *kv_out, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/*
 * rc_kv_project_store_rows -- rc_kv_project_store with a row count per
 * layer, as rc_kv_store_rows: layer l stores its first layer_rows[l] rows.
 *
 *   layer_rows    HOST array of L row counts, each 0 <= layer_rows[l] <= T
 *   other arguments as rc_kv_project_store
 */
rc_status rc_kv_project_store_rows(const uint16_t *normed, const uint16_t *W,
                                   int32_t w_layout, int32_t L, int64_t T, int32_t D,
                                   int32_t H, const int64_t *positions,
                                   const int64_t *const *slots,
                                   const uint16_t *cos_sin, int64_t max_position,
                                   uint16_t *const *caches, int32_t num_blocks,
                                   int32_t block_size, float eps, const int64_t *layer_rows,
                                   int32_t *err, uint16_t *kv_out, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/*
 * rc_context_kv -- the whole chain in one call (steps 1 to 4; [rt]
 * ContextKV.store / MuseSparkDSparkModel.precompute_and_store_context_kv),
 * with the norms fused into the projection (the scope's "norms fused into
 * the GEMM producer"): a row pass writes the hidden-norm output
 * z = bf16(hidden_norm(x)) and each row's layer-norm inverse RMS r once; the
 * projection forms each layer's operand bf16((z * r) * pre_w[l]) in shared
 * memory (bit-identical to rc_context_norms' output) and stores as
 * rc_kv_project_store does.  The [L, T, D] normed rows never reach memory.
 * The caches receive exactly the bits of rc_context_norms +
 * rc_kv_project_store with an equally split projection.
 *
 *   x, T, D, hidden_w, pre_w, L, eps      as rc_context_norms (D = 8192,
 *                                         L <= 64)
 *   W, w_layout, H                        as rc_kv_project (N = 128*H)
 *   positions ... err, kv_out             as rc_kv_project_store
 *   workspace   device scratch, 256-byte aligned, required: the row pass's
 *               z and r (T*D*2 + T*4 bytes, rounded up) — or, for T <= 128
 *               or H = 1, the normed rows [L, T, D] — followed by the split-K
 *               partials; rc_context_kv_workspace_size() gives the bytes of
 *               the full plan, and less space splits K less.
 */
rc_status rc_context_kv(const uint16_t *x, int64_t T, int32_t D,
                        const uint16_t *hidden_w, const uint16_t *pre_w,
                        int32_t L, float eps, const uint16_t *W,
                        int32_t w_layout, int32_t H, const int64_t *positions,
                        const int64_t *const *slots, const uint16_t *cos_sin,
                        int64_t max_position, uint16_t *const *caches,
                        int32_t num_blocks, int32_t block_size, int64_t rows,
                        int32_t *err, uint16_t *kv_out, void *workspace,
                        size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes of rc_context_kv for these sizes on the current device
   (0 for unsupported sizes). */
size_t rc_context_kv_workspace_size(int32_t L, int64_t T, int32_t D, int32_t H);

/*
 * rc_context_kv_chunked -- steps 1 to 4 ([rt] ContextKV.store /
 * MuseSparkDSparkModel.precompute_and_store_context_kv) as
 * rc_context_norms followed by rc_kv_project_store, by row chunks: the
 * norms of chunk c + 1 run on the GPU beside the projection + store of
 * chunk c (each SM holds one persistent projection CTA and one norms CTA),
 * so that the norms' HBM traffic overlaps the tensor-bound projection.  The
 * caches receive exactly the bits of rc_context_norms + rc_kv_project_store
 * (the normed rows, each projection sum and each stored bit are the same;
 * only the order in which rows are stored differs, so two rows sharing a
 * slot may leave either row's values, as in rc_kv_project_store).
 *
 *   x, T, D, hidden_w, pre_w, L, eps   as rc_context_norms (D = 8192,
 *                                      L <= 64)
 *   W, w_layout, H                     as rc_kv_project (N = 128*H)
 *   positions ... err                  as rc_kv_project_store (no kv_out)
 *   chunks      row chunks wanted (<= 0: chosen for the sizes and for where
 *               x lives); fewer are used where a chunk's projection would
 *               not run as persistent CTA pairs without workspace
 *               (rc_context_kv_chunks says how many); x may be page-locked
 *               host memory (its device address, rc_device_address), which
 *               the norms of each chunk read over the host link
 *   workspace   device scratch, 256-byte aligned, required, not
 *               overlapping x or W: the normed rows [L, T, D] (chunk by
 *               chunk), then a 256-byte tile counter per chunk (or, with one
 *               chunk, the projection's workspace, or where single CTAs
 *               project without a K split a bf16 copy of the projection
 *               that the store reads); rc_context_kv_chunked_workspace_size()
 *               gives enough bytes
 * The call ends with the last chunk's projection, which starts after every
 * earlier kernel of the call has completed; a later kernel or copy in the
 * stream sees all of the call's writes.  Errors as rc_kv_project_store
 * (RC_ERR_INVALID_ARG for a workspace too small for the plan).
 */
rc_status rc_context_kv_chunked(const uint16_t *x, int64_t T, int32_t D,
                                const uint16_t *hidden_w, const uint16_t *pre_w,
                                int32_t L, float eps, const uint16_t *W,
                                int32_t w_layout, int32_t H, const int64_t *positions,
                                const int64_t *const *slots, const uint16_t *cos_sin,
                                int64_t max_position, uint16_t *const *caches,
                                int32_t num_blocks, int32_t block_size, int64_t rows,
                                int32_t *err, int32_t chunks, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream);

/*
 * rc_context_kv_chunked_ex -- rc_context_kv_chunked with every norm option
 * of rc_context_norms_ex and a row count per layer: the caches receive
 * exactly the bits of rc_context_norms_ex + rc_kv_project_store_rows.
 *
 *   x, T, D, hidden, pre, L       as rc_context_norms_ex (D = 8192)
 *   W, w_layout, H                as rc_kv_project (N = 128*H)
 *   positions ... block_size      as rc_kv_project_store
 *   eps                           the K-norm's eps (the norms carry their
 *                                 own in hidden and pre)
 *   layer_rows                    HOST array of L row counts, each in
 *                                 [0, T] (layer l stores its first
 *                                 layer_rows[l] rows), or NULL for T rows
 *                                 in every layer
 *   err, chunks, workspace, ...   as rc_context_kv_chunked (the same
 *                                 workspace size); with x in device memory
 *                                 and a norm option beyond bf16 output-scale
 *                                 weights without a centre, chunks <= 0
 *                                 means one chunk (the option kernel beside
 *                                 the projection costs more than the overlap
 *                                 gains), while x in host memory is chunked
 *                                 as rc_context_kv_chunks says
 * Errors as rc_context_norms_ex and rc_context_kv_chunked.
 */
rc_status rc_context_kv_chunked_ex(const uint16_t *x, int64_t T, int32_t D,
                                   const rc_norm_params *hidden, const rc_norm_params *pre,
                                   int32_t L, const uint16_t *W, int32_t w_layout, int32_t H,
                                   const int64_t *positions, const int64_t *const *slots,
                                   const uint16_t *cos_sin, int64_t max_position,
                                   uint16_t *const *caches, int32_t num_blocks, int32_t block_size,
                                   float eps, const int64_t *layer_rows, int32_t *err,
                                   int32_t chunks, void *workspace, size_t workspace_bytes,
                                   cudaStream_t stream);

/* Workspace bytes of rc_context_kv_chunked for these sizes on the current
   device, enough for any chunk request and for x in device or host memory
   (0 for unsupported sizes; `chunks` is accepted for symmetry). */
size_t rc_context_kv_chunked_workspace_size(int32_t L, int64_t T, int32_t D, int32_t H,
                                            int32_t chunks);

/* Host only: the number of row chunks rc_context_kv_chunked uses for these
   sizes and chunk request on a GPU of num_sms SMs, with x in device memory
   (x_on_host = 0) or page-locked host memory read over the host link
   (x_on_host != 0; the call tells the two apart itself); 0 for unsupported
   sizes.  row0, when not NULL, receives the chunks' first rows and T
   (count + 1 entries; room for 17). */
int32_t rc_context_kv_chunks(int32_t L, int64_t T, int32_t D, int32_t H, int32_t chunks,
                             int32_t x_on_host, int32_t num_sms, int64_t *row0);

/*
 * rc_context_kv in two calls.  rc_context_rows is the row pass: per row t,
 *   z[t]  = bf16(hidden_norm(x[t]))          bf16 [T, 8192], 16-byte aligned
 *   r2[t] = 1/sqrt(fma(sum z[t]^2, 1/D, eps)) FP32 [T] (the layer norms'
 *                                            inverse RMS, shared by all layers)
 * in the order and roundings of rc_context_norms.  rc_context_kv_from_rows
 * then projects and stores from (z, r2, pre_w): each layer's operand
 * bf16((z * r2) * pre_w[l]) is formed in shared memory.  It takes
 * T > 128 and H >= 2 (CTA-pair tiles) only; `workspace` holds the split-K
 * partials (rc_kv_project_workspace_size() bytes; may be NULL).
 */
rc_status rc_context_rows(const uint16_t *x, int64_t T, int32_t D,
                          const uint16_t *hidden_w, float eps, uint16_t *z,
                          float *r2, cudaStream_t stream);
rc_status rc_context_kv_from_rows(const uint16_t *z, const float *r2, int64_t T,
                                  int32_t D, const uint16_t *pre_w, int32_t L,
                                  float eps, const uint16_t *W, int32_t w_layout,
                                  int32_t H, const int64_t *positions,
                                  const int64_t *const *slots,
                                  const uint16_t *cos_sin, int64_t max_position,
                                  uint16_t *const *caches, int32_t num_blocks,
                                  int32_t block_size, int64_t rows, int32_t *err,
                                  uint16_t *kv_out, void *workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/*
 * rc_kv_project_no_alloc -- rc_kv_project for callers that cannot allocate.
 * The pages have no counterpart: it is an addition of this library.
 *
 * Some callers cannot call cudaMalloc or provide a workspace (code running
 * inside an allocator or memory-pool callback, plug-ins whose host framework
 * owns every device allocation, serving paths that must not touch the
 * allocator once running).  This call takes the same operands as
 * rc_kv_project minus the workspace and allocates nothing: its split-K
 * scratch is an array of RC_NO_ALLOC_SCRATCH_BYTES (24 MiB) inside the
 * library, held on every GPU that loads the library until the process
 * exits.  Arguments are checked as rc_kv_project checks them (sizes, layout,
 * NULL and 16-byte alignment, out overlapping normed or W); out, normed or
 * W overlapping the array itself is refused too.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it; make that first call before any
 *     stream capture.
 *   - Sizes whose split-K plan needs more than 24 MiB are refused with
 *     RC_ERR_UNSUPPORTED (on a 152-SM GB300 no size needs more than 20 MB).
 *   - All calls share the array and it keeps the last call's contents; two
 *     calls whose work overlaps on the GPU (e.g. on different streams) race
 *     on it, so order them on one stream.  Nothing in it needs clearing:
 *     each call writes every partial it reads and zeroes the tile counter
 *     it uses (an asynchronous memset on `stream`, which allocates nothing).
 * Results are bit-identical to rc_kv_project's given a workspace of
 * rc_kv_project_workspace_size() bytes (the same plan, the same kernels).
 */
#define RC_NO_ALLOC_SCRATCH_BYTES ((size_t)24 << 20)
rc_status rc_kv_project_no_alloc(const uint16_t *normed, const uint16_t *W,
                                 int32_t w_layout, uint16_t *out, int32_t L,
                                 int64_t T, int32_t D, int32_t N,
                                 cudaStream_t stream);

/*
 * rc_qkv_front -- the decode QKV front of one draft layer on 1 to 16 tokens:
 * QKV projection, QK-norm, GPT-J RoPE and KV insert in one kernel ([rt]
 * _fused_qkv_projection, _attention, may_fuse_qkv_front; the pages' kernel
 * source is not among them, so its arithmetic is read from what they state).
 *
 *   proj[m, n] = bf16(sum_k hidden[m, k] * W[n, k])   FP32 accumulation
 * Each output row is [Q | K | V | O-gate]: q_size = 64*num_heads columns of
 * Q, kv_size = 64*num_kv_heads of K, kv_size of V, q_size of the gate
 * (_attention's split).  Then, per token m:
 *   out[m, Q and K heads] = per 64-wide head: bf16(head * r) with r the
 *       weightless inverse RMS 1/sqrt(fma(sum e^2, 1/64, eps)) (the context
 *       K-norm's lane-pair order), then GPT-J RoPE at positions[m] from
 *       cos_sin (cos_sin may be NULL: no rotation), rounded to bf16;
 *   out[m, V and gate]    = proj;
 *   cache[s/bs, h, s%bs, 0:64] = out[m, K head h] and [64:128] = V head h,
 *       for s = slots[m] >= 0.
 * A token whose slot is >= num_blocks*block_size, or (with a table) whose
 * position is outside [0, max_position), adds one to *err and inserts
 * nothing; with a bad position its Q and K are normed but not rotated.
 *
 *   hidden      bf16 [M, D] contiguous, 16-byte aligned
 *   M           tokens, 0 <= M <= 16 (0: nothing launched); else RC_ERR_UNSUPPORTED
 *   D           a positive multiple of 64
 *   W           bf16 [Nqkv, D] (the nn.Linear weight), Nqkv = 64*(2*num_heads +
 *               2*num_kv_heads), 16-byte aligned
 *   positions   int64 [M] (read with a table), 8-byte aligned
 *   slots       int64 [M] slot mapping, or NULL (nothing inserted)
 *   cache       bf16 [num_blocks, num_kv_heads, block_size, 128], 4-byte
 *               aligned; num_blocks*block_size < 2^31
 *   out         bf16 [M, Nqkv], 16-byte aligned, overlapping no input
 *   raw_out     optional bf16 [M, Nqkv]: also write the projection itself
 *   err         optional device int32 counter
 * Bit 8 and up of rc_read_device_faults are this kernel's fault bits.
 */
rc_status rc_qkv_front(const uint16_t *hidden, int32_t M, int32_t D, const uint16_t *W,
                       int32_t num_heads, int32_t num_kv_heads, const int64_t *positions,
                       const uint16_t *cos_sin, int64_t max_position, const int64_t *slots,
                       uint16_t *cache, int32_t num_blocks, int32_t block_size, float eps,
                       uint16_t *out, uint16_t *raw_out, int32_t *err, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * The drafted tokens' step over the caches above: rotary positions in any
 * layout and scaling, attention of a tree of drafted tokens over the paged
 * cache, and the adjustment of their logits.  The pages have no counterpart.
 */

/* Element types of the calls below. */
typedef enum { RC_BF16 = 1, RC_F32 = 2 } rc_dtype;

/* How the frequencies of a rotary table are scaled for contexts longer than
   the trained ones. */
typedef enum {
    RC_ROPE_SCALE_NONE = 0,
    RC_ROPE_SCALE_LINEAR = 1,  /* every frequency divided by factor */
    RC_ROPE_SCALE_BASE = 2,    /* theta * factor^(rot_dim / (rot_dim - 2)) */
    RC_ROPE_SCALE_PARTS = 3    /* frequencies that turn more than beta_fast times
                                  over original_max_position kept, those that turn
                                  less than beta_slow times divided by factor, a
                                  linear ramp over the columns between */
} rc_rope_scale;

typedef struct {
    int32_t kind;                   /* rc_rope_scale */
    double factor;                  /* > 0 (not read with NONE) */
    double original_max_position;   /* > 0 (PARTS) */
    double beta_fast, beta_slow;    /* beta_fast > beta_slow > 0 (PARTS) */
    double attention_factor;        /* multiplies every cos and sin */
} rc_rope_scaling;

/*
 * rc_rope_table -- the cos|sin table that the store, the front and
 * rc_rope_apply read: row p holds attention_factor * cos(p * inv_j) in columns
 * j < rot_dim/2 and attention_factor * sin(p * inv_j) in rot_dim/2 + j, with
 * inv_j = theta^(-2j/rot_dim), scaled.  PARTS: with
 *   d(beta) = rot_dim * ln(original / (2 pi beta)) / (2 ln theta),
 *   lo = max(floor(d(beta_fast)), 0), hi = min(ceil(d(beta_slow)), rot_dim - 1),
 *   ramp_j = clamp((j - lo) / max(hi - lo, 0.001), 0, 1):
 *   inv_j * (1 - ramp_j) + inv_j / factor * ramp_j.
 * Angles are reduced in 64-bit turns, so the values hold alike at any position:
 * before their rounding to `dtype` they are within 2^-21 (RC_F32) or 2^-20
 * (RC_BF16) of the formula's, times attention_factor.
 *
 *   out          [max_position, rot_dim] of `dtype` (rc_dtype), contiguous,
 *                16-byte aligned
 *   max_position 0 <= max_position < 2^31 (0: nothing launched, out may be NULL)
 *   rot_dim      even, 2 <= rot_dim <= 512
 *   theta        > 1
 *   scaling      HOST pointer, or NULL (no scaling, factor 1)
 */
rc_status rc_rope_table(void *out, int32_t dtype, int64_t max_position, int32_t rot_dim,
                        double theta, const rc_rope_scaling *scaling, cudaStream_t stream);

typedef enum {
    RC_ROPE_PAIRS = 0,    /* elements (2j, 2j+1) turn together (GPT-J) */
    RC_ROPE_HALVES = 1    /* elements (j, rot_dim/2 + j) */
} rc_rope_layout;

/*
 * rc_rope_apply -- rotary positions on any heads: for token t, head h and
 * pair j of the first rot_dim elements, with c = cos_sin[positions[t], j] and
 * s = cos_sin[positions[t], rot_dim/2 + j],
 *   (a, b) -> (fma(a, c, -(b*s)), fma(b, c, a*s))
 * in FP32, rounded once to the type of x; elements from rot_dim on are
 * copied.  With `inverse` the transposed rotation ((a, b) -> (a c + b s,
 * b c - a s)): the gradient with respect to x, given that of the output.
 * A token whose position lies outside [0, max_position) passes through and
 * adds one to *err.
 *
 *   x, out        `dtype` (rc_dtype) [T, heads, head_dim]: element (t, h, e) at
 *                 t*row_stride + h*head_stride + e (strides in elements, >= 0,
 *                 either order of tokens and heads; aligned to the element).
 *                 out may be x with x's strides (in place), or else must not
 *                 overlap it; it overlaps no other operand, and its elements are
 *                 distinct
 *   T, heads      T >= 0, heads >= 1, T*heads < 2^31 (T == 0: nothing launched, and x,
 *                 out and positions may be NULL)
 *   rot_dim       even, 2 <= rot_dim <= min(head_dim, 512); PAIRS needs an even
 *                 head_dim, which is at most 65536
 *   positions     int64 [T], 8-byte aligned
 *   cos_sin       `table_dtype` [max_position, rot_dim], contiguous, aligned to
 *                 its element, max_position >= 1
 *   err           optional device int32 counter
 * 16-byte aligned pointers, strides, head_dim and rot_dim (half of it in
 * HALVES) move 16 bytes at a time; anything else element by element.
 */
rc_status rc_rope_apply(const void *x, int32_t dtype, int64_t x_row_stride, int64_t x_head_stride,
                        int64_t T, int32_t heads, int32_t head_dim, const int64_t *positions,
                        const void *cos_sin, int32_t table_dtype, int64_t max_position,
                        int32_t rot_dim, int32_t layout, int32_t inverse, void *out,
                        int64_t out_row_stride, int64_t out_head_stride, int32_t *err,
                        cudaStream_t stream);

/*
 * rc_tree_attention -- attention of drafted tokens over a paged cache that the
 * calls above fill.  Rows are the drafted tokens (nodes) of `seqs` sequences,
 * row_start[b] .. row_start[b+1] - 1 those of sequence b (n_b of them, in tree
 * or generation order).  Sequence b's logical keys are its context_len[b]
 * cached tokens, then its nodes: node j's K and V are at logical key
 * context_len[b] + j.  Logical key p lies in block
 * block_table[b, p / block_size] at offset p % block_size.  Row i of the
 * sequence sees every context key, and node j where bit j of its mask row is
 * set (tree_mask NULL: every j <= i; one row: plain decoding).
 *   out[i, h] = sum_p w_p v_p / sum_p w_p,  w_p = exp(scale * q[i, h].k_p)
 * over the keys p that row i sees, h's KV head being h / (num_heads /
 * num_kv_heads).  A row that sees nothing gives 0 (lse -infinity); what a row
 * does not see never reaches it, be it infinite or NaN.  Scores, running
 * maximum, sums and outputs are FP32; the weights are rounded to bf16 for the
 * product with V (tensor cores), the output once to bf16.
 *
 *   q            bf16 [rows, num_heads, 64]: element (i, h, e) at
 *                i*q_row_stride + 64*h + e (e.g. the Q columns of
 *                rc_qkv_front's output), 16-byte aligned, q_row_stride a
 *                multiple of 8
 *   rows         0 <= rows, rows*num_heads < 2^31 - 256 (0: nothing launched, q and
 *                out may be NULL)
 *   num_heads    a multiple of num_kv_heads; num_kv_heads >= 1
 *   row_start    device int32 [seqs + 1], non-decreasing, within [0, rows]
 *                (values outside are clamped); rows of no sequence are left
 *   seqs         1 <= seqs < 2^24
 *   context_len  device int32 [seqs]
 *   block_table  device int32 [seqs, table_width], row stride table_stride
 *                elements.  Keys past table_width*block_size are not seen (one
 *                is added to *err per such sequence), nor are those of a block
 *                outside [0, num_blocks) (one per block that is needed)
 *   tree_mask    device uint64 [rows, mask_words], or NULL: bit j%64 of word
 *                j/64; nodes past the last word are not seen
 *   cache        bf16 [num_blocks, num_kv_heads, block_size, 128] (K | V),
 *                16-byte aligned; num_blocks*block_size < 2^31
 *   scale        > 0, finite (1/8 for 64-wide heads)
 *   out          bf16 [rows, num_heads, 64], as q with out_row_stride; 16-byte
 *                aligned; out, lse and the workspace overlap no other operand
 *   lse          optional FP32 [rows, num_heads]: log of the row's sum of
 *                exp(scale * q.k), to join results over several caches
 *   err          optional device int32 counter
 *   workspace    device scratch, 16-byte aligned, of
 *                rc_tree_attention_workspace_size() bytes, or NULL: then the
 *                keys of a sequence's KV head are not split over the GPU
 *                (slower for few rows over long contexts).  Calls sharing one
 *                must not overlap on the GPU; its contents need no set-up
 * Lengths stay on the device and the launches depend on the arguments alone,
 * so a captured call may be replayed with other lengths.  Results depend on
 * the arguments, not on timing.
 */
rc_status rc_tree_attention(const uint16_t *q, int64_t q_row_stride, int64_t rows, int32_t num_heads,
                            int32_t num_kv_heads, const int32_t *row_start, int32_t seqs,
                            const int32_t *context_len, const int32_t *block_table,
                            int64_t table_stride, int32_t table_width, const uint64_t *tree_mask,
                            int32_t mask_words, const uint16_t *cache, int32_t num_blocks,
                            int32_t block_size, float scale, uint16_t *out, int64_t out_row_stride,
                            float *lse, int32_t *err, void *workspace, size_t workspace_bytes,
                            cudaStream_t stream);

/* Workspace bytes of rc_tree_attention for these sizes on the current device
   (0 for sizes it refuses).  They never shrink with more rows, fewer sequences or
   more heads per KV head, so a workspace for the most rows, the fewest sequences
   that have them (one serves any) and the largest num_heads / num_kv_heads
   serves every call up to those. */
size_t rc_tree_attention_workspace_size(int64_t rows, int32_t seqs, int32_t num_heads,
                                        int32_t num_kv_heads);

/*
 * rc_logits_adjust -- penalties for repeated tokens, biases and grammar masks
 * on the logits of drafted (or single) tokens.  Rows belong to sequences as in
 * rc_tree_attention.  For row r of sequence b and token t, g counts t among
 * the sequence's generated history (its history past the first prompt_len[b]
 * tokens) and among the drafted tokens that the row's node sees (itself as the
 * mask says; without a mask every node up to its own); `said` is whether t
 * is in the prompt or g > 0.  In FP32, in this order (the quotient as a product
 * with the rounded 1 / repetition):
 *   x = logit;  if said: x = x > 0 ? x / repetition : x * repetition;
 *   if g > 0: x = x - frequency * g (fused), x = x - presence;
 *   x = x + bias of t;  if t is not allowed: x = -infinity
 * rounded once to `dtype`.
 *
 *   logits       `dtype` (rc_dtype) [rows, vocab], row stride row_stride
 *                elements, aligned to its element
 *   out          as logits with out_row_stride; may be logits with its stride
 *                (in place), else must not overlap it; overlaps no other operand
 *   rows         0 <= rows <= 2^30 (0: nothing launched, logits and out may be
 *                NULL); rows of no sequence
 *                are left
 *   vocab        1 <= vocab <= 2^30;  seqs: 1 .. 65535
 *   row_start    device int32 [seqs + 1], as in rc_tree_attention
 * Each of the following may be NULL, for none of it (repetition 1, frequency
 * and presence 0, everything allowed):
 *   history      device int32 [history_size], history_start[b] ..
 *                history_start[b+1] - 1 that of sequence b (device int64
 *                [seqs + 1]); history_size < 2^28
 *   prompt_len   device int32 [seqs] (NULL: no prompt, all generated)
 *   draft_tokens device int32 [rows], with tree_mask as in rc_tree_attention
 *   repetition, frequency, presence    device FP32 [seqs]
 *   bias_tokens, bias_values   device int32 and FP32 [bias_size],
 *                bias_start[b] .. bias_start[b+1] - 1 those of sequence b
 *                (device int32 [seqs + 1]); a token listed twice takes its last
 *                entry; bias_size < 2^31
 *   allowed      device uint32 words [rows, >= ceil(vocab / 32)], row stride
 *                allowed_stride words: bit t%32 of word t/32 set where t may
 *                come
 *   err          device int32 counter: one per token outside [0, vocab) in
 *                the history, the drafted tokens or the biases of a sequence
 *                with rows (such tokens count for nothing)
 */
typedef struct {
    const int32_t *history;
    int64_t history_size;
    const int64_t *history_start;
    const int32_t *prompt_len;
    const int32_t *draft_tokens;
    const uint64_t *tree_mask;
    int32_t mask_words;
    const float *repetition, *frequency, *presence;
    const int32_t *bias_start, *bias_tokens;
    const float *bias_values;
    int64_t bias_size;
    const uint32_t *allowed;
    int64_t allowed_stride;
} rc_logits_params;

rc_status rc_logits_adjust(const void *logits, int32_t dtype, int64_t row_stride, int64_t rows,
                           int32_t vocab, const int32_t *row_start, int32_t seqs,
                           const rc_logits_params *params, void *out, int64_t out_row_stride,
                           int32_t *err, cudaStream_t stream);

/* rc_device_address -- the address at which the current device reads p:
   p itself for device or managed memory; for page-locked host memory
   mapped into the device's address space (cudaHostAlloc, or
   cudaHostRegister with mapping), its device address (the same value under
   unified addressing).  Pass the start of the page-locked allocation; the
   device address of a byte inside it is the result plus that byte's offset
   (the Python binding maps slices of pinned tensors this way).
   RC_ERR_INVALID_ARG when the device cannot address p through the CUDA
   runtime (pageable host memory, NULL); dev untouched then.  Host-only; no
   page counterpart. */
rc_status rc_device_address(const void *p, const void **dev);

/* Sticky fault bits raised on the device when a bounded wait gives up: bits
   0-3 by the projection kernels, bits 8-11 by the QKV front, bits 16-19 by
   the tree attention (per kernel: load pipeline, tensor-core pipeline,
   accumulator, drain).  A kernel that
   sees a raised bit of its own kind skips its work, so after a fault its
   outputs are wrong until the bits are cleared.  Reads (and with clear != 0
   resets) the bits of the current device; synchronises the device.  No
   page counterpart. */
rc_status rc_read_device_faults(uint32_t *flags, int32_t clear);

#ifdef __cplusplus
}
#endif

#endif /* ROPE_CHAIN_H */
