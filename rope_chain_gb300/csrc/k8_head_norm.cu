// K8: RMS norm of each query and key head with its rotary position, and the
// gradients.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = R (n w)
//   g = R^T dy,  dw = sum g n,  dx = r (g w - n mean(g w n))
// in FP32, R the rotation of pairs (a, b) -> (a c - b s, b c + a s) by the table
// row of the token, each result rounded once.
//
// Bound by memory: forward one read and one write of every element, backward two
// reads (r is made again from x, which the gradient needs anyway) and one write.
#include "rc_paged.cuh"

#include <algorithm>

namespace rc {

namespace {

constexpr int kThreads = 256;

// kN elements of T as 32-bit words (bf16 in pairs).  kOne: in accesses of 16
// bytes, else element by element.
template <typename T, int kN> struct Run {
    static constexpr int kWords = (int)sizeof(T) * kN >= 4 ? (int)sizeof(T) * kN / 4 : 1;
    uint32_t w[kWords];

    template <bool kOne> __device__ __forceinline__ void get(const T *p) {
        if constexpr (kOne) {
            const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
            w[0] = v.x;
            w[1 % kWords] = v.y;
            w[2 % kWords] = v.z;
            w[3 % kWords] = v.w;
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                w[i] = reinterpret_cast<const uint32_t *>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < kN; i += 2)
                w[i / 2] = (uint32_t)reinterpret_cast<const uint16_t *>(p)[i] |
                           (i + 1 < kN ? (uint32_t)reinterpret_cast<const uint16_t *>(p)[i + 1] << 16 : 0u);
        }
    }
    template <bool kOne> __device__ __forceinline__ void put(T *p) const {
        if constexpr (kOne) {
            __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1 % kWords], w[2 % kWords], w[3 % kWords]));
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                reinterpret_cast<uint32_t *>(p)[i] = w[i];
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[i] = 0u;
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
    __device__ __forceinline__ void set(const float (&v)[kN]) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            if constexpr (sizeof(T) == 4)
                w[i] = __float_as_uint(v[i]);
            else if (i % 2 == 0)
                w[i / 2] = pack_bf16x2(v[i], i + 1 < kN ? v[(i + 1) % kN] : 0.0f);
        }
    }
};

// kN values at element `at` of a bf16 or FP32 array; kOne: it is aligned to the
// bytes of kN of its elements (at most 16).
template <int kN, bool kOne>
__device__ __forceinline__ void values(const void *p, bool f32, int64_t at, float (&v)[kN]) {
    if (f32) {
        const float *src = static_cast<const float *>(p) + at;
        if constexpr (kOne && kN >= 4) {
#pragma unroll
            for (int i = 0; i < kN; i += 4) {
                const float4 q = __ldg(reinterpret_cast<const float4 *>(src + i));
                v[i] = q.x;
                v[i + 1] = q.y;
                v[i + 2] = q.z;
                v[i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                v[i] = __ldg(src + i);
        }
        return;
    }
    const uint16_t *src = static_cast<const uint16_t *>(p) + at;
    if constexpr (kOne && kN % 2 == 0) {
        uint32_t w[kN / 2];
        if constexpr (kN == 8) {
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(src));
            w[0] = q.x;
            w[1] = q.y;
            w[2] = q.z;
            w[3] = q.w;
        } else if constexpr (kN == 4) {
            const uint2 q = __ldg(reinterpret_cast<const uint2 *>(src));
            w[0] = q.x;
            w[1] = q.y;
        } else {
#pragma unroll
            for (int i = 0; i < kN / 2; ++i)
                w[i] = __ldg(reinterpret_cast<const uint32_t *>(src) + i);
        }
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
            v[i] = bf16_lo(w[i / 2]);
            v[i + 1] = bf16_hi(w[i / 2]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i)
            v[i] = __uint_as_float((uint32_t)__ldg(src + i) << 16);
    }
}

// The rotation of pair (a, b), or (kBack) its transpose.
template <bool kBack> __device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    if (kBack)
        s = -s;
    const float x = __fmaf_rn(a, c, -__fmul_rn(b, s));
    b = __fmaf_rn(b, c, __fmul_rn(a, s));
    a = x;
}

// The sum over the `lanes` (a power of two) lanes of a head, in every one of them.
__device__ __forceinline__ float head_sum(float v, int lanes) {
    for (int o = lanes >> 1; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

struct NormArgs : HeadNormLaunch {
    int32_t lanes;                       // lanes of a head: a power of two <= 32
    int32_t groups[2];                   // groups of kHeads heads of the queries and of the keys
    float inv_width;
    int32_t blocks;                      // of a kind (gradient)
};

// A head's units of kVec elements (HALVES: kVec of each half; past rot_dim kVec) go
// to consecutive lanes, kU to a lane.  What a lane has of kHeads heads of one kind
// (queries or keys) of one token, whose table columns and weights are read once.
template <typename T, bool kHalves, int kVec, int kU, int kHeads> struct Lane {
    static constexpr bool kOne = kVec * sizeof(T) == 16;
    static constexpr int kParts = kHalves ? 2 : 1;          // runs of kVec elements of a unit
    static constexpr int kPairs = kHalves ? kVec : (kVec > 1 ? kVec / 2 : 1);

    // the unit's first element, or -1 past the last unit; whether it is turned
    static __device__ __forceinline__ int place(const NormArgs &a, int i, bool &rot) {
        const int u = (threadIdx.x & (a.lanes - 1)) + i * a.lanes;
        const int rotated = kHalves ? a.rot / (2 * kVec) : a.rot / kVec;
        rot = u < rotated;
        const int at = rot ? u * kVec : a.rot + (u - rotated) * kVec;
        return at < a.width ? at : -1;
    }
    static __device__ __forceinline__ void load(const NormArgs &a, const T *head, Run<T, kVec> (&v)[kU][kParts]) {
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            bool rot;
            const int at = place(a, i, rot);
#pragma unroll
            for (int p = 0; p < kParts; ++p)
                v[i][p].clear();
            if (at >= 0) {
                v[i][0].template get<kOne>(head + at);
                if (kHalves && rot)
                    v[i][kParts - 1].template get<kOne>(head + at + a.rot / 2);
            }
        }
    }
    static __device__ __forceinline__ void table(const NormArgs &a, int64_t pos, int at, bool rot, float (&c)[kPairs],
                                                 float (&s)[kPairs]) {
        if (rot) {
            const int64_t from = pos * a.rot + (kHalves ? at : at / 2);
            values<kPairs, kOne>(a.table, a.table_f32 != 0, from, c);
            values<kPairs, kOne>(a.table, a.table_f32 != 0, from + a.rot / 2, s);
        }
    }
    // a unit's values, turned by (c, s)
    template <bool kBack>
    static __device__ __forceinline__ void rotate(float (&y)[kParts][kVec], const float (&c)[kPairs], const float (&s)[kPairs]) {
        if constexpr (kHalves) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                turn<kBack>(y[0][j], y[1][j], c[j], s[j]);
        } else if constexpr (kVec > 1) {
#pragma unroll
            for (int j = 0; j < kVec; j += 2)
                turn<kBack>(y[0][j], y[0][j + 1], c[j / 2], s[j / 2]);
        }
    }
};

// Items are (token, group of heads); a group holds heads of one kind.
template <int kHeads> struct Item {
    int64_t t;
    int kind, h0, heads;                 // heads: how many of the group exist
    __device__ __forceinline__ Item(const NormArgs &a, int64_t item, int groups, int only) {
        const uint32_t token = (uint32_t)item / (uint32_t)groups;
        int g = (int)((uint32_t)item - token * (uint32_t)groups);
        t = token;
        kind = only >= 0 ? only : (g < a.groups[0] ? 0 : 1);
        if (only < 0 && kind == 1)
            g -= a.groups[0];
        const int first = kind == 0 ? 0 : a.q_heads, last = kind == 0 ? a.q_heads : a.heads;
        h0 = first + g * kHeads;
        heads = min(kHeads, last - h0);
    }
};

template <typename T, bool kHalves, int kVec, int kU, int kHeads>
__global__ void __launch_bounds__(kThreads)
k8_head_norm(const __grid_constant__ NormArgs a)
{
    using L = Lane<T, kHalves, kVec, kU, kHeads>;
    pdl_trigger();
    pdl_wait();
    const int groups = a.groups[0] + a.groups[1];
    const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / a.lanes;
    const bool live = item < a.T * groups;               // (all lanes stay for the sums)
    const Item<kHeads> it(a, live ? item : 0, groups, -1);
    const int64_t pos = __ldg(a.positions + it.t);
    const bool bad = pos < 0 || pos >= a.max_position;
    const T *src = static_cast<const T *>(a.x) + it.t * a.x_row_stride + it.h0 * a.x_head_stride;
    Run<T, kVec> v[kHeads][kU][L::kParts];
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
        if (live && k < it.heads)
            L::load(a, src + k * a.x_head_stride, v[k]);
        else
#pragma unroll
            for (int i = 0; i < kU; ++i)
#pragma unroll
                for (int p = 0; p < L::kParts; ++p)
                    v[k][i][p].clear();
    if (live && bad && it.h0 == 0 && (threadIdx.x & (a.lanes - 1)) == 0 && a.err != nullptr)
        atomicAdd(a.err, 1);
    float r[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kU; ++i)
#pragma unroll
            for (int p = 0; p < L::kParts; ++p)
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    sum = __fmaf_rn(v[k][i][p].at(j), v[k][i][p].at(j), sum);
        r[k] = rsqrtf(__fmaf_rn(head_sum(sum, a.lanes), a.inv_width, a.eps));
    }
    if (!live)
        return;
    T *dst = static_cast<T *>(a.out) + it.t * a.out_row_stride + it.h0 * a.out_head_stride;
    const void *weight = a.weight[it.kind];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        bool rot;
        const int at = L::place(a, i, rot);
        if (at < 0)
            continue;
        float c[L::kPairs], s[L::kPairs], w[L::kParts][kVec];
        L::table(a, pos, at, rot && !bad, c, s);
#pragma unroll
        for (int p = 0; p < L::kParts; ++p) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                w[p][j] = 1.0f;
            if (weight != nullptr && (p == 0 || rot))
                values<kVec, L::kOne>(weight, a.weight_f32 != 0, at + p * (a.rot / 2), w[p]);
        }
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            if (k >= it.heads)
                break;
            float y[L::kParts][kVec];
#pragma unroll
            for (int p = 0; p < L::kParts; ++p)
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    y[p][j] = v[k][i][p].at(j) * r[k] * w[p][j];
            if (rot && !bad)
                L::template rotate<false>(y, c, s);
#pragma unroll
            for (int p = 0; p < L::kParts; ++p) {
                if (p > 0 && !rot)
                    continue;
                Run<T, kVec> o;
                o.set(y[p]);
                o.template put<L::kOne>(dst + k * a.out_head_stride + at + p * (a.rot / 2));
            }
        }
    }
}

// The gradient.  blockIdx.y is the kind (queries, keys), so that a thread's part
// of dw is of one weight and of the same elements throughout; a kind's blocks take
// its items in turn, and leave their sums, joined over the block's heads, in the
// workspace, which k8_weight_grad adds up in the order of the blocks.
template <typename T, bool kHalves, int kVec, int kU, int kHeads>
__global__ void __launch_bounds__(kThreads)
k8_head_norm_grad(const __grid_constant__ NormArgs a)
{
    using L = Lane<T, kHalves, kVec, kU, kHeads>;
    __shared__ float s_sum[kThreads / 32][kMaxNormDim];
    pdl_trigger();
    pdl_wait();
    const int kind = blockIdx.y, groups = a.groups[kind];
    const int64_t items = a.T * groups;
    const int side = kThreads / a.lanes;                  // heads side by side in a block
    const void *weight = a.weight[kind];
    const bool wanted = a.dweight[kind] != nullptr;
    float w[kU][L::kParts][kVec], dw[kU][L::kParts][kVec];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        bool rot;
        const int at = L::place(a, i, rot);
#pragma unroll
        for (int p = 0; p < L::kParts; ++p) {
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                w[i][p][j] = 1.0f;
                dw[i][p][j] = 0.0f;
            }
            if (weight != nullptr && at >= 0 && (p == 0 || rot))
                values<kVec, L::kOne>(weight, a.weight_f32 != 0, at + p * (a.rot / 2), w[i][p]);
        }
    }
    // uniform over the block: all lanes stay for the sums
    for (int64_t base = (int64_t)blockIdx.x * side; base < items; base += (int64_t)gridDim.x * side) {
        const int64_t item = base + threadIdx.x / a.lanes;
        const bool live = item < items;
        const Item<kHeads> it(a, live ? item : 0, groups, kind);
        const int64_t pos = __ldg(a.positions + it.t);
        const bool bad = pos < 0 || pos >= a.max_position;
        const T *src = static_cast<const T *>(a.x) + it.t * a.x_row_stride + it.h0 * a.x_head_stride;
        const T *dsrc = static_cast<const T *>(a.dy) + it.t * a.dy_row_stride + it.h0 * a.dy_head_stride;
        Run<T, kVec> v[kHeads][kU][L::kParts], d[kHeads][kU][L::kParts];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            if (live && k < it.heads) {
                L::load(a, src + k * a.x_head_stride, v[k]);
                L::load(a, dsrc + k * a.dy_head_stride, d[k]);
            } else {
#pragma unroll
                for (int i = 0; i < kU; ++i)
#pragma unroll
                    for (int p = 0; p < L::kParts; ++p) {
                        v[k][i][p].clear();
                        d[k][i][p].clear();
                    }
            }
        }
        if (live && bad && it.h0 == 0 && (threadIdx.x & (a.lanes - 1)) == 0 && a.err != nullptr)
            atomicAdd(a.err, 1);
        float c[kU][L::kPairs], s[kU][L::kPairs];
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            bool rot;
            const int at = L::place(a, i, rot);
            L::table(a, pos, at, at >= 0 && rot && !bad, c[i], s[i]);
        }
        T *dst = static_cast<T *>(a.out) + it.t * a.out_row_stride + it.h0 * a.out_head_stride;
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            float g[kU][L::kParts][kVec], sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                bool rot;
                const int at = L::place(a, i, rot);
#pragma unroll
                for (int p = 0; p < L::kParts; ++p)
#pragma unroll
                    for (int j = 0; j < kVec; ++j)
                        g[i][p][j] = d[k][i][p].at(j);
                if (at >= 0 && rot && !bad)
                    L::template rotate<true>(g[i], c[i], s[i]);
#pragma unroll
                for (int p = 0; p < L::kParts; ++p)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        const float x = v[k][i][p].at(j);
                        sum = __fmaf_rn(x, x, sum);
                        dot = __fmaf_rn(g[i][p][j] * w[i][p][j], x, dot);
                    }
            }
            const float r = rsqrtf(__fmaf_rn(head_sum(sum, a.lanes), a.inv_width, a.eps));
            const float along = head_sum(dot, a.lanes) * r * a.inv_width;        // mean(g w n)
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                bool rot;
                const int at = L::place(a, i, rot);
                float y[L::kParts][kVec];
#pragma unroll
                for (int p = 0; p < L::kParts; ++p)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        const float n = v[k][i][p].at(j) * r;
                        if (live && k < it.heads)         // (else r may be infinite)
                            dw[i][p][j] = __fmaf_rn(g[i][p][j], n, dw[i][p][j]);
                        y[p][j] = r * __fmaf_rn(g[i][p][j], w[i][p][j], -(n * along));
                    }
                if (!live || at < 0 || k >= it.heads)
                    continue;
#pragma unroll
                for (int p = 0; p < L::kParts; ++p) {
                    if (p > 0 && !rot)
                        continue;
                    Run<T, kVec> o;
                    o.set(y[p]);
                    o.template put<L::kOne>(dst + k * a.out_head_stride + at + p * (a.rot / 2));
                }
            }
        }
    }
    if (!wanted)
        return;
    // over the heads of a warp, then over the warps
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        bool rot;
        const int at = L::place(a, i, rot);
#pragma unroll
        for (int p = 0; p < L::kParts; ++p)
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                float x = dw[i][p][j];
                for (int o = 16; o >= a.lanes; o >>= 1)
                    x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                if (at >= 0 && lane < a.lanes && (p == 0 || rot))
                    s_sum[warp][at + p * (a.rot / 2) + j] = x;
            }
    }
    __syncthreads();
    float *part = a.partial + ((int64_t)kind * a.blocks + blockIdx.x) * a.width;
    for (int e = threadIdx.x; e < a.width; e += kThreads) {
        float x = 0.0f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k)
            x += s_sum[k][e];
        part[e] = x;
    }
}

// dw from the blocks' sums: a block has 32 columns, its warps take every eighth
// part each and are joined in order.
__global__ void __launch_bounds__(kThreads)
k8_weight_grad(const __grid_constant__ NormArgs a)
{
    __shared__ float s_sum[kThreads / 32][32];
    pdl_trigger();
    pdl_wait();
    const int kind = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    if (a.dweight[kind] == nullptr)
        return;
    float x = 0.0f;
    // (no block of a kind without heads has left any)
    const int blocks = a.groups[kind] > 0 && a.T > 0 ? a.blocks : 0;
    if (e < a.width)
        for (int b = warp; b < blocks; b += kThreads / 32)
            x += a.partial[((int64_t)kind * a.blocks + b) * a.width + e];
    s_sum[warp][lane] = x;
    __syncthreads();
    if (warp == 0 && e < a.width) {
#pragma unroll
        for (int k = 1; k < kThreads / 32; ++k)
            x += s_sum[k][lane];
        a.dweight[kind][e] = x;
    }
}

constexpr int kGradBlocksPerSm = 4;

template <typename T, bool kHalves, int kVec, int kU, int kHeads>
cudaError_t launch_kind(const HeadNormLaunch &p, int units, int num_sms, cudaStream_t stream)
{
    NormArgs a{};
    static_cast<HeadNormLaunch &>(a) = p;
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes < units)
        a.lanes *= 2;
    a.groups[0] = (p.q_heads + kHeads - 1) / kHeads;
    a.groups[1] = (p.heads - p.q_heads + kHeads - 1) / kHeads;
    a.inv_width = 1.0f / (float)p.width;
    if (p.dy == nullptr) {
        const int64_t threads = p.T * (a.groups[0] + a.groups[1]) * a.lanes;
        return launch_pdl(k8_head_norm<T, kHalves, kVec, kU, kHeads>, dim3((unsigned)((threads + kThreads - 1) / kThreads)),
                          dim3(kThreads), 0, stream, 1, a);
    }
    const bool weights = a.dweight[0] != nullptr || a.dweight[1] != nullptr;
    const int side = kThreads / a.lanes;
    const int64_t items = p.T * std::max(a.groups[0], a.groups[1]);
    a.blocks = (int)std::max<int64_t>(1, std::min<int64_t>((items + side - 1) / side, (int64_t)num_sms * kGradBlocksPerSm));
    cudaError_t e = cudaSuccess;
    if (p.T > 0)
        e = launch_pdl(k8_head_norm_grad<T, kHalves, kVec, kU, kHeads>, dim3((unsigned)a.blocks, 2), dim3(kThreads), 0,
                       stream, 1, a);
    if (e == cudaSuccess && weights)
        e = launch_pdl(k8_weight_grad, dim3((unsigned)((p.width + 31) / 32), 2), dim3(kThreads), 0, stream, 1, a);
    return e;
}

template <typename T, bool kHalves>
cudaError_t launch_type(const HeadNormLaunch &a, bool wide, int num_sms, cudaStream_t stream)
{
    constexpr int kWide = 16 / (int)sizeof(T), kNarrow = kHalves ? 1 : 2;
    const int vec = wide ? kWide : kNarrow;
    const int units = (kHalves ? a.rot / (2 * vec) : a.rot / vec) + (a.width - a.rot) / vec;
    if (!wide)                              // up to 511 units of an element or two
        return launch_kind<T, kHalves, kNarrow, 16, 1>(a, units, num_sms, stream);
    if (units > 32)                         // up to 128
        return launch_kind<T, kHalves, kWide, 4, 1>(a, units, num_sms, stream);
    // Several heads a thread, whose table columns are read once, where there is
    // work to fill the GPU that way.
    constexpr int kMany = 2;
    const bool many = a.T * a.heads * units >= (int64_t)kMany * num_sms * 2048;
    return many ? launch_kind<T, kHalves, kWide, 1, kMany>(a, units, num_sms, stream)
                : launch_kind<T, kHalves, kWide, 1, 1>(a, units, num_sms, stream);
}

}  // namespace

size_t head_norm_grad_workspace(int32_t width, int num_sms)
{
    return (size_t)2 * num_sms * kGradBlocksPerSm * width * sizeof(float);
}

cudaError_t launch_head_norm_rope(const HeadNormLaunch &a, bool f32, bool halves, bool wide, int num_sms,
                                  cudaStream_t stream)
{
    if (f32)
        return halves ? launch_type<float, true>(a, wide, num_sms, stream) : launch_type<float, false>(a, wide, num_sms, stream);
    return halves ? launch_type<uint16_t, true>(a, wide, num_sms, stream)
                  : launch_type<uint16_t, false>(a, wide, num_sms, stream);
}

}  // namespace rc
