// K8: RMS norm of each query and key head with its rotary position, and the
// gradients.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = R (n w)
//   g = R^T dy,  dw = sum g n,  dx = r (g w - n mean(g w n))
// in FP32, R the rotation of pairs (a, b) -> (a c - b s, b c + a s) by the table
// row of the token, each result rounded once.
//
// Bound by memory: forward one read and one write of every element, backward two
// reads (r is made again from x, which the gradient needs anyway) and one write.  To be
// there the work of an element must stay small, so a lane takes 16 bytes or two times
// 16 of a head, up to eight heads one after another, whose table columns and weights it
// loads once, and FP32 arithmetic goes in pairs.  Measured, 16384 tokens of 32 + 8 heads
// of 128: bf16 halves 53 us forward (6.4 TB/s) and 86 backward (5.9), pairs 53 and 86,
// FP32 halves 100 and 155; one head at a time straight into registers 67 and 107.
// Heads of 96 leave four lanes of 16 idle (49 and 90 us for 40 of them).
#include "rc_paged.cuh"
#include "rc_tcgen05.cuh"

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
    __device__ __forceinline__ void from_shared(uint32_t at) {      // 16 bytes
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1 % kWords]), "=r"(w[2 % kWords]), "=r"(w[3 % kWords]) : "r"(at) : "memory");
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

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

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

// The sum over the `lanes` (a power of two) lanes of a head, in every one of them.
__device__ __forceinline__ float head_sum(float v, int lanes) {
    for (int o = lanes >> 1; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

struct NormArgs : HeadNormLaunch {
    int32_t lanes, lanes_log2;           // lanes of a head: a power of two <= 32
    int32_t per;                         // heads of an item at most
    int32_t groups[2];                   // items of the queries and of the keys of a token
    float inv_width;
    int32_t blocks;                      // of a kind (gradient)
};

// A head's units of kVec elements (HALVES: kVec of each half, and past rot_dim kVec of
// each half of the rest, whose first may be one longer) go to consecutive lanes, kU to a
// lane.  In FP32 a unit is kPairs pairs (p, q): the pairs that turn, or two elements that
// do not (12000 x 16 heads of 64 in BF16, 32 elements of which turn, 10.6 us and the
// gradient 19.8; with one run to a unit of the rest 19.0 and 34.8).
template <typename T, bool kHalves, int kVec, int kU> struct Lane {
    static constexpr bool kOne = kVec * sizeof(T) == 16;
    static constexpr int kParts = kHalves ? 2 : 1;          // runs of kVec elements of a unit
    static constexpr int kPairs = kHalves ? kVec : kVec / 2;
    using Raw = Run<T, kVec>[kU][kParts];

    // Of each unit of the lane: its first element (turned: below rot), or -1 past the last
    // unit; HALVES: how far behind it its second run is, 0 without one.
    struct Spots {
        int at[kU], by[kU];
        __device__ __forceinline__ explicit Spots(const NormArgs &a) {
            const int turned = a.rot / (2 * kVec), rest = (a.width - a.rot) / kVec, units = (rest + 1) / 2;
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const int u = (threadIdx.x & (a.lanes - 1)) + i * a.lanes, v = u - turned;
                at[i] = !kHalves || v < 0 ? u * kVec : a.rot + v * kVec;
                if (kHalves ? v >= units : at[i] >= a.width)
                    at[i] = -1;
                by[i] = !kHalves ? 0 : (v < 0 ? a.rot / 2 : (v + units < rest ? units * kVec : 0));
            }
        }
        // Whether unit i's pairs turn, at a position that the table has (not `bad`).  Where
        // they do not, nothing of one element goes to the other, not even 0 times it, which
        // is NaN for an infinity (the branch costs at most 1 % forward, 1 to 3 backward;
        // predicated products instead cost 1 to 5).
        __device__ __forceinline__ bool turned(const NormArgs &a, int i, bool bad) const {
            return at[i] >= 0 && at[i] < a.rot && !bad;
        }
    };
    // what a lane has of the head at `head` (NULL: zeros)
    static __device__ __forceinline__ void load(const Spots &spot, const T *head, Raw &v) {
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            const int at = spot.at[i], by = spot.by[i];
#pragma unroll
            for (int p = 0; p < kParts; ++p)
                v[i][p].clear();
            if (head != nullptr && at >= 0) {
                v[i][0].template get<kOne>(head + at);
                if (kHalves && by != 0)
                    v[i][kParts - 1].template get<kOne>(head + at + by);
            }
        }
    }
    // The same through shared memory (16-byte accesses): copied there ahead, into the
    // lane's own places from `to` on, kThreads * 16 bytes apart, and read by it alone.
    static constexpr uint32_t kBytes = kU * kParts * kThreads * 16;
    static __device__ __forceinline__ void copy(const Spots &spot, const T *head, uint32_t to) {
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            const int at = spot.at[i], by = spot.by[i];
            if (head == nullptr || at < 0)
                continue;
            copy16(to + (i * kParts) * (kThreads * 16), head + at);
            if (kHalves && by != 0)
                copy16(to + (i * kParts + 1) * (kThreads * 16), head + at + by);
        }
    }
    static __device__ __forceinline__ void copied(const Spots &spot, bool there, uint32_t from, Raw &v) {
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            const int at = spot.at[i], by = spot.by[i];
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                v[i][p].clear();
                if (there && at >= 0 && (p == 0 || by != 0))
                    v[i][p].from_shared(from + (i * kParts + p) * (kThreads * 16));
            }
        }
    }
    static __device__ __forceinline__ void store(const Spots &spot, T *head, int i, const float (&p)[kPairs], const float (&q)[kPairs]) {
        const int at = spot.at[i], by = spot.by[i];
        if (at < 0)
            return;
        Run<T, kVec> o;
        if constexpr (kHalves) {
            o.set(p);
            o.template put<kOne>(head + at);
            if (by != 0) {
                o.set(q);
                o.template put<kOne>(head + at + by);
            }
        } else {
            float both[kVec];
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                both[2 * j] = p[j];
                both[2 * j + 1] = q[j];
            }
            o.set(both);
            o.template put<kOne>(head + at);
        }
    }
    static __device__ __forceinline__ void pairs(const Run<T, kVec> (&v)[kParts], float (&p)[kPairs], float (&q)[kPairs]) {
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            p[j] = v[0].at(kHalves ? j : 2 * j);
            q[j] = kHalves ? v[kParts - 1].at(j) : v[0].at(2 * j + 1);
        }
    }
    // the table's columns of unit i (1 and 0 where it is not turned)
    static __device__ __forceinline__ void table(const NormArgs &a, const Spots &spot, int64_t pos, bool bad, int i, float (&c)[kPairs], float (&s)[kPairs]) {
        const int at = spot.at[i], by = spot.by[i];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            c[j] = 1.0f;
            s[j] = 0.0f;
        }
        if (spot.turned(a, i, bad)) {
            const int64_t from = pos * a.rot + (kHalves ? at : at / 2);
            values<kPairs, kOne>(a.table, a.table_f32 != 0, from, c);
            values<kPairs, kOne>(a.table, a.table_f32 != 0, from + a.rot / 2, s);
        }
    }
    static __device__ __forceinline__ void weights(const NormArgs &a, const Spots &spot, int kind, int i, float (&p)[kPairs], float (&q)[kPairs]) {
        const int at = spot.at[i], by = spot.by[i];
#pragma unroll
        for (int j = 0; j < kPairs; ++j)
            p[j] = q[j] = 1.0f;
        if (a.weight[kind] == nullptr || at < 0)
            return;
        if constexpr (kHalves) {
            values<kPairs, kOne>(a.weight[kind], a.weight_f32 != 0, at, p);
            if (by != 0)
                values<kPairs, kOne>(a.weight[kind], a.weight_f32 != 0, at + by, q);
        } else {
            float both[kVec];
            values<kVec, kOne>(a.weight[kind], a.weight_f32 != 0, at, both);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) {
                p[j] = both[2 * j];
                q[j] = both[2 * j + 1];
            }
        }
    }
};

// Two at a time where there are two: (a, b) <- f(a, b), FP32 pairs.
template <int kN> __device__ __forceinline__ void scale(float (&v)[kN], float r) {
#pragma unroll
    for (int j = 0; j + 1 < kN; j += 2)
        mul2_rn(v[j], v[j + 1], r, r);
    if (kN % 2)
        v[kN - 1] *= r;
}
// v * w
template <int kN> __device__ __forceinline__ void times(float (&v)[kN], const float (&w)[kN]) {
#pragma unroll
    for (int j = 0; j + 1 < kN; j += 2)
        mul2_rn(v[j], v[j + 1], w[j], w[j + 1]);
    if (kN % 2)
        v[kN - 1] *= w[kN - 1];
}
// d <- v * w + d
template <int kN> __device__ __forceinline__ void add_product(float (&d)[kN], const float (&v)[kN], const float (&w)[kN]) {
#pragma unroll
    for (int j = 0; j + 1 < kN; j += 2) {
        float x = v[j], y = v[j + 1];
        fma2_rn(x, y, w[j], w[j + 1], d[j], d[j + 1]);
        d[j] = x;
        d[j + 1] = y;
    }
    if (kN % 2)
        d[kN - 1] = __fmaf_rn(v[kN - 1], w[kN - 1], d[kN - 1]);
}
template <int kN> __device__ __forceinline__ float sum_of(const float (&v)[kN]) {
    float x = v[0];
#pragma unroll
    for (int j = 1; j < kN; ++j)
        x += v[j];
    return x;
}

// Items are (token, up to `per` heads of one kind), of consecutive lanes.
struct Item {
    int64_t t;
    int kind, h0, heads;                 // heads: how many of them exist
    __device__ __forceinline__ Item(const NormArgs &a, int64_t item, int groups, int only) {
        const uint32_t token = (uint32_t)item / (uint32_t)groups;
        int g = (int)((uint32_t)item - token * (uint32_t)groups);
        t = token;
        kind = only >= 0 ? only : (g < a.groups[0] ? 0 : 1);
        if (only < 0 && kind == 1)
            g -= a.groups[0];
        const int first = kind == 0 ? 0 : a.q_heads, last = kind == 0 ? a.q_heads : a.heads;
        h0 = first + g * a.per;
        heads = min(a.per, last - h0);
    }
};

// What a token and a weight make of a pair's turn is the same for all heads of an
// item: y_p = r (p w_p c - q w_q s), y_q = r (q w_q c + p w_p s), four factors a pair.
// Heads come through a ring of kStages copies per lane in shared memory (kRing), which
// no other lane reads, so nothing is waited for but the copy; or, with an item of one
// head or in narrow accesses, straight into registers.
constexpr int kStages = 4;
template <typename T, bool kHalves, int kVec, int kU, bool kRing>
__global__ void __launch_bounds__(kThreads, kRing && kU == 1 ? 3 : 1)
k8_head_norm(const __grid_constant__ NormArgs a)
{
    using L = Lane<T, kHalves, kVec, kU>;
    constexpr int kP = L::kPairs;
    const typename L::Spots spot(a);
    extern __shared__ __align__(16) uint8_t s_ring[];
    pdl_trigger();
    pdl_wait();
    const int groups = a.groups[0] + a.groups[1];
    const int64_t item = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> a.lanes_log2;
    const bool live = item < a.T * groups;               // (all lanes stay for the sums)
    const Item it(a, live ? item : 0, groups, -1);
    const int heads = live ? it.heads : 0;
    const T *src = static_cast<const T *>(a.x) + it.t * a.x_row_stride + it.h0 * a.x_head_stride;
    T *dst = static_cast<T *>(a.out) + it.t * a.out_row_stride + it.h0 * a.out_head_stride;
    typename L::Raw v;
    const uint32_t ring = smem_u32(s_ring) + threadIdx.x * 16;
    if constexpr (kRing) {
#pragma unroll
        for (int h = 0; h < kStages - 1; ++h) {
            L::copy(spot, h < heads ? src + h * a.x_head_stride : nullptr, ring + h * L::kBytes);
            copy_commit();
        }
    } else {
        L::load(spot, heads > 0 ? src : nullptr, v);
    }
    const int64_t pos = __ldg(a.positions + it.t);
    const bool bad = pos < 0 || pos >= a.max_position;
    if (live && bad && it.h0 == 0 && (threadIdx.x & (a.lanes - 1)) == 0 && a.err != nullptr)
        atomicAdd(a.err, 1);
    float pp[kU][kP], pq[kU][kP], qp[kU][kP], qq[kU][kP];    // to p from p and from q, to q from p and from q
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        float wp[kP], wq[kP];
        L::table(a, spot, pos, bad, i, pp[i], pq[i]);
        L::weights(a, spot, it.kind, i, wp, wq);
#pragma unroll
        for (int j = 0; j < kP; ++j) {
            const float c = pp[i][j], s = pq[i][j];
            pp[i][j] = wp[j] * c;
            pq[i][j] = -(wq[j] * s);
            qp[i][j] = wp[j] * s;
            qq[i][j] = wq[j] * c;
        }
    }
    int st = 0;
    for (int h = 0; h < (kRing ? a.per : 1); ++h) {
        if constexpr (kRing) {
            copy_wait<kStages - 2>();
            L::copied(spot, h < heads, ring + st * L::kBytes, v);
        }
        float p[kU][kP], q[kU][kP], squares[kP];
#pragma unroll
        for (int j = 0; j < kP; ++j)
            squares[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            L::pairs(v[i], p[i], q[i]);
            add_product(squares, p[i], p[i]);
            add_product(squares, q[i], q[i]);
        }
        const float sum = head_sum(sum_of(squares), a.lanes);
        if constexpr (kRing) {
            // into the place of the head before, long read
            const int next = h + kStages - 1;
            L::copy(spot, next < heads ? src + next * a.x_head_stride : nullptr, ring + ((st + kStages - 1) % kStages) * L::kBytes);
            copy_commit();
            st = st + 1 == kStages ? 0 : st + 1;
        }
        const float r = rsqrtf(__fmaf_rn(sum, a.inv_width, a.eps));
        if (h >= heads)
            continue;
        T *head = dst + h * a.out_head_stride;
#pragma unroll
        for (int i = 0; i < kU; ++i) {
            scale(p[i], r);
            scale(q[i], r);
            float y[kP], z[kP];
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                y[j] = p[i][j];
                z[j] = 0.0f;
            }
            times(y, pp[i]);
            if (spot.turned(a, i, bad)) {
                add_product(y, q[i], pq[i]);
#pragma unroll
                for (int j = 0; j < kP; ++j)
                    z[j] = p[i][j];
                times(z, qp[i]);
            }
            add_product(z, q[i], qq[i]);
            L::store(spot, head, i, y, z);
        }
    }
}

// The gradient.  blockIdx.y is the kind (queries, keys), so that a thread's part
// of dw is of one weight and of the same elements throughout; a kind's blocks take
// its items in turn, and leave their sums, joined over the block's heads, in the
// workspace, which k8_weight_grad adds up in the order of the blocks.
// The heads' x and dy come through the ring, which runs on from item to item.
// Blocks that an SM holds, and as many of a kind are launched: more of them only begin
// and end more often.
constexpr int kMaxGradPerSm = 2;
template <typename T, bool kHalves, int kU> constexpr int kGradPerSm = kU > 2 || (kHalves && kU == 2) ? 1 : kMaxGradPerSm;
template <typename T, bool kHalves, int kVec, int kU, bool kRing>
__global__ void __launch_bounds__(kThreads, kGradPerSm<T, kHalves, kU>)
k8_head_norm_grad(const __grid_constant__ NormArgs a)
{
    using L = Lane<T, kHalves, kVec, kU>;
    constexpr int kP = L::kPairs;
    const typename L::Spots spot(a);
    extern __shared__ __align__(16) uint8_t s_ring[];
    __shared__ float s_sum[kThreads / 32][kMaxNormDim];
    pdl_trigger();
    pdl_wait();
    const int kind = blockIdx.y, groups = a.groups[kind];
    const int64_t items = a.T * groups;
    const int side = kThreads >> a.lanes_log2;            // heads side by side in a block
    const bool wanted = a.dweight[kind] != nullptr;
    float wp[kU][kP], wq[kU][kP], dp[kU][kP], dq[kU][kP];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        L::weights(a, spot, kind, i, wp[i], wq[i]);
#pragma unroll
        for (int j = 0; j < kP; ++j)
            dp[i][j] = dq[i][j] = 0.0f;
    }
    const uint32_t ring = smem_u32(s_ring) + threadIdx.x * 16;
    const int64_t stride = (int64_t)gridDim.x * side, mine = (int64_t)blockIdx.x * side + (threadIdx.x >> a.lanes_log2);
    // the head that is copied next: item `ahead`, head h_ahead of it
    int64_t ahead = mine;
    int h_ahead = 0, heads_ahead = 0;
    const T *x_ahead = nullptr, *dy_ahead = nullptr;
    auto copy_next = [&](int st) {
        if (h_ahead == 0) {
            heads_ahead = 0;
            if (ahead < items) {
                const Item it(a, ahead, groups, kind);
                heads_ahead = it.heads;
                x_ahead = static_cast<const T *>(a.x) + it.t * a.x_row_stride + it.h0 * a.x_head_stride;
                dy_ahead = static_cast<const T *>(a.dy) + it.t * a.dy_row_stride + it.h0 * a.dy_head_stride;
            }
        }
        const bool there = h_ahead < heads_ahead;
        L::copy(spot, there ? x_ahead : nullptr, ring + (2 * st) * L::kBytes);
        L::copy(spot, there ? dy_ahead : nullptr, ring + (2 * st + 1) * L::kBytes);
        copy_commit();
        x_ahead += a.x_head_stride;
        dy_ahead += a.dy_head_stride;
        if (++h_ahead == a.per) {
            h_ahead = 0;
            ahead += stride;
        }
    };
    if constexpr (kRing) {
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            copy_next(i);
    }
    int st = 0;
    // uniform over the block: all lanes stay for the sums
    for (int64_t base = (int64_t)blockIdx.x * side; base < items; base += stride) {
        const int64_t item = base + (threadIdx.x >> a.lanes_log2);
        const bool live = item < items;
        const Item it(a, live ? item : 0, groups, kind);
        const int heads = live ? it.heads : 0;
        const T *src = static_cast<const T *>(a.x) + it.t * a.x_row_stride + it.h0 * a.x_head_stride;
        const T *dsrc = static_cast<const T *>(a.dy) + it.t * a.dy_row_stride + it.h0 * a.dy_head_stride;
        T *dst = static_cast<T *>(a.out) + it.t * a.out_row_stride + it.h0 * a.out_head_stride;
        const int64_t pos = __ldg(a.positions + it.t);
        const bool bad = pos < 0 || pos >= a.max_position;
        if (live && bad && it.h0 == 0 && (threadIdx.x & (a.lanes - 1)) == 0 && a.err != nullptr)
            atomicAdd(a.err, 1);
        float c[kU][kP], s[kU][kP];
#pragma unroll
        for (int i = 0; i < kU; ++i)
            L::table(a, spot, pos, bad, i, c[i], s[i]);
        for (int h = 0; h < a.per; ++h) {
            typename L::Raw v, d;
            if constexpr (kRing) {
                copy_wait<kStages - 2>();
                L::copied(spot, h < heads, ring + (2 * st) * L::kBytes, v);
                L::copied(spot, h < heads, ring + (2 * st + 1) * L::kBytes, d);
            } else {
                L::load(spot, h < heads ? src + h * a.x_head_stride : nullptr, v);
                L::load(spot, h < heads ? dsrc + h * a.dy_head_stride : nullptr, d);
            }
            float p[kU][kP], q[kU][kP], g[kU][kP], k[kU][kP], squares[kP], dots[kP];   // x, the gradient of n w
#pragma unroll
            for (int j = 0; j < kP; ++j)
                squares[j] = dots[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                L::pairs(v[i], p[i], q[i]);
                float e[kP], f[kP];                       // dy, turned back
                L::pairs(d[i], e, f);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    g[i][j] = e[j];
                    k[i][j] = -e[j];
                }
                times(g[i], c[i]);
                if (spot.turned(a, i, bad)) {
                    add_product(g[i], f, s[i]);
                    times(k[i], s[i]);
                } else {
#pragma unroll
                    for (int j = 0; j < kP; ++j)
                        k[i][j] = 0.0f;
                }
                add_product(k[i], f, c[i]);
                add_product(squares, p[i], p[i]);
                add_product(squares, q[i], q[i]);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    e[j] = g[i][j];
                    f[j] = k[i][j];
                }
                times(e, wp[i]);
                times(f, wq[i]);
                add_product(dots, e, p[i]);
                add_product(dots, f, q[i]);
            }
            const float r = rsqrtf(__fmaf_rn(head_sum(sum_of(squares), a.lanes), a.inv_width, a.eps));
            const float along = -(head_sum(sum_of(dots), a.lanes) * r * a.inv_width);   // -mean(g w n)
            if constexpr (kRing) {
                copy_next((st + kStages - 1) % kStages);  // into the place of the head before, long read
                st = st + 1 == kStages ? 0 : st + 1;
            }
            if (h >= heads)                               // (then r may be infinite)
                continue;
            T *head = dst + h * a.out_head_stride;
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                scale(p[i], r);                           // n
                scale(q[i], r);
                add_product(dp[i], g[i], p[i]);
                add_product(dq[i], k[i], q[i]);
                times(g[i], wp[i]);
                times(k[i], wq[i]);
                float m[kP];
#pragma unroll
                for (int j = 0; j < kP; ++j)
                    m[j] = along;
                add_product(g[i], p[i], m);
                add_product(k[i], q[i], m);
                scale(g[i], r);
                scale(k[i], r);
                L::store(spot, head, i, g[i], k[i]);
            }
        }
    }
    if (!wanted)
        return;
    // over the heads of a warp, then over the warps
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
        const int at = spot.at[i], by = spot.by[i];
#pragma unroll
        for (int j = 0; j < kP; ++j) {
            float x = dp[i][j], y = dq[i][j];
            for (int o = 16; o >= a.lanes; o >>= 1) {
                x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
                y += __shfl_xor_sync(0xFFFFFFFFu, y, o);
            }
            if (at >= 0 && lane < a.lanes) {
                s_sum[warp][kHalves ? at + j : at + 2 * j] = x;
                if (!kHalves || by != 0)
                    s_sum[warp][kHalves ? at + by + j : at + 2 * j + 1] = y;
            }
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

// dw from the blocks' sums: a block has 32 columns, its warps take every 32nd part
// each, several at once, and are joined in order.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
k8_weight_grad(const __grid_constant__ NormArgs a)
{
    __shared__ float s_sum[kJoinWarps][32];
    pdl_trigger();
    pdl_wait();
    const int kind = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    if (a.dweight[kind] == nullptr)
        return;
    float x = 0.0f;
    // (no block of a kind without heads has left any)
    const int blocks = a.groups[kind] > 0 && a.T > 0 ? a.blocks : 0;
    const float *part = a.partial + (int64_t)kind * a.blocks * a.width + e;
    if (e < a.width) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += kJoinWarps)
            x += part[(int64_t)b * a.width];
    }
    s_sum[warp][lane] = x;
    __syncthreads();
    if (warp == 0 && e < a.width) {
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k)
            x += s_sum[k][lane];
        a.dweight[kind][e] = x;
    }
}

// Heads of an item: the most, up to `most`, with which hardly a place stays empty.
int heads_of_item(int q_heads, int k_heads, int most)
{
    const int heads = q_heads + k_heads;
    for (int per = most; per > 1; --per)
        if (((q_heads + per - 1) / per + (k_heads + per - 1) / per) * per - heads <= heads / 16)
            return per;
    return 1;
}

template <typename T, bool kHalves, int kVec, int kU, bool kRing>
cudaError_t launch_kind(const HeadNormLaunch &p, int units, int most, int num_sms, cudaStream_t stream)
{
    NormArgs a{};
    static_cast<HeadNormLaunch &>(a) = p;
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes * (kU == 2 ? 2 : 1) < units) {
        a.lanes *= 2;
        ++a.lanes_log2;
    }
    const int k_heads = p.heads - p.q_heads;
    a.per = kRing ? heads_of_item(p.q_heads, k_heads, most) : 1;
    a.groups[0] = (p.q_heads + a.per - 1) / a.per;
    a.groups[1] = (k_heads + a.per - 1) / a.per;
    a.inv_width = 1.0f / (float)p.width;
    constexpr size_t kSmem = kRing ? kStages * Lane<T, kHalves, kVec, kU>::kBytes : 0;
    static bool configured[2][64] = {};
    if (p.dy == nullptr) {
        const auto kernel = k8_head_norm<T, kHalves, kVec, kU, kRing>;
        const cudaError_t e = kRing ? allow_smem(kernel, kSmem, configured[0]) : cudaSuccess;
        if (e != cudaSuccess)
            return e;
        const int64_t threads = p.T * (a.groups[0] + a.groups[1]) * a.lanes;
        return launch_pdl(kernel, dim3((unsigned)((threads + kThreads - 1) / kThreads)), dim3(kThreads), kSmem, stream, 1, a);
    }
    const bool weights = a.dweight[0] != nullptr || a.dweight[1] != nullptr;
    const int side = kThreads / a.lanes;
    const int64_t items = p.T * std::max(a.groups[0], a.groups[1]);
    a.blocks = (int)std::max<int64_t>(1, std::min<int64_t>((items + side - 1) / side, (int64_t)num_sms * kGradPerSm<T, kHalves, kU>));
    cudaError_t e = cudaSuccess;
    if (p.T > 0) {
        const auto kernel = k8_head_norm_grad<T, kHalves, kVec, kU, kRing>;
        e = kRing ? allow_smem(kernel, 2 * kSmem, configured[1]) : cudaSuccess;
        if (e == cudaSuccess)
            e = launch_pdl(kernel, dim3((unsigned)a.blocks, 2), dim3(kThreads), 2 * kSmem, stream, 1, a);
    }
    if (e == cudaSuccess && weights)
        e = launch_pdl(k8_weight_grad, dim3((unsigned)((p.width + 31) / 32), 2), dim3(32 * kJoinWarps), 0, stream, 1, a);
    return e;
}

template <typename T, bool kHalves>
cudaError_t launch_type(const HeadNormLaunch &a, bool wide, int num_sms, cudaStream_t stream)
{
    constexpr int kWide = 16 / (int)sizeof(T), kNarrow = kHalves ? 1 : 2;
    const int vec = wide ? kWide : kNarrow;
    const int units = kHalves ? a.rot / (2 * vec) + ((a.width - a.rot) / vec + 1) / 2 : a.width / vec;
    // Several heads an item, whose table columns and weights are read once, where
    // there is work to fill the GPU that way.
    const int64_t threads = a.T * a.heads * units;
    const int most = (int)std::min<int64_t>(8, std::max<int64_t>(1, threads / ((int64_t)num_sms * 2048)));
    if (!wide)                              // up to 256 units of two elements
        return launch_kind<T, kHalves, kNarrow, 8, false>(a, units, 1, num_sms, stream);
    if constexpr (!kHalves)
        if (units > 64)                     // up to 128
            return launch_kind<T, kHalves, kWide, 4, false>(a, units, 1, num_sms, stream);
    if (units > 32 || (most > 1 && !kHalves && a.dy != nullptr && units > 1))    // (the gradient in pairs: two units a lane)
        return most > 1 ? launch_kind<T, kHalves, kWide, 2, true>(a, units, most, num_sms, stream)
                        : launch_kind<T, kHalves, kWide, 2, false>(a, units, 1, num_sms, stream);
    return most > 1 ? launch_kind<T, kHalves, kWide, 1, true>(a, units, most, num_sms, stream)
                    : launch_kind<T, kHalves, kWide, 1, false>(a, units, 1, num_sms, stream);
}

}  // namespace

size_t head_norm_grad_workspace(int32_t width, int num_sms)
{
    return (size_t)2 * num_sms * kMaxGradPerSm * width * sizeof(float);
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
