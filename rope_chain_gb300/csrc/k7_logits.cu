// K7: logits adjustment -- penalties for repeated tokens, biases and grammar
// masks on the logits of every drafted token.
//
// Row r of sequence b, token t, with g = how often t was generated (the
// history past the prompt, and the drafted tokens that the row's node sees,
// itself among them) and `seen` = g > 0 or t is in the prompt:
//   x = logit;  x = seen ? (x > 0 ? x / rep : x * rep) : x
//   x = x - freq * g - (g > 0 ? pres : 0);  x = x + bias;  disallowed -> -inf
// in FP32 in this order, rounded once to the logits' type.
//
// The floor is one read and one write of the logits.  A CTA owns a tile of
// the vocabulary for the rows of one sequence: it scans the history once,
// counts the tile's tokens in shared memory, lists those that need arithmetic
// and then streams its columns of every row, 16 bytes at a time.  Few tokens
// are listed (what the history, the tree and the biases name), but they lie
// scattered, so that computing them in place would make nearly every warp
// walk the whole formula for a lane or two.  Instead the listed tokens of the
// next row are computed side by side, one per thread, into shared memory while
// the current row streams, and the stream only picks their values up where a
// bit map says so.
#include "rc_internal.cuh"

#include <algorithm>

namespace rc {

namespace {

constexpr int kThreads = 256;
constexpr int kPad = 32;                     // tokens kept before a tile (rows may start unaligned)
constexpr int kNodes = 512;                  // drafted tokens a tile lists
constexpr uint32_t kPrompt = 1u << 31;       // count word: in the prompt
constexpr uint32_t kDraft = 1u << 30;        //   drafted in the tree: the count changes by row
constexpr uint32_t kBias = 1u << 29;         //   has a bias
constexpr uint32_t kCount = kBias - 1;       //   occurrences in the generated history

template <typename T> struct Io;
template <> struct Io<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float load(float v) { return v; }
    static __device__ __forceinline__ float store(float v) { return v; }
};
template <> struct Io<uint16_t> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float load(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
    static __device__ __forceinline__ uint16_t store(float v) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
};

template <typename T> __device__ __forceinline__ T minus_inf();
template <> __device__ __forceinline__ float minus_inf<float>() { return __int_as_float((int)0xFF800000); }
template <> __device__ __forceinline__ uint16_t minus_inf<uint16_t>() { return 0xFF80u; }

// 32 bits of a bit map (words 32 bits wide) from bit `at` on.
__device__ __forceinline__ uint32_t window(const uint32_t *words, int at) {
    return __funnelshift_r(words[at >> 5], words[(at >> 5) + 1], at & 31);
}

template <int kTile> struct Smem {
    static constexpr int kWords = kTile + kPad;
    uint32_t word[kWords];                           // count and flags of a token
    uint32_t bias[kWords];                           // 1 + the entry of its bias, then the bias itself
    float value[2][kWords];                          // a row's adjusted logits of the listed tokens
    uint32_t special[kWords / 32 + 2];               // bit: word != 0
    uint16_t list[kWords];                           // the tokens with word != 0
    int32_t node[kNodes];                            // the tile's drafted tokens: node index,
    int32_t token[kNodes];                           //   and place in the tile
    int32_t nodes, listed;
};

// kAligned: `logits` and `out` rows start at the same offset from a 16-byte
// boundary, so both move 16 bytes at a time; else element by element.
template <typename T, int kTile, bool kAligned>
__global__ void __launch_bounds__(kThreads)
k7_logits(const __grid_constant__ LogitsLaunch a)
{
    constexpr int kVec = kAligned ? Io<T>::kVec : 1;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<kTile> &s = *reinterpret_cast<Smem<kTile> *>(smem_raw);
    pdl_trigger();
    for (int i = threadIdx.x; i < kTile + kPad; i += kThreads) {
        s.word[i] = 0u;
        s.bias[i] = 0u;
    }
    if (threadIdx.x == 0)
        s.nodes = s.listed = 0;
    __syncthreads();
    pdl_wait();

    const int b = blockIdx.y;
    const int first = blockIdx.x * kTile;            // the tile: tokens first - kPad + 1 on
    const int base = first - kPad;
    const int r0 = (int)max((int64_t)0, min((int64_t)a.row_start[b], a.rows));
    const int r1 = (int)max((int64_t)r0, min((int64_t)a.row_start[b + 1], a.rows));
    if (r0 + (int)blockIdx.z >= r1)
        return;
    // counted by one CTA of the sequence
    const bool teller = blockIdx.x == 0 && blockIdx.z == 0 && a.err != nullptr;
    int bad = 0;

    // Each row: its vectors and their mask bits are loaded while the row
    // before it is worked on (the first while the history is counted).
    struct alignas(kAligned ? 16 : sizeof(T)) Vec { T v[kVec]; };
    constexpr int kPer = (kTile / kVec + kThreads - 1) / kThreads;
    const int words = (a.V + 31) / 32;
    auto shift_of = [&](int row) {
        // vectors start on 16-byte boundaries: `shift` tokens before the tile
        return kAligned ? (int)((reinterpret_cast<uintptr_t>(static_cast<const T *>(a.logits) +
                                                             (int64_t)row * a.row_stride) & 15u) / sizeof(T)) : 0;
    };
    auto load = [&](int row, Vec (&v)[kPer], uint32_t (&ok)[kPer]) {
        const T *src = static_cast<const T *>(a.logits) + (int64_t)row * a.row_stride;
        const uint32_t *mask = a.allowed != nullptr ? a.allowed + (int64_t)row * a.allowed_stride : nullptr;
        const int shift = shift_of(row);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = (threadIdx.x + k * kThreads) * kVec, t = first - shift + i;
            ok[k] = 0xFFFFFFFFu;
            if (i >= kTile || t >= a.V)
                continue;
            if (t >= 0 && t + kVec <= a.V) {
                v[k] = *reinterpret_cast<const Vec *>(src + t);
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    v[k].v[j] = t + j >= 0 && t + j < a.V ? src[t + j] : T(0);
            }
            if (mask != nullptr) {
                // the mask words around t; before token 0 and past the last word: not used
                const int w0 = t >> 5;
                const uint32_t lo = w0 >= 0 ? __ldg(mask + w0) : 0u;
                const uint32_t hi = (t & 31) + kVec > 32 && w0 + 1 < words ? __ldg(mask + w0 + 1) : 0u;
                ok[k] = __funnelshift_r(lo, hi, t & 31);
            }
        }
    };
    Vec next[kPer];
    uint32_t next_ok[kPer];
    int row = r0 + (int)blockIdx.z;
    load(row, next, next_ok);

    // The history's tokens of this tile.
    if (a.history != nullptr) {
        const int64_t h0 = max((int64_t)0, min(a.history_start[b], a.history_size));
        const int64_t h1 = max(h0, min(a.history_start[b + 1], a.history_size));
        const int64_t made = h0 + (a.prompt_len != nullptr ? max(a.prompt_len[b], 0) : 0);
        for (int64_t i0 = h0 + threadIdx.x; i0 < h1; i0 += 8 * kThreads) {
            int32_t t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                t[j] = i0 + j * kThreads < h1 ? __ldg(a.history + i0 + j * kThreads) : 0x7FFFFFFF;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t i = i0 + j * kThreads;
                if (i >= h1)
                    break;
                bad += t[j] < 0 || t[j] >= a.V;
                const uint32_t at = (uint32_t)t[j] - (uint32_t)base;
                if (t[j] >= 0 && t[j] < a.V && at < (uint32_t)(kTile + kPad)) {
                    if (i < made)
                        atomicOr(&s.word[at], kPrompt);
                    else
                        atomicAdd(&s.word[at], 1u);
                }
            }
        }
    }
    __syncthreads();
    // The biases: a token listed twice takes its last entry.
    if (a.bias_start != nullptr) {
        const int64_t e0 = max((int64_t)0, min((int64_t)a.bias_start[b], a.bias_size));
        const int64_t e1 = max(e0, min((int64_t)a.bias_start[b + 1], a.bias_size));
        for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) {
            const int32_t t = __ldg(a.bias_tokens + e);
            bad += t < 0 || t >= a.V;
            const uint32_t at = (uint32_t)t - (uint32_t)base;
            if (t >= 0 && t < a.V && at < (uint32_t)(kTile + kPad)) {
                atomicOr(&s.word[at], kBias);
                atomicMax(&s.bias[at], (uint32_t)(e + 1));
            }
        }
    }
    // The tokens drafted in this tree.
    if (a.draft_tokens != nullptr) {
        for (int r = r0 + threadIdx.x; r < r1; r += kThreads) {
            const int32_t t = __ldg(a.draft_tokens + r);
            bad += t < 0 || t >= a.V;
            const uint32_t at = (uint32_t)t - (uint32_t)base;
            if (t >= 0 && t < a.V && at < (uint32_t)(kTile + kPad)) {
                atomicOr(&s.word[at], kDraft);
                const int k = atomicAdd(&s.nodes, 1);
                if (k < kNodes) {
                    s.node[k] = r - r0;
                    s.token[k] = (int32_t)at;
                }
            }
        }
    }
    if (teller && bad)
        atomicAdd(a.err, bad);
    __syncthreads();
    for (int i = threadIdx.x; i < kTile + kPad + 64; i += kThreads) {     // a whole number of warps
        const uint32_t w = i < kTile + kPad ? s.word[i] : 0u;
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, w != 0u);
        const int lane = threadIdx.x & 31;
        int at = 0;
        if (lane == 0) {
            s.special[i >> 5] = bits;
            at = bits != 0u ? atomicAdd(&s.listed, __popc(bits)) : 0;
        }
        at = __shfl_sync(0xFFFFFFFFu, at, 0) + __popc(bits & ((1u << lane) - 1u));
        if (w != 0u)
            s.list[at] = (uint16_t)i;
        if (w & kBias)
            s.bias[i] = __float_as_uint(__ldg(a.bias_values + (s.bias[i] - 1u)));
    }
    __syncthreads();

    const float rep = a.repetition != nullptr ? a.repetition[b] : 1.0f;
    const float freq = a.frequency != nullptr ? a.frequency[b] : 0.0f;
    const float pres = a.presence != nullptr ? a.presence[b] : 0.0f;
    const int listed = s.listed, nodes = s.nodes;

    // The logits of row `row`'s listed tokens: thread i takes entries i, i +
    // kThreads, ...; the first kAhead of them are loaded before they are due.
    constexpr int kAhead = 2;
    auto fetch = [&](int row, float (&x)[kAhead]) {
        const T *src = static_cast<const T *>(a.logits) + (int64_t)row * a.row_stride;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int e = threadIdx.x + k * kThreads;
            const int t = e < listed ? base + s.list[e] : -1;
            x[k] = t >= 0 && t < a.V ? Io<T>::load(src[t]) : 0.0f;
        }
    };
    auto adjust = [&](int row, const float (&ahead)[kAhead], float *value) {
        const T *src = static_cast<const T *>(a.logits) + (int64_t)row * a.row_stride;
        const uint64_t *see = a.tree_mask != nullptr ? a.tree_mask + (int64_t)row * a.mask_words : nullptr;
        auto sees = [&](int j) {
            if (see == nullptr)
                return j <= row - r0;
            return (j >> 6) < a.mask_words && ((__ldg(see + (j >> 6)) >> (j & 63)) & 1u) != 0u;
        };
        auto one = [&](int e, float x) {
            const int at = s.list[e];
            const uint32_t w = s.word[at];
            uint32_t g = w & kCount;
            if (w & kDraft) {
                if (nodes <= kNodes) {
                    for (int k = 0; k < nodes; ++k)
                        g += s.token[k] == at && sees(s.node[k]);
                } else {
                    for (int j = 0; j < r1 - r0; ++j)
                        g += __ldg(a.draft_tokens + r0 + j) == at + base && sees(j);
                }
            }
            if (g != 0u || (w & kPrompt) != 0u)
                x = x > 0.0f ? __fdiv_rn(x, rep) : __fmul_rn(x, rep);
            x = __fsub_rn(x, __fmul_rn(freq, (float)g));
            if (g != 0u)
                x = __fsub_rn(x, pres);
            if (w & kBias)
                x = __fadd_rn(x, __uint_as_float(s.bias[at]));
            value[at] = x;
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (threadIdx.x + k * kThreads < listed)
                one(threadIdx.x + k * kThreads, ahead[k]);
        for (int e = threadIdx.x + kAhead * kThreads; e < listed; e += kThreads)
            one(e, Io<T>::load(src[base + s.list[e]]));
    };
    float ahead[kAhead];
    fetch(row, ahead);
    adjust(row, ahead, s.value[0]);
    int turn = 0;
    for (; row < r1; row += (int)gridDim.z) {
        __syncthreads();                                 // this row's values are there, the last row's are free
        Vec v[kPer];
        uint32_t ok[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            v[k] = next[k];
            ok[k] = next_ok[k];
        }
        const bool more = row + (int)gridDim.z < r1;
        if (more) {
            load(row + (int)gridDim.z, next, next_ok);
            fetch(row + (int)gridDim.z, ahead);
        }
        const float *value = s.value[turn];
        T *dst = static_cast<T *>(a.out) + (int64_t)row * a.out_row_stride;
        const int shift = shift_of(row);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = (threadIdx.x + k * kThreads) * kVec;
            const int t = first - shift + i;
            if (i >= kTile || t >= a.V)
                continue;
            const int at = t - base;
            const uint32_t todo = window(s.special, at) & ((1u << kVec) - 1u);
            if (todo != 0u) {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if ((todo >> j) & 1u)
                        v[k].v[j] = Io<T>::store(value[at + j]);
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (!((ok[k] >> j) & 1u))
                    v[k].v[j] = minus_inf<T>();
            if (t >= 0 && t + kVec <= a.V) {
                *reinterpret_cast<Vec *>(dst + t) = v[k];
            } else {
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    if (t + j >= 0 && t + j < a.V)
                        dst[t + j] = v[k].v[j];
            }
        }
        turn ^= 1;
        if (more)
            adjust(row + (int)gridDim.z, ahead, s.value[turn]);
    }
}

template <typename T, int kTile, bool kAligned>
cudaError_t launch_one(const LogitsLaunch &a, int num_sms, cudaStream_t stream)
{
    const size_t smem = sizeof(Smem<kTile>);
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    auto kernel = k7_logits<T, kTile, kAligned>;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            configured[dev] = true;
    }
    // a row's vectors start up to kVec - 1 tokens before its first token
    const int64_t tiles = ((int64_t)a.V + (kAligned ? Io<T>::kVec - 1 : 0) + kTile - 1) / kTile;
    // a sequence's rows are shared out to as many CTAs as fill the GPU
    const int64_t rows = std::max<int64_t>(1, a.rows / a.seqs);
    const int64_t chunks = std::min<int64_t>(rows, std::max<int64_t>(1, 4LL * num_sms / (tiles * a.seqs)));
    return launch_pdl(kernel, dim3((unsigned)tiles, (unsigned)a.seqs, (unsigned)chunks), dim3(kThreads),
                      smem, stream, 1, a);
}

template <typename T>
cudaError_t launch_type(const LogitsLaunch &a, int num_sms, cudaStream_t stream)
{
    const uintptr_t src = reinterpret_cast<uintptr_t>(a.logits), dst = reinterpret_cast<uintptr_t>(a.out);
    const bool aligned = (src & 15u) == (dst & 15u) &&
                         (a.rows <= 1 || ((a.row_stride - a.out_row_stride) * (int64_t)sizeof(T)) % 16 == 0);
    if ((int64_t)((a.V + 2047) / 2048) * a.seqs >= 2 * num_sms)
        return aligned ? launch_one<T, 2048, true>(a, num_sms, stream)
                       : launch_one<T, 2048, false>(a, num_sms, stream);
    return aligned ? launch_one<T, 1024, true>(a, num_sms, stream)
                   : launch_one<T, 1024, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_logits_adjust(const LogitsLaunch &a, bool f32, int num_sms, cudaStream_t stream)
{
    return f32 ? launch_type<float>(a, num_sms, stream) : launch_type<uint16_t>(a, num_sms, stream);
}

}  // namespace rc
