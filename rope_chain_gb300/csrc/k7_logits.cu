// K7: logits adjustment -- penalties for repeated tokens, biases and grammar
// masks on the logits of every drafted token.
//
// Row r of sequence b, token t, with g = how often t was generated (the
// history past the prompt, and the drafted tokens that the row's node sees,
// itself among them) and `seen` = g > 0 or t is in the prompt:
//   x = logit;  x = seen ? (x > 0 ? x / rep : x * rep) : x
//   x = g > 0 ? x - freq * g - pres : x;  x = x + bias;  disallowed -> -inf
// in FP32 in this order (x / rep as x times the rounded 1 / rep, freq * g fused
// into its difference), rounded once to the logits' type.
//
// The floor is one read and one write of the logits.  A CTA owns a tile of
// the vocabulary for the rows of one sequence: it scans the history once,
// counts the tile's tokens in shared memory, and then streams its columns of
// every row, 16 bytes at a time, each warp by itself.  Few tokens need
// arithmetic (what the history, the tree and the biases name).  Each warp lists
// those of its columns once; with every row its logits go through shared memory,
// where the lanes take the listed ones 32 at a time.  (Lanes that walked what
// was listed in their own 16 bytes were bound by instructions, as long as the
// fullest of 32: 16 x 64 rows of 131072, history 4096, 221 us FP32 and 178 bf16;
// now 192 to 195, 5.6 TB/s, bound by memory, and 125 to 128, 4.3 TB/s.)  The nodes that draft
// a token of the tile are a 64-bit set, so that a row's count of it is a
// population count.  Trees of more than 64 nodes are walked node by node instead,
// for each listed token of each row: 4 x 64 rows of 131072 73 us, 4 x 65 1390.
// Small calls are latency: one row of 32000 takes 4.0 us, 39 rows of 100003 bf16
// with skewed histories of 9001 15.8 us, of which the tile with the most frequent
// tokens makes 5 and the scan of the history 2.
#include "rc_draft.cuh"

#include <algorithm>
#include <type_traits>

namespace rc {

namespace {

constexpr int kThreads = 256;
constexpr int kPad = 32;                     // tokens kept before a tile (rows may start unaligned)
constexpr int kNodes = 64;                   // nodes of a tree whose drafted tokens a tile lists
constexpr uint32_t kPrompt = 1u << 31;       // count word: in the prompt
constexpr uint32_t kDraft = 1u << 30;        //   drafted in the tree: the count differs by row
constexpr uint32_t kBias = 1u << 29;         //   has a bias
constexpr uint32_t kCount = kBias - 1;       //   occurrences in the generated history

// kVec logits of one access as 32-bit words: FP32 values, or bf16 in pairs (a
// single one alone).
template <typename T, int kVec> struct Vec;
template <int kVec> struct alignas(kVec > 1 ? 16 : 4) Vec<float, kVec> {
    float w[kVec];
    __device__ __forceinline__ void load(const float *p) { *this = *reinterpret_cast<const Vec *>(p); }
    __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<Vec *>(p) = *this; }
    __device__ __forceinline__ float get(int j) const {
        float x = w[0];
#pragma unroll
        for (int i = 1; i < kVec; ++i)
            x = i == j ? w[i] : x;
        return x;
    }
    __device__ __forceinline__ void set(int j, float x) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            w[i] = i == j ? x : w[i];
    }
    // -inf where a token's bit of `ok` is not set
    __device__ __forceinline__ void mask(uint32_t ok) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            w[i] = (ok >> i) & 1u ? w[i] : __int_as_float((int)0xFF800000);
    }
};
template <> struct alignas(16) Vec<uint16_t, 8> {
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint16_t *p) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
    __device__ __forceinline__ void store(uint16_t *p) const {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ float get(int j) const {
        const uint32_t lo = j & 2 ? w[1] : w[0], hi = j & 2 ? w[3] : w[2], x = j & 4 ? hi : lo;
        return __uint_as_float(j & 1 ? x & 0xFFFF0000u : x << 16);
    }
    __device__ __forceinline__ void set(int j, float x) {
        const uint32_t v = __bfloat16_as_ushort(__float2bfloat16_rn(x));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t with = j & 1 ? (w[i] & 0xFFFFu) | (v << 16) : (w[i] & 0xFFFF0000u) | v;
            w[i] = i == j >> 1 ? with : w[i];
        }
    }
    __device__ __forceinline__ void mask(uint32_t ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t two = (ok >> (2 * i)) & 3u;       // bits 0 and 1 to halves 0 and 1
            const uint32_t keep = ((two | (two << 15)) & 0x00010001u) * 0xFFFFu;
            w[i] = (w[i] & keep) | (0xFF80FF80u & ~keep);
        }
    }
};
template <> struct Vec<uint16_t, 1> {
    uint32_t w;
    __device__ __forceinline__ void load(const uint16_t *p) { w = *p; }
    __device__ __forceinline__ void store(uint16_t *p) const { *p = (uint16_t)w; }
    __device__ __forceinline__ float get(int) const { return __uint_as_float(w << 16); }
    __device__ __forceinline__ void set(int, float x) { w = __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
    __device__ __forceinline__ void mask(uint32_t ok) { w = ok & 1u ? w : 0xFF80u; }
};

// 32 bits of a bit map (words 32 bits wide) from bit `at` on.
__device__ __forceinline__ uint32_t window(const uint32_t *words, int at) {
    return __funnelshift_r(words[at >> 5], words[(at >> 5) + 1], at & 31);
}

template <typename T, int kTile, int kVec, int kR, bool kSame> struct Smem {
    static constexpr int kWords = kTile + kPad, kWarps = kThreads / 32;
    static constexpr int kWindow = 32 * kVec;        // tokens of a warp's access
    T stage[kWarps][kR][kWindow];                    // a warp's logits while its listed ones are worked on
    uint64_t set[kNodes];                            // the nodes that draft a listed token
    uint32_t word[kWords];                           // count and flags of a token
    uint32_t bias[kWords];                           // 1 + the entry of its bias, then the bias itself
    uint32_t special[kWords / 32 + 2];               // bit: word != 0
    uint16_t listed[kWords];                         // where the drafted token's set is
    int16_t node[kNodes], token[kNodes];             // a listed node, and its token's place in the tile
    int32_t nodes;
    // per access of a warp, the places of what is listed (kSame: within the 256
    // tokens at most; else of the rows' windows together)
    using Place = typename std::conditional<kSame, uint8_t, uint16_t>::type;
    Place order[kWarps][kTile / (kVec * kThreads)][kWindow + (kSame ? 0 : kVec - 1)];
};

// The history, four tokens a load where it is aligned: f(token, whether it is
// one of the first `made`).  A thread's first kLoads accesses and the unaligned
// ends are on their way before any of it is looked at (prompt and generated part
// one after the other, ends apart: 32000 logits with 600 tokens of history
// 4.5 us instead of 3.8).
template <typename F>
__device__ __forceinline__ void each_token(const int32_t *p, int n, int made, F f) {
    const int me = (int)threadIdx.x;
    const int lead = min(n, (int)((16u - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / 4);
    const int quads = (n - lead) / 4, rest = n - lead - 4 * quads;
    const int4 *q = reinterpret_cast<const int4 *>(p + lead);
    constexpr int kLoads = 5;
    // the ends: up to three tokens each, by threads 0 .. 2 and 4 .. 6
    const int end = me < 4 ? me : n - rest + me - 4;
    const bool has = me < 4 ? me < lead : me - 4 < rest;
    const int32_t lone = has ? __ldg(p + end) : 0;
    for (int i = me; i < quads; i += kLoads * kThreads) {
        int4 t[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (i + j * kThreads < quads)
                t[j] = __ldg(q + i + j * kThreads);
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (i + j * kThreads < quads) {
                const int at = lead + 4 * (i + j * kThreads);
                f(t[j].x, at < made);
                f(t[j].y, at + 1 < made);
                f(t[j].z, at + 2 < made);
                f(t[j].w, at + 3 < made);
            }
    }
    if (has)
        f(lone, end < made);
}

// Rows move 16 bytes at a time where `logits` and `out` rows start at the same
// offset from a 16-byte boundary (kVec > 1): a thread's vectors then start up
// to kVec - 1 tokens (`shift`) before its place in the tile.  kSame: every row
// has the same shift, so that where a thread's tokens lie, and which of them
// are listed, is found once.  kR rows are in flight per thread.  bf16 vectors
// want 80 registers, three blocks on an SM (16 x 64 rows of 131072 125 us, with
// four blocks 172); FP32 fits the 64 of four.
template <typename T, int kTile, int kVec, int kR, bool kSame>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && kVec > 1 ? 3 : 4)
k7_logits(const __grid_constant__ LogitsLaunch a)
{
    constexpr int kPer = kTile / (kVec * kThreads);
    using V = Vec<T, kVec>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    using S = Smem<T, kTile, kVec, kR, kSame>;
    S &s = *reinterpret_cast<S *>(smem_raw);
    pdl_trigger();
    for (int i = threadIdx.x; i < kTile + kPad; i += kThreads) {
        s.word[i] = 0u;
        s.bias[i] = 0u;
    }
    if (threadIdx.x < kNodes)
        s.set[threadIdx.x] = 0u;
    if (threadIdx.x == 0)
        s.nodes = 0;
    __syncthreads();
    pdl_wait();

    // (the sequence's scalars first: one latency for all of them)
    const int b = blockIdx.y;
    const int64_t start0 = a.row_start[b], start1 = a.row_start[b + 1];
    const int64_t hist0 = a.history != nullptr ? a.history_start[b] : 0;
    const int64_t hist1 = a.history != nullptr ? a.history_start[b + 1] : 0;
    const int32_t prompt = a.prompt_len != nullptr ? a.prompt_len[b] : 0;
    const int32_t bias0 = a.bias_start != nullptr ? a.bias_start[b] : 0;
    const int32_t bias1 = a.bias_start != nullptr ? a.bias_start[b + 1] : 0;
    const float rep = a.repetition != nullptr ? a.repetition[b] : 1.0f;
    const float freq = a.frequency != nullptr ? a.frequency[b] : 0.0f;
    const float pres = a.presence != nullptr ? a.presence[b] : 0.0f;
    const int first = blockIdx.x * kTile;            // the tile: tokens first - kVec + 1 on
    const int base = first - kPad;
    const int r0 = (int)max((int64_t)0, min(start0, a.rows));
    const int r1 = (int)max((int64_t)r0, min(start1, a.rows));
    const int step = (int)gridDim.z;                 // this CTA's rows: r0 + blockIdx.z, + step, ...
    if (r0 + (int)blockIdx.z >= r1)
        return;

    // A thread's vector k of a row: its first token, whether all of it is in
    // the vocabulary, whether any is, and the shift of its bits in a mask word.
    const int words = (a.V + 31) / 32;
    auto shift_of = [&](int row) {
        return kVec > 1 ? (int)((reinterpret_cast<uintptr_t>(static_cast<const T *>(a.logits) +
                                                             (int64_t)row * a.row_stride) & 15u) / sizeof(T)) : 0;
    };
    const int shift0 = shift_of(r0 + (int)blockIdx.z);
    auto token = [&](int row, int k) {
        return first - (kSame ? shift0 : shift_of(row)) + ((int)threadIdx.x + k * kThreads) * kVec;
    };
    // The rows of a turn: their vectors and mask words are loaded while those of
    // the turn before are worked on (the first while the history is counted).
    // Nothing here looks at what it loads: a thread that did would wait for
    // each load in turn (measured: 6000 cycles a turn instead of 1000).
    struct Words { uint32_t lo, hi; };               // around a vector's first token
    auto load = [&](int row, V (&v)[kPer], Words (&ok)[kPer], uint64_t &see) {
        see = a.tree_mask != nullptr ? __ldg(a.tree_mask + (int64_t)row * a.mask_words) : 0u;
        const T *src = static_cast<const T *>(a.logits) + (int64_t)row * a.row_stride;
        const uint32_t *mask = a.allowed != nullptr ? a.allowed + (int64_t)row * a.allowed_stride : nullptr;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int t = token(row, k);
            ok[k].lo = ok[k].hi = 0xFFFFFFFFu;
            if (t + kVec <= 0 || t >= a.V)
                continue;
            if (t >= 0 && t + kVec <= a.V) {
                v[k].load(src + t);
            } else {
                // an end of the row
                for (int j = 0; j < kVec; ++j)
                    if (t + j >= 0 && t + j < a.V) {
                        Vec<T, 1> one;
                        one.load(src + t + j);
                        v[k].set(j, one.get(0));
                    }
            }
            if (mask != nullptr) {
                const int w = t >> 5;                // (the word before token 0's is not there)
                if (w >= 0)
                    ok[k].lo = __ldg(mask + w);
                if (kVec > 1 && (t & 31) + kVec > 32 && w + 1 < words)      // (only with a shift)
                    ok[k].hi = __ldg(mask + w + 1);
            }
        }
    };
    V next[kR][kPer];
    Words next_ok[kR][kPer];
    uint64_t next_see[kR];
    int row = r0 + (int)blockIdx.z;
#pragma unroll
    for (int q = 0; q < kR; ++q)
        if (row + q * step < r1)
            load(row + q * step, next[q], next_ok[q], next_see[q]);

    // (so are this thread's first bias and drafted token)
    const int64_t e0 = max((int64_t)0, min((int64_t)bias0, a.bias_size));
    const int64_t e1 = max(e0, min((int64_t)bias1, a.bias_size));
    const int32_t bias_token = e0 + threadIdx.x < e1 ? __ldg(a.bias_tokens + e0 + threadIdx.x) : 0;
    const int32_t draft_token = a.draft_tokens != nullptr && r0 + (int)threadIdx.x < r1
                                    ? __ldg(a.draft_tokens + r0 + threadIdx.x) : 0;

    // The history's tokens of this tile (what lies outside the vocabulary may
    // land beside it, where nothing is read): the prompt's marked, the generated
    // ones counted.
    const bool teller = blockIdx.x == 0 && blockIdx.z == 0 && a.err != nullptr;
    int bad = 0;                                     // counted by one CTA of the sequence
    if (a.history != nullptr) {
        const int64_t h0 = max((int64_t)0, min(hist0, a.history_size));
        const int64_t h1 = max(h0, min(hist1, a.history_size));
        each_token(a.history + h0, (int)(h1 - h0), max(prompt, 0), [&](int32_t t, bool prompted) {
            const uint32_t at = (uint32_t)t - (uint32_t)base;
            if (at < (uint32_t)(kTile + kPad)) {
                if (prompted)
                    atomicOr(&s.word[at], kPrompt);
                else
                    atomicAdd(&s.word[at], 1u);
            }
            bad += teller && (t < 0 || t >= a.V);
        });
    }
    // The biases: a token listed twice takes its last entry.
    if (a.bias_start != nullptr) {
        for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) {
            const int32_t t = e < e0 + kThreads ? bias_token : __ldg(a.bias_tokens + e);
            bad += teller && (t < 0 || t >= a.V);
            const uint32_t at = (uint32_t)t - (uint32_t)base;
            if (at < (uint32_t)(kTile + kPad)) {
                atomicOr(&s.word[at], kBias);
                atomicMax(&s.bias[at], (uint32_t)(e + 1));
            }
        }
    }
    // The tokens drafted in this tree.
    if (a.draft_tokens != nullptr) {
        for (int r = r0 + threadIdx.x; r < r1; r += kThreads) {
            const int32_t t = r < r0 + kThreads ? draft_token : __ldg(a.draft_tokens + r);
            bad += teller && (t < 0 || t >= a.V);
            const uint32_t at = (uint32_t)t - (uint32_t)base;
            if (at < (uint32_t)(kTile + kPad)) {
                atomicOr(&s.word[at], kDraft);
                const int k = atomicAdd(&s.nodes, 1);
                if (k < kNodes && r - r0 < kNodes) {
                    s.node[k] = (int16_t)(r - r0);
                    s.token[k] = (int16_t)at;
                    s.listed[at] = (uint16_t)k;          // any one of a token's entries
                }
            }
        }
    }
    if (bad)
        atomicAdd(a.err, bad);
    __syncthreads();
    // Trees of more nodes than are listed are walked node by node for each of their
    // tokens.
    const bool few = r1 - r0 <= kNodes;
    if (few && (int)threadIdx.x < s.nodes)
        atomicOr(reinterpret_cast<unsigned long long *>(&s.set[s.listed[s.token[threadIdx.x]]]),
                 1ull << s.node[threadIdx.x]);
    {
        constexpr int kGroups = (kTile + kPad + 64) / 32, kTurns = (kGroups + kThreads / 32 - 1) / (kThreads / 32);
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
        for (int g = 0; g < kTurns; ++g) {
            const int at = warp + g * (kThreads / 32), i = at * 32 + lane;
            const uint32_t w = i < kTile + kPad ? s.word[i] : 0u;
            const uint32_t bits = __ballot_sync(0xFFFFFFFFu, w != 0u);
            if (lane == 0 && at < kGroups)
                s.special[at] = bits;
            if (w & kBias)
                s.bias[i] = __float_as_uint(__ldg(a.bias_values + (s.bias[i] - 1u)));
        }
    }
    __syncthreads();

    // What is listed among the tokens that this warp's access k reaches, in
    // order, as places from start_of(k) on.
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto start_of = [&](int k) {
        return first - (kSame ? shift0 : kVec - 1) + (warp * 32 + k * kThreads) * kVec - base;
    };
    int listed[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int from = start_of(k) + lane * kVec, own = kSame || lane < 31 ? kVec : 2 * kVec - 1;
        uint32_t bits = window(s.special, from) & ((1u << own) - 1u);
        int at = __popc(bits);
        const int mine = at;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int other = __shfl_up_sync(0xFFFFFFFFu, at, d);
            at += lane >= d ? other : 0;
        }
        listed[k] = __shfl_sync(0xFFFFFFFFu, at, 31);
        for (at -= mine; bits != 0u; bits &= bits - 1u)
            s.order[warp][k][at++] = (typename S::Place)(lane * kVec + __ffs(bits) - 1);
    }
    __syncwarp();

    // The quotient as a product: at most 1.5 ulp, where the division has half a one.
    // 16 x 64 rows of 131072: 193 us; with the product corrected by its remainder
    // 203, with the division 210.
    const float less = __fdiv_rn(1.0f, rep);
    // The logit of a token whose word w is set, in row r, whose node sees `see`
    // (its first 64 nodes).
    auto adjusted = [&](int r, uint64_t see, int at, uint32_t w, float x) {
        uint32_t g = w & kCount;
        if (w & kDraft) {
            if (few) {
                g += __popcll(see & s.set[s.listed[at]]);
            } else {
                const uint64_t *all = a.tree_mask != nullptr ? a.tree_mask + (int64_t)r * a.mask_words : nullptr;
                for (int j = 0; j < r1 - r0; ++j) {
                    const bool sees = all == nullptr ? j <= r - r0
                                                     : (j >> 6) < a.mask_words && ((__ldg(all + (j >> 6)) >> (j & 63)) & 1u);
                    g += sees && __ldg(a.draft_tokens + r0 + j) == at + base;
                }
            }
        }
        if (g != 0u || (w & kPrompt) != 0u)
            x = __fmul_rn(x, x > 0.0f ? less : rep);
        // (without an occurrence there is nothing to subtract: an infinite penalty
        // times zero would be NaN)
        if (g != 0u)
            x = __fsub_rn(__fmaf_rn(-freq, (float)g, x), pres);
        if (w & kBias)
            x = __fadd_rn(x, __uint_as_float(s.bias[at]));
        return x;
    };
    while (row < r1) {
        V v[kR][kPer];
        Words ok[kR][kPer];
        uint64_t see[kR];
#pragma unroll
        for (int q = 0; q < kR; ++q) {
            const int me = row + q * step - r0;
            see[q] = a.tree_mask != nullptr ? next_see[q] : (me < 63 ? (2ull << me) - 1u : ~0ull);
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                v[q][k] = next[q][k];
                ok[q][k] = next_ok[q][k];
            }
        }
        const int coming = row + kR * step;
#pragma unroll
        for (int q = 0; q < kR; ++q)
            if (coming + q * step < r1)
                load(coming + q * step, next[q], next_ok[q], next_see[q]);
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            if (listed[k] != 0) {
                // through shared memory, so that a lane takes a listed logit
                // wherever it lies
#pragma unroll
                for (int q = 0; q < kR; ++q)
                    v[q][k].store(&s.stage[warp][q][lane * kVec]);
                __syncwarp();
                for (int e = lane; e < listed[k]; e += 32) {
                    const int i = s.order[warp][k][e], at = start_of(k) + i;
                    const uint32_t w = s.word[at];
#pragma unroll
                    for (int q = 0; q < kR; ++q) {
                        const int r = row + q * step;
                        const int j = kSame ? i : i + shift_of(r) - (kVec - 1);
                        if (r < r1 && (kSame || (uint32_t)j < (uint32_t)S::kWindow)) {
                            Vec<T, 1> x;
                            x.load(&s.stage[warp][q][j]);
                            x.set(0, adjusted(r, see[q], at, w, x.get(0)));
                            x.store(&s.stage[warp][q][j]);
                        }
                    }
                }
                __syncwarp();
#pragma unroll
                for (int q = 0; q < kR; ++q)
                    v[q][k].load(&s.stage[warp][q][lane * kVec]);
            }
#pragma unroll
            for (int q = 0; q < kR; ++q) {
                const int r = row + q * step;
                if (r >= r1)
                    break;
                const int t = token(r, k);
                T *dst = static_cast<T *>(a.out) + (int64_t)r * a.out_row_stride;
                v[q][k].mask(__funnelshift_r(ok[q][k].lo, ok[q][k].hi, t & 31));
                if (t >= 0 && t + kVec <= a.V) {
                    v[q][k].store(dst + t);
                } else if (t + kVec > 0 && t < a.V) {
                    for (int j = 0; j < kVec; ++j)
                        if (t + j >= 0 && t + j < a.V) {
                            Vec<T, 1> one;
                            one.set(0, v[q][k].get(j));
                            one.store(dst + t + j);
                        }
                }
            }
        }
        row = coming;
    }
}

template <typename T, int kTile, int kVec, int kR, bool kSame>
cudaError_t launch_one(const LogitsLaunch &a, int num_sms, cudaStream_t stream)
{
    const size_t smem = sizeof(Smem<T, kTile, kVec, kR, kSame>);
    static bool configured[64] = {};
    static int resident[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    auto kernel = k7_logits<T, kTile, kVec, kR, kSame>;
    int per_sm = dev < 64 && configured[dev] ? resident[dev] : 0;
    if (per_sm == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem);
        if (e != cudaSuccess)
            return e;
        per_sm = std::max(per_sm, 1);
        if (dev < 64) {
            resident[dev] = per_sm;
            configured[dev] = true;
        }
    }
    // a row's vectors start up to kVec - 1 tokens before its first token
    const int64_t tiles = ((int64_t)a.V + kVec - 1 + kTile - 1) / kTile;
    // A sequence's rows are shared out to as many CTAs as finish soonest.  A CTA's
    // start takes as long as some two rows, and the scan as one per 4096 tokens
    // (16 x 64 rows of 131072, FP32: with history 4096 193 us, 199 for eight rows
    // flat; with 65536 257 us, 321 for two rows flat).
    const int64_t start = 2 + (a.history != nullptr ? a.history_size / a.seqs / 4096 : 0);
    const int64_t rows = std::max<int64_t>(1, (a.rows + a.seqs - 1) / a.seqs), units = tiles * a.seqs;
    const int64_t wave = (int64_t)per_sm * num_sms;
    int64_t chunks = 1;
    double best = 0.0;
    for (int64_t c = 1; c <= std::max<int64_t>(1, std::min<int64_t>(rows / start, 64)); ++c) {
        const int64_t waves = (units * c + wave - 1) / wave;
        const double rate = 1.0 / (waves * ((rows + c - 1) / c + (double)start));
        if (rate > best * 1.02) {
            best = rate;
            chunks = c;
        }
    }
    // too few to fill the GPU once: as many as fill it
    if (units * chunks < wave)
        chunks = std::max(chunks, std::min<int64_t>(rows, wave / units));
    return launch_pdl(kernel, dim3((unsigned)tiles, (unsigned)a.seqs, (unsigned)chunks), dim3(kThreads),
                      smem, stream, 1, a);
}

template <typename T>
cudaError_t launch_type(const LogitsLaunch &a, int num_sms, cudaStream_t stream)
{
    constexpr int kVec = 16 / (int)sizeof(T);
    const uintptr_t src = reinterpret_cast<uintptr_t>(a.logits), dst = reinterpret_cast<uintptr_t>(a.out);
    const bool one = a.rows <= 1;
    if ((src & 15u) != (dst & 15u) || (!one && ((a.row_stride - a.out_row_stride) * (int64_t)sizeof(T)) % 16 != 0))
        return launch_one<T, 1024, 1, 1, true>(a, num_sms, stream);
    const bool same = one || (a.row_stride * (int64_t)sizeof(T)) % 16 == 0;
    // wide tiles (two accesses per thread and row) scan the history half as
    // often, very wide ones (four) where a CTA has a row or two, so that its
    // start is shared by more; narrow ones give twice the CTAs where there are
    // few.  One bf16 row in flight leaves more of a CTA's registers to the lists
    // (two: 16 x 64 rows of 131072 132 us, one 125); FP32 wants two (193, 206).
    constexpr int kNarrow = kThreads * kVec, kWide = 2 * kNarrow, kVery = 4 * kNarrow;
    if (same && a.rows <= 2LL * a.seqs && (int64_t)((a.V + kVery - 1) / kVery) * a.seqs >= 4 * num_sms)
        return launch_one<T, kVery, kVec, 1, true>(a, num_sms, stream);
    if ((int64_t)((a.V + kWide - 1) / kWide) * a.seqs >= 2 * num_sms)
        return same ? launch_one<T, kWide, kVec, sizeof(T) == 2 ? 1 : 2, true>(a, num_sms, stream)
                    : launch_one<T, kWide, kVec, sizeof(T) == 2 ? 1 : 2, false>(a, num_sms, stream);
    return same ? launch_one<T, kNarrow, kVec, 2, true>(a, num_sms, stream)
                : launch_one<T, kNarrow, kVec, 2, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_logits_adjust(const LogitsLaunch &a, bool f32, int num_sms, cudaStream_t stream)
{
    return f32 ? launch_type<float>(a, num_sms, stream) : launch_type<uint16_t>(a, num_sms, stream);
}

}  // namespace rc
