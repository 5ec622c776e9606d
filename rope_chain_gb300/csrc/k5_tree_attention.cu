// K5: attention of a tree of drafted tokens over the paged context cache.
//
// Sequence b has context_len[b] cached tokens and n drafted ones (nodes); the
// K | V row of context token p is logical key p, that of node j logical key
// context_len[b] + j, and logical key p lives in block block_table[b, p / bs]
// at offset p % bs.  Node i sees every context key and the nodes its mask row
// names (without a mask: j <= i).  With t = scale * q.k in FP32,
//   out = sum_j exp(t_j - m) v_j / sum_j exp(t_j - m),  m = max_j t_j
// over the seen keys, in one pass: m, the sum and the output are running
// values, rescaled when m grows (exponentials are powers of two: the scores
// carry a factor log2 e).  A row that sees nothing gives zeros.
//
// Work split.  The query heads of one KV head and the nodes of one sequence
// share its keys, so a unit is (sequence, KV head, tile of rows), its rows
// being (node, query head of the group).  All units' key tiles, laid end to
// end, are cut into equal ranges, one per CTA, from the lengths on the
// device: the host needs no lengths, and a single long context fills the GPU
// as a batch does.  A unit that crosses a cut leaves FP32 partials (output,
// m, sum) in the workspace, which a second kernel joins in key order (no
// atomics: the result does not depend on timing).
#include "rc_internal.cuh"
#include "rc_tcgen05.cuh"

#include <algorithm>
#include <cmath>

namespace rc {

__device__ unsigned int g_attention_faults;

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kKeyTile = 128;          // keys per step of a CTA

struct Args : TreeAttentionLaunch {
    float scale_log2;                  // scale * log2 e
    int32_t min_tiles;                 // fewest key tiles a CTA is given
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- schedule

struct Seq {
    int32_t r0, n;                     // first row, nodes
    int32_t ctx, keys;                 // context keys, all keys
};

__device__ __forceinline__ Seq seq_of(const Args &a, int b) {
    Seq s;
    s.r0 = (int32_t)max((int64_t)0, min((int64_t)__ldg(a.row_start + b), a.rows));
    const int32_t r1 = (int32_t)max((int64_t)s.r0, min((int64_t)__ldg(a.row_start + b + 1), a.rows));
    s.n = r1 - s.r0;
    const int64_t ctx = max(__ldg(a.context_len + b), 0);
    const int64_t room = (int64_t)a.table_width * a.block_size;
    s.keys = (int32_t)min(ctx + s.n, room);
    s.ctx = (int32_t)min(ctx, (int64_t)s.keys);
    return s;
}

template <int kRows> __device__ __forceinline__ int row_tiles(const Args &a, const Seq &s) {
    return (s.n * a.group + kRows - 1) / kRows;
}
__device__ __forceinline__ int key_tiles(const Seq &s) { return max(1, (s.keys + kKeyTile - 1) / kKeyTile); }

template <int kRows> __device__ __forceinline__ int64_t tiles_of(const Args &a, int b) {
    const Seq s = seq_of(a, b);
    return (int64_t)row_tiles<kRows>(a, s) * a.kv_heads * key_tiles(s);
}

struct Place {
    int64_t total, used;               // key tiles of all units; CTAs that have some
    int64_t lo, hi;                    // this CTA's range
    int32_t b;                         // the sequence of `at`
    int64_t off;                       // `at` within the sequence's tiles
};

// The range of CTA c of `ctas`, and where its first tile lies.  Called by all kThreads threads; each takes a run of
// sequences, and the thread whose run holds the tile walks it.
template <int kRows, int kThreads>
__device__ Place locate(const Args &a, int c, int ctas) {
    __shared__ int64_t warp_sum[kThreads / 32];
    __shared__ int64_t found_off;
    __shared__ int32_t found_b;
    const int per = (a.seqs + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, a.seqs), b1 = min(b0 + per, a.seqs);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += tiles_of<kRows>(a, b);
    int64_t run = mine;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o)
            run += v;
    }
    if (lane == 31)
        warp_sum[warp] = run;
    __syncthreads();
    Place p;
    p.total = 0;
    int64_t before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp)
            before += warp_sum[w];
        p.total += warp_sum[w];
    }
    before += run - mine;
    p.used = max((int64_t)1, min((int64_t)ctas, p.total / a.min_tiles));
    p.lo = c < p.used ? p.total * c / p.used : p.total;
    p.hi = c < p.used ? p.total * (c + 1) / p.used : p.total;
    p.b = 0;
    p.off = 0;
    if (p.lo >= p.hi)
        return p;                      // uniform
    if (p.lo >= before && p.lo < before + mine) {
        int64_t off = p.lo - before;
        int b = b0;
        for (int64_t t; off >= (t = tiles_of<kRows>(a, b)); ++b)
            off -= t;
        found_b = b;
        found_off = off;
    }
    __syncthreads();
    p.b = found_b;
    p.off = found_off;
    return p;
}

// One piece of a unit: key tiles k0 .. k0 + count - 1 of its kt.
struct Piece {
    Seq s;
    int32_t b, unit, h, tile;          // sequence, unit within it, its KV head and row tile
    int32_t k0, count, kt;
    int64_t begin;                     // the unit's first tile among all units'
    __device__ bool whole() const { return k0 == 0 && count == kt; }
};

// The pieces of a CTA's range, in order.
template <int kRows> struct Walk {
    int64_t pos, off, hi;
    int32_t b;
    __device__ explicit Walk(const Place &p) : pos(p.lo), off(p.off), hi(p.hi), b(p.b) {}
    __device__ bool next(const Args &a, Piece &u) {
        while (pos < hi) {
            u.s = seq_of(a, b);
            u.kt = key_tiles(u.s);
            const int rt = row_tiles<kRows>(a, u.s);
            const int64_t tiles = (int64_t)rt * a.kv_heads * u.kt;
            if (off >= tiles) {                         // the next sequence with rows
                off -= tiles;
                ++b;
                continue;
            }
            u.b = b;
            u.unit = (int32_t)(off / u.kt);
            u.k0 = (int32_t)(off - (int64_t)u.unit * u.kt);
            u.h = u.unit / rt;
            u.tile = u.unit - u.h * rt;
            u.count = (int32_t)min((int64_t)(u.kt - u.k0), hi - pos);
            u.begin = pos - u.k0;
            pos += u.count;
            off += u.count;
            if (a.partial == nullptr) {
                // without a workspace a unit belongs to the CTA of its first tile
                if (u.k0 != 0)
                    continue;
                u.count = u.kt;
            }
            return true;
        }
        return false;
    }
};

// A partial: a header, then kRows x 64 outputs (not divided by the sum), kRows
// maxima and kRows sums.  Each CTA has two: slot 2c for the unit that an
// earlier CTA began, slot 2c + 1 for one that it begins and a later CTA ends,
// whose header names the unit and its last CTA (or says that there is none).
struct Header {
    int32_t last;                      // slot 2c + 1: last CTA of the unit, 0 without a unit
    int32_t b, unit;
    int32_t unfinite;
};
constexpr int kHeaderFloats = sizeof(Header) / sizeof(float);
template <int kRows> constexpr int kSlotFloats = kHeaderFloats + kRows * (kHeadDim + 2);
template <int kRows> __device__ __forceinline__ float *slot_of(const Args &a, int64_t slot) {
    return a.partial + slot * kSlotFloats<kRows>;
}
template <int kRows> constexpr int kSlotOut = kHeaderFloats;
template <int kRows> constexpr int kSlotMax = kSlotOut<kRows> + kRows * kHeadDim;
template <int kRows> constexpr int kSlotSum = kSlotMax<kRows> + kRows;

__device__ __forceinline__ bool sees(const Args &a, const Seq &s, int i, int j) {
    if (a.tree_mask == nullptr)
        return j <= i;
    return (j >> 6) < a.mask_words &&
           ((__ldg(a.tree_mask + (int64_t)(s.r0 + i) * a.mask_words + (j >> 6)) >> (j & 63)) & 1u) != 0u;
}

// Element offset of logical key p's row in the cache, -1 without a valid block.
__device__ __forceinline__ int64_t key_offset(const Args &a, int b, int h, int p) {
    const uint32_t bs = (uint32_t)a.block_size, page = (uint32_t)p / bs;
    const int32_t blk = __ldg(a.block_table + b * a.table_stride + page);
    if (blk < 0 || blk >= a.num_blocks)
        return -1;
    return (((int64_t)blk * a.kv_heads + h) * bs + ((uint32_t)p - page * bs)) * (2 * kHeadDim);
}

// The header of this CTA's part of a split unit.
template <int kRows>
__device__ void write_header(const Args &a, const Place &p, const Piece &u, bool unfinite) {
    Header h{0, u.b, u.unit, unfinite ? 1 : 0};
    if (u.k0 == 0) {
        const int64_t end = u.begin + u.kt;
        int64_t last = (end - 1) * p.used / p.total;             // the CTA of the unit's last tile
        while (p.total * (last + 1) / p.used < end)
            ++last;
        while (p.total * last / p.used >= end)
            --last;
        h.last = (int32_t)last;
    }
    *reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + (u.k0 == 0 ? 1 : 0))) = h;
}

// A drafted V row that is infinite or NaN must not reach rows that do not see
// it (0 * inf in the matrix product), so the products take zeros in its place
// and the rows that see it get it added here.  Rare: only where the flag of a
// unit is set.
__device__ __noinline__ float add_unfinite(const Args &a, const Seq &s, int b, int h, int i, int d, float x) {
    for (int j = 0; j < min(s.n, s.keys - s.ctx); ++j) {
        if (!sees(a, s, i, j))
            continue;
        const int64_t o = key_offset(a, b, h, s.ctx + j);
        const uint32_t v = o < 0 ? 0u : (uint32_t)a.cache[o + kHeadDim + d] << 16;
        if ((v & 0x7F800000u) == 0x7F800000u)
            x += __uint_as_float(v);
    }
    return x;
}

// ------------------------------------------------- few rows: mma.sync tiles
//
// Up to 32 rows share a key (one drafted token of a group of 8, a small
// tree): the kernel is bound by reading the cache, each K | V row of 256
// bytes once.  Every warp of a CTA streams its own 16 of a tile's 128 keys
// through its own ring of cp.async stages, with its own running maximum,
// sum and output, so the warps never wait for one another until the unit's
// end, where they are joined in shared memory.  Products are m16n8k16: rows x
// keys for the scores, whose accumulator layout is the operand layout of the
// second product, so the weights stay in registers (rounded to bf16 there,
// which the tensor cores require; the sum takes them unrounded).

constexpr int kWarps = 8, kSmallThreads = 32 * kWarps;
constexpr int kChunk = 16;                                   // keys per warp and step
constexpr uint32_t kChunkBytes = kChunk * 2 * kHeadDim * 2;  // 4 KiB

template <int kTiles> constexpr int kRing = kTiles == 1 ? 3 : 5;
// The rings; at a unit's end they hold the warps' outputs (32 KiB per row tile).
template <int kTiles> constexpr uint32_t kSmallSmem = kWarps * kRing<kTiles> * kChunkBytes;

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy16_real(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void load4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void load4_t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Zeros in place of infinite and NaN halves of a register of V whose two keys
// are drafted ones (lo, hi); true if there was one.
__device__ __forceinline__ bool finite_only(uint32_t &w, bool lo, bool hi) {
    const bool x = lo && (w & 0x00007F80u) == 0x00007F80u, y = hi && (w & 0x7F800000u) == 0x7F800000u;
    if (x)
        w &= 0xFFFF0000u;
    if (y)
        w &= 0x0000FFFFu;
    return x || y;
}

template <int kTiles>
__global__ void __launch_bounds__(kSmallThreads, kTiles == 1 ? 2 : 1)
k5_small(const __grid_constant__ Args a)
{
    constexpr int kRows = 16 * kTiles, kStages = kRing<kTiles>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_max[kWarps][kRows], s_sum[kWarps][kRows];
    __shared__ uint32_t s_real[kWarps][kStages];       // which of a chunk's keys exist
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (kStages * kChunkBytes);
    pdl_trigger();
    pdl_wait();

    const Place at = locate<kRows, kSmallThreads>(a, blockIdx.x, gridDim.x);
    if (a.partial != nullptr && threadIdx.x == 0)
        reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + 1))->last = 0;
    Walk<kRows> walk(at);
    Piece u;
    while (walk.next(a, u)) {
        const Seq &s = u.s;
        const int b = u.b, h = u.h, tile = u.tile, unit = u.unit, k0 = u.k0, count = u.count;

        // this thread's rows: lane / 4 and lane / 4 + 8 of each row tile
        int node[kTiles][2];
        uint32_t qf[kTiles][4][4];
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
            const uint32_t *src[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = tile * kRows + m * 16 + 8 * e + (lane >> 2);
                const int i = r / a.group;
                node[m][e] = i < s.n ? i : -1;
                src[e] = reinterpret_cast<const uint32_t *>(
                    a.q + (int64_t)(s.r0 + i) * a.q_row_stride + (h * a.group + r - i * a.group) * kHeadDim);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    qf[m][k][e] = node[m][e & 1] >= 0 ? __ldg(src[e & 1] + 8 * k + (lane & 3) + 4 * (e >> 1)) : 0u;
            }
        }
        float o[kTiles][8][4], top[kTiles][2], sum[kTiles][2];
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                top[m][e] = -INFINITY;
                sum[m][e] = 0.0f;
            }
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[m][n][e] = 0.0f;
        }
        bool unfinite = false;

        // Chunk j's key of this lane: its row's offset in the cache, -1 for
        // none.  Looked up one chunk before the copies that use it.
        auto look_up = [&](int j) -> int64_t {
            const int p = (k0 + j) * kKeyTile + warp * kChunk + (lane & 15);
            if (j >= count || p >= s.keys)
                return -1;
            const int64_t src = key_offset(a, b, h, p);
            if (src < 0 && lane < 16 && unit == 0 && p % a.block_size == 0 && a.err != nullptr)
                atomicAdd(a.err, 1);                   // once per block: at its first key
            return src;
        };
        int64_t from = look_up(0);
        auto issue = [&](int j) {
            const int st = j % kStages;
            const uint32_t real = __ballot_sync(0xFFFFFFFFu, from >= 0) & 0xFFFFu;
            const int64_t first = __shfl_sync(0xFFFFFFFFu, from, 0);
            // a chunk in one block is 4 KiB in a row (any block size where it
            // happens to be; always with blocks of a multiple of 16)
            const bool run = __all_sync(0xFFFFFFFFu, from == first + (lane & 15) * (2 * kHeadDim)) && first >= 0;
            if (lane == 0)
                s_real[warp][st] = real;
            const uint32_t at = ring + st * kChunkBytes + ((lane >> 3) & 1) * (kChunkBytes / 2) + (lane >> 4) * 128;
            if (run) {
                const uint16_t *src = a.cache + first + 8 * lane;
#pragma unroll
                for (int i = 0; i < kChunk / 2; ++i)
                    copy16_real(at + i * 256 + (((lane & 7) ^ ((2 * i + (lane >> 4)) & 7)) << 4), src + i * (4 * kHeadDim));
            } else {
#pragma unroll
                for (int i = 0; i < kChunk / 2; ++i) {
                    const int64_t row = __shfl_sync(0xFFFFFFFFu, from, 2 * i + (lane >> 4));
                    copy16(at + i * 256 + (((lane & 7) ^ ((2 * i + (lane >> 4)) & 7)) << 4),
                           a.cache + (row >= 0 ? row + 8 * (lane & 15) : 0), row >= 0);
                }
            }
            from = look_up(j + 1);
        };
#pragma unroll
        for (int j = 0; j < kStages - 1; ++j) {
            if (j < count)
                issue(j);
            copy_commit();
        }
        for (int j = 0; j < count; ++j) {
            copy_wait<kStages - 2>();
            __syncwarp();
            if (j + kStages - 1 < count)
                issue(j + kStages - 1);
            copy_commit();
            const uint32_t k_at = ring + (j % kStages) * kChunkBytes, v_at = k_at + kChunkBytes / 2;
            const int p0 = (k0 + j) * kKeyTile + warp * kChunk;
            const uint32_t real = s_real[warp][j % kStages];
            const bool drafted = p0 + kChunk > s.ctx;
            float t[kTiles][2][4];
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        t[m][n][e] = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t kf[4];
                const int row = (lane >> 4) * 8 + (lane & 7), c = 2 * k + ((lane >> 3) & 1);
                load4(kf, k_at + row * 128 + ((c ^ (row & 7)) << 4));
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    mma16816(t[m][0], qf[m][k], kf[0], kf[1]);
                    mma16816(t[m][1], qf[m][k], kf[2], kf[3]);
                }
            }
            if (real != 0xFFFFu || drafted) {
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int in = 8 * n + 2 * (lane & 3) + (e & 1), i = node[m][e >> 1];
                            const int p = p0 + in;
                            if (!((real >> in) & 1u) || (p >= s.ctx && (i < 0 || !sees(a, s, i, p - s.ctx))))
                                t[m][n][e] = -INFINITY;
                        }
            }
            uint32_t pf[kTiles][4];
            float now[kTiles][2];
            bool grew = false;
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(fmaxf(t[m][0][2 * e], t[m][0][2 * e + 1]),
                                    fmaxf(t[m][1][2 * e], t[m][1][2 * e + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
                    now[m][e] = fmaxf(top[m][e], x * a.scale_log2);
                    grew |= now[m][e] > top[m][e];
                }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float shrink = now[m][e] == -INFINITY ? 1.0f : ex2(top[m][e] - now[m][e]);
                        top[m][e] = now[m][e];
                        sum[m][e] *= shrink;
#pragma unroll
                        for (int n = 0; n < 8; ++n) {
                            o[m][n][2 * e] *= shrink;
                            o[m][n][2 * e + 1] *= shrink;
                        }
                    }
            }
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = top[m][e] == -INFINITY ? 0.0f : -top[m][e];
                    float part = 0.0f;
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            float &w = t[m][n][2 * e + f];
                            w = ex2(__fmaf_rn(w, a.scale_log2, ref));
                            part += w;
                        }
                    sum[m][e] += part;
                }
                pf[m][0] = pack_bf16x2(t[m][0][0], t[m][0][1]);
                pf[m][1] = pack_bf16x2(t[m][0][2], t[m][0][3]);
                pf[m][2] = pack_bf16x2(t[m][1][0], t[m][1][1]);
                pf[m][3] = pack_bf16x2(t[m][1][2], t[m][1][3]);
            }
#pragma unroll
            for (int n = 0; n < 8; n += 2) {
                uint32_t vf[4];
                const int row = ((lane >> 3) & 1) * 8 + (lane & 7), c = n + (lane >> 4);
                load4_t(vf, v_at + row * 128 + ((c ^ (row & 7)) << 4));
                if (drafted) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int p = p0 + 8 * (q & 1) + 2 * (lane & 3);
                        unfinite |= finite_only(vf[q], p >= s.ctx, p + 1 >= s.ctx);
                    }
                }
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    mma16816(o[m][n], pf[m], vf[0], vf[1]);
                    mma16816(o[m][n + 1], pf[m], vf[2], vf[3]);
                }
            }
            __syncwarp();
        }
        copy_wait<0>();

        // The warps' parts, joined.
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x = sum[m][e];
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
                if ((lane & 3) == 0) {
                    const int r = m * 16 + 8 * e + (lane >> 2);
                    s_max[warp][r] = top[m][e];
                    s_sum[warp][r] = x;
                }
            }
        unfinite = __syncthreads_or(unfinite) != 0;     // also: every ring is drained
        float *outs = reinterpret_cast<float *>(smem) + warp * (16 * kHeadDim);
        const bool whole = u.whole();
        float *slot = whole ? nullptr : slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + (k0 == 0 ? 1 : 0));
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * e + (lane >> 2);
                float now = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    now = fmaxf(now, s_max[w][m * 16 + r]);
                const float f = ex2(top[m][e] - (now == -INFINITY ? 0.0f : now));
#pragma unroll
                for (int n = 0; n < 8; ++n) {
                    // two columns of row r; the column pairs of odd rows are
                    // turned so that a warp's stores spread over the banks
                    const int col = (8 * n + 2 * (lane & 3)) ^ ((r & 3) << 3);
                    *reinterpret_cast<float2 *>(outs + r * kHeadDim + col) =
                        make_float2(o[m][n][2 * e] * f, o[m][n][2 * e + 1] * f);
                }
            }
            __syncthreads();
            // 16 rows of 64: thread -> row threadIdx / 16, four columns
            const int r = threadIdx.x >> 4, col = (threadIdx.x & 15) * 4;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float now = -INFINITY, total = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                now = fmaxf(now, s_max[w][m * 16 + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 y = *reinterpret_cast<const float4 *>(
                    reinterpret_cast<const float *>(smem) + w * (16 * kHeadDim) + r * kHeadDim + (col ^ ((r & 3) << 3)));
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
                total = __fmaf_rn(s_sum[w][m * 16 + r], ex2(s_max[w][m * 16 + r] - (now == -INFINITY ? 0.0f : now)), total);
            }
            const int row = tile * kRows + m * 16 + r, i = row / a.group;
            if (!whole) {
                *reinterpret_cast<float4 *>(slot + kSlotOut<kRows> + (m * 16 + r) * kHeadDim + col) = x;
                if (col == 0) {
                    slot[kSlotMax<kRows> + m * 16 + r] = now;
                    slot[kSlotSum<kRows> + m * 16 + r] = total;
                }
                if (threadIdx.x == 0 && m == 0)
                    write_header<kRows>(a, at, u, unfinite);
            } else if (i < s.n) {
                const int head = h * a.group + row - i * a.group;
                if (unfinite) {
                    x.x = add_unfinite(a, s, b, h, i, col, x.x);
                    x.y = add_unfinite(a, s, b, h, i, col + 1, x.y);
                    x.z = add_unfinite(a, s, b, h, i, col + 2, x.z);
                    x.w = add_unfinite(a, s, b, h, i, col + 3, x.w);
                }
                const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
                *reinterpret_cast<uint2 *>(a.out + (int64_t)(s.r0 + i) * a.out_row_stride + head * kHeadDim + col) =
                    make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
                if (col == 0 && a.lse != nullptr)
                    a.lse[(int64_t)(s.r0 + i) * (a.kv_heads * a.group) + head] =
                        total == 0.0f ? -INFINITY : __fmaf_rn(now, kLn2, logf(total));
                if (threadIdx.x == 0 && m == 0 && unit == 0 && s.n > 0 && a.err != nullptr &&
                    (int64_t)max(__ldg(a.context_len + b), 0) + s.n > s.keys)
                    atomicAdd(a.err, 1);
            }
            __syncthreads();
        }
    }
}

// ------------------------------------------------ many rows: tcgen05 tiles
//
// From 33 rows per unit on the tensor cores are the bound, and the work goes
// to tcgen05: one 128-row tile of Q per group of four softmax warps (kQ of
// them share each key tile), 128 keys per step.  S = Q K^T lands in TMEM (128
// columns); a thread owns one row, so its maximum and sum need no shuffles;
// the weights go back to TMEM as bf16 over the scores (64 columns), from where
// they are the A operand of O += P V, and O stays in TMEM (64 columns).  O is
// rescaled only when a row's maximum has grown by more than 2^8 since its last
// reference (the weights then stay below 2^8, harmless in FP32 and bf16): by
// the row's own thread, a rare path.
//   loader warp   K and V tiles of 16 KiB by TMA, in boxes of the largest
//                 power of two of keys that divides a block (8 to 128), each
//                 box's block looked up in the table by its own lane
//   MMA warp      S of tile t, then for each further step O of tile t followed
//                 by the next S of tile t, so that one tile's products run
//                 while the other tiles' softmax does
//   softmax       4 warps per tile
// Key tiles that hold drafted keys, or the end, take a masked path; there the
// V rows past the end are zeroed and what is infinite or NaN in a drafted one
// is taken out (see add_unfinite).  Every wait is bounded; on timeout a sticky
// fault bit is raised and all roles leave.

enum : unsigned { kFaultLoad = 1u, kFaultMma = 2u, kFaultSoftmax = 4u, kFaultDrain = 8u };

constexpr uint32_t kTileBytes = kKeyTile * kHeadDim * 2;           // K or V of a step, Q of a tile: 16 KiB
template <int kQ> constexpr int kWideThreads = 128 * kQ + 128;
template <int kQ> constexpr int kWideStages = kQ == 1 ? 3 : 5;
template <int kQ> constexpr uint32_t kTmemCols = kQ == 1 ? 256u : 512u;
template <int kQ> constexpr uint32_t kOCol = 128u * kQ;            // after the scores of all tiles
template <int kQ> constexpr size_t kWideSmem = 1024 + kQ * kTileBytes + kWideStages<kQ> * 2 * kTileBytes;
constexpr float kGrow = 8.0f;                                      // log2: when O is rescaled

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int col, int off, int h, int blk,
                                        uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(off), "r"(h), "r"(blk), "r"(bar)
                 : "memory");
}
// D[tmem] (+)= A[tmem] x B[smem]
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(bdesc), "r"(idesc), "r"(acc) : "memory");
}
// 32 columns of this warp's 32 lanes; complete after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32_async(uint32_t at, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(at));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The values of a load, to be used no earlier than here (after the wait).
__device__ __forceinline__ void loaded32(float *r) {
    asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]),
                      "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]),
                      "+f"(r[15]));
    asm volatile("" : "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]),
                      "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]),
                      "+f"(r[30]), "+f"(r[31]));
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// Which of the keys base .. base + 31 node i sees (bit k: key base + k);
// i < 0: none of the drafted ones.
__device__ uint32_t seen32(const Args &a, const Seq &s, int i, int base) {
    auto below = [](int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); };
    const uint32_t ctx = below(s.ctx - base);
    uint32_t drafted = 0u;
    if (i >= 0 && ctx != 0xFFFFFFFFu) {
        if (a.tree_mask == nullptr) {
            drafted = below(s.ctx + i + 1 - base);
        } else {
            const uint64_t *row = a.tree_mask + (int64_t)(s.r0 + i) * a.mask_words;
            const int j0 = base - s.ctx;                // node of bit 0, negative inside the context
            auto word = [&](int w) { return w >= 0 && w < a.mask_words ? __ldg(row + w) : (uint64_t)0; };
            if (j0 < 0) {
                drafted = (uint32_t)(word(0) << -j0);
            } else {
                const int w = j0 >> 6, sh = j0 & 63;
                uint64_t v = word(w) >> sh;
                if (sh > 32)
                    v |= word(w + 1) << (64 - sh);
                drafted = (uint32_t)v;
            }
        }
    }
    return (ctx | (drafted & ~ctx)) & below(s.keys - base);
}

template <int kQ>
__global__ void __launch_bounds__(kWideThreads<kQ>, kQ == 1 ? 2 : 1)
k5_wide(const __grid_constant__ CUtensorMap map, const __grid_constant__ Args a, int box)
{
    constexpr int kRows = 128 * kQ, kStages = kWideStages<kQ>, kThreads = kWideThreads<kQ>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const uint32_t sQ = smem_u32(smem), sK = sQ + kQ * kTileBytes;     // a stage: K, then V
    __shared__ uint64_t bars[2 * kStages + 4 * kQ + 2];
    __shared__ uint32_t s_tmem, s_skip, s_bad[kStages], s_unfinite[2];
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * kStages, q_ready0 = empty0 + 8u * kStages;
    const uint32_t s_full0 = q_ready0 + 8u * kQ, p_ready0 = s_full0 + 8u * kQ, o_done0 = p_ready0 + 8u * kQ;
    const uint32_t drain = o_done0 + 8u * kQ, v_fixed = drain + 8u;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    constexpr int kLoadWarp = 4 * kQ, kMmaWarp = 4 * kQ + 1;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full0 + 8u * i, 1);
            mbar_init(empty0 + 8u * i, 1);
        }
        for (int t = 0; t < kQ; ++t) {
            mbar_init(q_ready0 + 8u * t, 128);
            mbar_init(s_full0 + 8u * t, 1);
            mbar_init(p_ready0 + 8u * t, 128);
            mbar_init(o_done0 + 8u * t, 1);
        }
        mbar_init(drain, 1);
        mbar_init(v_fixed, 128 * kQ);
        s_unfinite[0] = s_unfinite[1] = 0u;
        // one decision for the CTA: a raised fault skips the work
        s_skip = *reinterpret_cast<volatile unsigned int *>(&g_attention_faults);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tensormap(&map);
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&s_tmem)), "r"(kTmemCols<kQ>) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    pdl_wait();
    auto wait = [&](uint32_t bar, uint32_t parity, unsigned fault) {
        if (mbar_wait_flag(bar, parity, &g_attention_faults))
            return true;
        atomicOr(&g_attention_faults, fault);
        return false;
    };

    const Place at = locate<kRows, kThreads>(a, blockIdx.x, gridDim.x);
    if (a.partial != nullptr && threadIdx.x == 0)
        reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + 1))->last = 0;
    Walk<kRows> walk(at);
    if (s_skip != 0u)
        walk.hi = walk.pos;
    Piece u;
    uint32_t n = 0;                                     // key tiles of earlier pieces
    uint32_t piece = 0;

    if (warp >= 4 * kQ) {
        if (kQ == 1)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == kLoadWarp) {
            const int boxes = kKeyTile / box;           // <= 16
            bool fine = true;
            while (fine && walk.next(a, u)) {
                const Seq &s = u.s;
                // this lane's box of tile j: its block, or -1 for one that is not there
                auto look_up = [&](int j) -> int {
                    const int p = (u.k0 + j) * kKeyTile + lane * box;
                    return j < u.count && lane < boxes && p < s.keys
                               ? __ldg(a.block_table + u.b * a.table_stride + (uint32_t)p / (uint32_t)a.block_size) : 0;
                };
                int blk = look_up(0);
                for (int j = 0; j < u.count; ++j, ++n) {
                    const uint32_t st = n % kStages, full = full0 + 8u * st;
                    const int p = (u.k0 + j) * kKeyTile + lane * box;
                    const bool mine = lane < boxes && p < s.keys;
                    const int off = mine ? (int)((uint32_t)p % (uint32_t)a.block_size) : 0;
                    const bool bad = mine && (blk < 0 || blk >= a.num_blocks);
                    if (bad && u.unit == 0 && off == 0 && a.err != nullptr)
                        atomicAdd(a.err, 1);            // once per block: at its first key
                    fine = wait(empty0 + 8u * st, ((n / kStages) & 1u) ^ 1u, kFaultLoad);
                    fine = __all_sync(0xFFFFFFFFu, fine);
                    if (!fine)
                        break;
                    const uint32_t bads = __ballot_sync(0xFFFFFFFFu, bad), loads = __ballot_sync(0xFFFFFFFFu, mine);
                    if (lane == 0) {
                        s_bad[st] = bads;
                        mbar_expect_tx(full, (uint32_t)__popc(loads) * box * 256u);
                    }
                    __syncwarp();
                    if (mine) {
                        // a block out of range reads zeros: one past the last
                        const int from = bad ? a.num_blocks : blk;
                        const uint32_t dst = sK + st * (2 * kTileBytes) + (uint32_t)(lane * box) * 128u;
                        tma_box(dst, &map, 0, off, u.h, from, full);
                        tma_box(dst + kTileBytes, &map, kHeadDim, off, u.h, from, full);
                    }
                    blk = look_up(j + 1);
                }
            }
            // what was loaded has landed before shared memory is given back
            for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i)
                if (!mbar_wait_own(full0 + 8u * (i % kStages), (i / kStages) & 1u)) {
                    atomicOr(&g_attention_faults, kFaultDrain);
                    break;
                }
        } else if (warp == kMmaWarp) {
            if (lane == 0) {
                constexpr uint32_t idesc_s = make_idesc(128, kKeyTile, false), idesc_o = make_idesc(128, kHeadDim, true);
                auto scores = [&](int t, uint32_t st) {
                    const uint32_t q = sQ + t * kTileBytes, k = sK + st * (2 * kTileBytes);
#pragma unroll
                    for (int kk = 0; kk < kHeadDim / 16; ++kk)
                        mma_bf16(tmem + 128u * t, smem_desc_sw128(q + 32u * kk, 16u, 1024u),
                                 smem_desc_sw128(k + 32u * kk, 16u, 1024u), idesc_s, kk != 0);
                    mma_commit(s_full0 + 8u * t);
                };
                bool fine = true;
                while (fine && walk.next(a, u)) {
                    for (int t = 0; t < kQ && fine; ++t)
                        fine = wait(q_ready0 + 8u * t, piece & 1u, kFaultMma);
                    fine = fine && wait(full0 + 8u * (n % kStages), (n / kStages) & 1u, kFaultMma);
                    if (!fine)
                        break;
                    tc_fence_after();
                    for (int t = 0; t < kQ; ++t)
                        scores(t, n % kStages);
                    for (int j = 0; j < u.count && fine; ++j, ++n) {
                        const uint32_t st = n % kStages, nx = (n + 1) % kStages;
                        const uint32_t v = sK + st * (2 * kTileBytes) + kTileBytes;
                        for (int t = 0; t < kQ; ++t) {
                            fine = wait(p_ready0 + 8u * t, n & 1u, kFaultMma);
                            if (!fine)
                                break;
                            tc_fence_after();
#pragma unroll
                            for (int kk = 0; kk < kKeyTile / 16; ++kk)
                                mma_bf16_ta(tmem + kOCol<kQ> + 64u * t, tmem + 128u * t + 8u * kk,
                                            smem_desc_sw128(v + 2048u * kk, 8192u, 1024u), idesc_o, (j | kk) != 0);
                            mma_commit(o_done0 + 8u * t);
                            if (t == kQ - 1)
                                mma_commit(empty0 + 8u * st);
                            if (j + 1 < u.count) {
                                if (t == 0)
                                    fine = wait(full0 + 8u * nx, ((n + 1) / kStages) & 1u, kFaultMma);
                                if (!fine)
                                    break;
                                tc_fence_after();
                                scores(t, nx);
                            }
                        }
                    }
                    ++piece;
                }
                mma_commit(drain);
                if (!mbar_wait_own(drain, 0u))
                    atomicOr(&g_attention_faults, kFaultDrain);
            }
            __syncwarp();
        }
    } else {
        if (kQ == 1)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2;                        // this group's row tile
        const int r = threadIdx.x & 127;                // this thread's row of it, and its TMEM lane
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + 128u * t, tO = tmem + lanes + kOCol<kQ> + 64u * t;
        const uint32_t q_at = sQ + t * kTileBytes + (uint32_t)r * 128u;
        uint32_t fixes = 0;                             // tiles whose V was looked through
        bool fine = true;
        while (fine && walk.next(a, u)) {
            const Seq &s = u.s;
            const int row = u.tile * kRows + 128 * t + r, node = row / a.group, i = node < s.n ? node : -1;
            const int head = u.h * a.group + row - node * a.group;
            {
                const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (int64_t)(s.r0 + node) * a.q_row_stride +
                                                                   head * kHeadDim);
                uint4 w[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    w[c] = i >= 0 ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    st_shared_v4(q_at + (uint32_t)((c ^ (r & 7)) << 4), w[c]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive_local(q_ready0 + 8u * t);
            }
            float top = -INFINITY, sum = 0.0f;          // reference (log2) and sum of the row
            bool unfinite = false;
            for (int j = 0; j < u.count; ++j, ++n) {
                const int p0 = (u.k0 + j) * kKeyTile;
                fine = wait(s_full0 + 8u * t, n & 1u, kFaultSoftmax);
                fine = __all_sync(0xFFFFFFFFu, fine);
                if (!fine)
                    break;
                tc_fence_after();
                float x[128];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_ld32_async(tS + 32u * c, x + 32 * c);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    loaded32(x + 32 * c);
                const uint32_t st = n % kStages;
                const bool last_keys = p0 + kKeyTile > s.ctx;
                const uint32_t bads = *reinterpret_cast<volatile uint32_t *>(&s_bad[st]);
                if (last_keys || bads != 0u) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t see = seen32(a, s, i, p0 + 32 * c);
                        if (bads != 0u) {
                            for (int k = 0; k < 32; ++k)
                                if ((bads >> ((32 * c + k) / box)) & 1u)
                                    see &= ~(1u << k);
                        }
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            x[32 * c + k] = (see >> k) & 1u ? x[32 * c + k] : -INFINITY;
                    }
                }
                if (last_keys) {
                    // the tile's V: zeros past the end, and in place of what is
                    // not finite in drafted keys.  The groups share the work and
                    // wait for one another; a piece that met such a value leaves
                    // its number (in the word of its parity: a group is never two
                    // tiles ahead of one that has not read it).
                    fine = wait(full0 + 8u * st, (n / kStages) & 1u, kFaultSoftmax);    // complete: seen through S
                    const uint32_t v = sK + st * (2 * kTileBytes) + kTileBytes;
                    bool found = false;
                    for (int e = threadIdx.x; e < kKeyTile * 8; e += 128 * kQ) {
                        const int key = p0 + (e >> 3);
                        if (key < s.ctx)
                            continue;
                        const uint32_t chunk = v + 16u * e;
                        uint4 w = make_uint4(0, 0, 0, 0);
                        bool write = true;
                        if (key < s.keys) {
                            w = ld_shared_v4(chunk);
                            write = finite_only(w.x, true, true);
                            write |= finite_only(w.y, true, true);
                            write |= finite_only(w.z, true, true);
                            write |= finite_only(w.w, true, true);
                            found |= write;
                        }
                        if (write)
                            st_shared_v4(chunk, w);
                    }
                    if (found)
                        *reinterpret_cast<volatile uint32_t *>(&s_unfinite[piece & 1u]) = piece + 1u;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive_local(v_fixed);
                    fine = wait(v_fixed, fixes & 1u, kFaultSoftmax) && fine;
                    ++fixes;
                    unfinite |= *reinterpret_cast<volatile uint32_t *>(&s_unfinite[piece & 1u]) == piece + 1u;
                }
                float m = max3(x[0], x[1], x[2]);
#pragma unroll
                for (int k = 3; k + 1 < 128; k += 2)
                    m = max3(m, x[k], x[k + 1]);
                m = fmaxf(m, x[127]) * a.scale_log2;
                const bool grew = m > top + kGrow || (top == -INFINITY && m > -INFINITY);
                if (__any_sync(0xFFFFFFFFu, grew)) {
                    const float shrink = grew ? ex2(top - m) : 1.0f;    // top -inf: 0
                    if (j > 0) {
                        fine = wait(o_done0 + 8u * t, (n - 1) & 1u, kFaultSoftmax);
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float o[32];
                            uint32_t w[32];
                            tmem_ld32_async(tO + 32u * c, o);
                            tmem_wait_ld();
                            loaded32(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                w[k] = __float_as_uint(o[k] * shrink);
                            tmem_st32(tO + 32u * c, w);
                        }
                        tmem_wait_st();
                    }
                    sum *= shrink;
                    if (grew)
                        top = m;
                }
                const float ref = top == -INFINITY ? 0.0f : -top;
                float part[2] = {0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t w[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        float x0 = x[64 * c + 2 * k], x1 = x[64 * c + 2 * k + 1];
                        fma2_rn(x0, x1, a.scale_log2, a.scale_log2, ref, ref);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        add2_rn(part[0], part[1], x0, x1);
                        w[k] = pack_bf16x2(x0, x1);
                    }
                    tmem_st32(tS + 32u * c, w);
                }
                tmem_wait_st();
                sum += part[0] + part[1];
                tc_fence_before();
                mbar_arrive_local(p_ready0 + 8u * t);
            }
            if (!fine)
                break;
            // the row's output
            fine = wait(o_done0 + 8u * t, (n - 1) & 1u, kFaultSoftmax);
            fine = __all_sync(0xFFFFFFFFu, fine);
            if (!fine)
                break;
            tc_fence_after();
            float o[64];
            tmem_ld32_async(tO, o);
            tmem_ld32_async(tO + 32u, o + 32);
            tmem_wait_ld();
            loaded32(o);
            loaded32(o + 32);
            tc_fence_before();
            if (!u.whole()) {
                float *slot = slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + (u.k0 == 0 ? 1 : 0));
                const int rr = 128 * t + r;
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    *reinterpret_cast<float4 *>(slot + kSlotOut<kRows> + rr * kHeadDim + 4 * k) =
                        make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                slot[kSlotMax<kRows> + rr] = top;
                slot[kSlotSum<kRows> + rr] = sum;
                if (threadIdx.x == 0)
                    write_header<kRows>(a, at, u, unfinite);
            } else if (i >= 0) {
                if (unfinite) {
#pragma unroll
                    for (int k = 0; k < 64; ++k)
                        o[k] = add_unfinite(a, s, u.b, u.h, i, k, o[k]);
                }
                const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
                uint4 *dst = reinterpret_cast<uint4 *>(a.out + (int64_t)(s.r0 + i) * a.out_row_stride + head * kHeadDim);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    dst[k] = make_uint4(pack_bf16x2(o[8 * k] * inv, o[8 * k + 1] * inv),
                                        pack_bf16x2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                        pack_bf16x2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                        pack_bf16x2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
                if (a.lse != nullptr)
                    a.lse[(int64_t)(s.r0 + i) * (a.kv_heads * a.group) + head] =
                        sum == 0.0f ? -INFINITY : __fmaf_rn(top, kLn2, logf(sum));
                if (threadIdx.x == 0 && u.unit == 0 && a.err != nullptr &&
                    (int64_t)max(__ldg(a.context_len + u.b), 0) + s.n > s.keys)
                    atomicAdd(a.err, 1);
            }
            ++piece;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols<kQ>)
                     : "memory");
    }
}

// ----------------------------------------------------------- joining parts
//
// Block (c, y) joins kJoinRows rows of the unit that CTA c began and did not
// end: its own part and those of the CTAs after it, in key order.  The parts'
// weights are made first, one per thread, then four groups of 64 threads (16
// columns of four, four rows) add every fourth part each, and the groups are
// added in order.
constexpr int kJoinThreads = 256, kJoinRows = 4, kJoinParts = 512;

template <int kRows>
__global__ void __launch_bounds__(kJoinThreads)
k5_join(const __grid_constant__ Args a)
{
    __shared__ float s_part[kJoinParts][kJoinRows];        // the part's maximum, then its weight
    __shared__ float s_sum[kJoinParts][kJoinRows];
    __shared__ float4 s_out[3][64];
    __shared__ float s_top[kJoinRows], s_total[kJoinRows];
    pdl_trigger();
    pdl_wait();
    const int c = blockIdx.x;
    const float *own = slot_of<kRows>(a, 2 * (int64_t)c + 1);
    const Header hd = *reinterpret_cast<const Header *>(own);
    if (hd.last == 0)
        return;
    const Seq s = seq_of(a, hd.b);
    const int rt = row_tiles<kRows>(a, s);
    const int h = hd.unit / rt, tile = hd.unit - h * rt;
    const int r0 = blockIdx.y * kJoinRows, parts = hd.last - c + 1;
    if (threadIdx.x == 0 && blockIdx.y == 0 && hd.unit == 0 && a.err != nullptr &&
        (int64_t)max(__ldg(a.context_len + hd.b), 0) + s.n > s.keys)
        atomicAdd(a.err, 1);
    if (tile * kRows + r0 >= s.n * a.group)
        return;
    auto part_of = [&](int k) { return k == 0 ? own : slot_of<kRows>(a, 2 * (int64_t)(c + k)); };
    const int group = threadIdx.x >> 6, r = (threadIdx.x >> 4) & 3, col = (threadIdx.x & 15) * 4;
    bool unfinite = false;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float top = -INFINITY, total = 0.0f;
    // more parts than the table holds are joined in runs of kJoinParts
    for (int k0 = 0; k0 < parts; k0 += kJoinParts) {
        const int n = min(kJoinParts, parts - k0);
        for (int i = threadIdx.x; i < n * kJoinRows; i += kJoinThreads) {
            const float *part = part_of(k0 + i / kJoinRows);
            s_part[i / kJoinRows][i % kJoinRows] = part[kSlotMax<kRows> + r0 + i % kJoinRows];
            s_sum[i / kJoinRows][i % kJoinRows] = part[kSlotSum<kRows> + r0 + i % kJoinRows];
            unfinite |= reinterpret_cast<const Header *>(part)->unfinite != 0;
        }
        unfinite = __syncthreads_or(unfinite) != 0;
        if (threadIdx.x < kJoinRows * 32) {                // a warp per row
            const int row = threadIdx.x >> 5, lane = threadIdx.x & 31;
            float m = k0 == 0 ? -INFINITY : s_top[row];
            const float before = m;
            for (int k = lane; k < n; k += 32)
                m = fmaxf(m, s_part[k][row]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const float ref = m == -INFINITY ? 0.0f : m;
            float sum = 0.0f;
            for (int k = lane; k < n; k += 32) {
                const float f = ex2(s_part[k][row] - ref);
                s_part[k][row] = f;
                sum = __fmaf_rn(s_sum[k][row], f, sum);
            }
            sum = warp_butterfly_sum(sum);
            if (lane == 0) {
                s_total[row] = k0 == 0 ? sum : __fmaf_rn(s_total[row], ex2(before - ref), sum);
                s_top[row] = m;
            }
        }
        __syncthreads();
        const float shrink = k0 == 0 ? 0.0f : ex2(top - (s_top[r] == -INFINITY ? 0.0f : s_top[r]));
        top = s_top[r];
        total = s_total[r];
        x.x *= shrink;
        x.y *= shrink;
        x.z *= shrink;
        x.w *= shrink;
#pragma unroll 8
        for (int k = group; k < n; k += 4) {
            const float f = s_part[k][r];
            const float4 y = *reinterpret_cast<const float4 *>(part_of(k0 + k) + kSlotOut<kRows> + (r0 + r) * kHeadDim + col);
            x.x = __fmaf_rn(y.x, f, x.x);
            x.y = __fmaf_rn(y.y, f, x.y);
            x.z = __fmaf_rn(y.z, f, x.z);
            x.w = __fmaf_rn(y.w, f, x.w);
        }
        __syncthreads();
    }
    if (group > 0)
        s_out[group - 1][threadIdx.x & 63] = x;
    __syncthreads();
    const int row = tile * kRows + r0 + r, i = row / a.group;
    if (group > 0 || i >= s.n)
        return;
#pragma unroll
    for (int g = 0; g < 3; ++g) {
        const float4 y = s_out[g][threadIdx.x];
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
    }
    const int head = h * a.group + row - i * a.group;
    if (unfinite) {
        x.x = add_unfinite(a, s, hd.b, h, i, col, x.x);
        x.y = add_unfinite(a, s, hd.b, h, i, col + 1, x.y);
        x.z = add_unfinite(a, s, hd.b, h, i, col + 2, x.z);
        x.w = add_unfinite(a, s, hd.b, h, i, col + 3, x.w);
    }
    const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
    *reinterpret_cast<uint2 *>(a.out + (int64_t)(s.r0 + i) * a.out_row_stride + head * kHeadDim + col) =
        make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
    if (col == 0 && a.lse != nullptr)
        a.lse[(int64_t)(s.r0 + i) * (a.kv_heads * a.group) + head] =
            total == 0.0f ? -INFINITY : __fmaf_rn(top, kLn2, logf(total));
}

// Which kernel takes a call, by the average rows of a unit (only the totals are
// known on the host; any kernel is right for any unit):
//   up to 16 rows  k5_small<1>;  up to 32  k5_small<2>: the cache's bytes bound
//   beyond         k5_wide: 128 rows a CTA up to 128, else 256 (two row tiles
//                  share each key tile); its TMA boxes need blocks of a
//                  multiple of 8 keys, other block sizes stay with k5_small<2>
enum Variant { kSmall16, kSmall32, kWide128, kWide256 };

Variant variant_for(int64_t rows, int32_t seqs, int32_t group, int32_t block_size) {
    const int64_t mean = (rows + seqs - 1) / seqs * group;
    if (mean <= 16)
        return kSmall16;
    if (mean <= 32 || block_size % 8 != 0)
        return kSmall32;
    return mean <= 128 ? kWide128 : kWide256;
}

// CTAs of a launch (all resident at once) and floats of a partial.
int ctas_of(Variant v, int num_sms) { return v == kSmall16 || v == kWide128 ? 2 * num_sms : num_sms; }
size_t slot_floats(Variant v) {
    switch (v) {
    case kSmall16: return kSlotFloats<16>;
    case kSmall32: return kSlotFloats<32>;
    case kWide128: return kSlotFloats<128>;
    default: return kSlotFloats<256>;
    }
}

template <typename Kernel> cudaError_t allow_smem(Kernel kernel, size_t bytes, bool (&configured)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && configured[dev]))
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64)
        configured[dev] = true;
    return e;
}

template <int kRows> cudaError_t launch_join(const Args &a, int ctas, cudaStream_t stream, const char **why) {
    if (a.partial == nullptr)
        return cudaSuccess;
    *why = "tree attention join launch";
    return launch_pdl(k5_join<kRows>, dim3((unsigned)ctas, kRows / kJoinRows), dim3(kJoinThreads), 0, stream, 1, a);
}

template <int kTiles>
cudaError_t launch_small(const Args &a, int ctas, cudaStream_t stream, const char **why)
{
    static bool configured[64] = {};
    cudaError_t e = allow_smem(k5_small<kTiles>, kSmallSmem<kTiles>, configured);
    if (e != cudaSuccess)
        return e;
    *why = "tree attention launch";
    e = launch_pdl(k5_small<kTiles>, dim3((unsigned)ctas), dim3(kSmallThreads), kSmallSmem<kTiles>, stream, 1, a);
    return e != cudaSuccess ? e : launch_join<16 * kTiles>(a, ctas, stream, why);
}

template <int kQ>
cudaError_t launch_wide(const Args &a, int ctas, cudaStream_t stream, const char **why)
{
    static bool configured[64] = {};
    cudaError_t e = allow_smem(k5_wide<kQ>, kWideSmem<kQ>, configured);
    if (e != cudaSuccess)
        return e;
    // the cache as [num_blocks, kv_heads, block_size, 128], boxes of 64 columns
    // (K or V) and the largest power of two of keys, at most a tile, in a block
    const int box = std::min(kKeyTile, a.block_size & -a.block_size);
    const uint64_t row = 2 * kHeadDim * 2;
    const cuuint64_t dims[4] = {2 * kHeadDim, (cuuint64_t)a.block_size, (cuuint64_t)a.kv_heads, (cuuint64_t)a.num_blocks};
    const cuuint64_t strides[3] = {row, row * a.block_size, row * a.block_size * a.kv_heads};
    const cuuint32_t boxes[4] = {kHeadDim, (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
    CUtensorMap map;
    const EncodeTiledFn enc = encode_fn();
    *why = "tensor map of the cache could not be encoded";
    if (!enc || enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(a.cache), dims, strides, boxes,
                    ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    *why = "tree attention launch";
    e = launch_pdl(k5_wide<kQ>, dim3((unsigned)ctas), dim3(kWideThreads<kQ>), kWideSmem<kQ>, stream, 1, map, a, box);
    return e != cudaSuccess ? e : launch_join<128 * kQ>(a, ctas, stream, why);
}

}  // namespace

size_t tree_attention_workspace(int64_t rows, int32_t seqs, int32_t group, int num_sms)
{
    size_t most = 0;
    for (int32_t block_size : {8, 1}) {                 // whichever the cache has
        const Variant v = variant_for(rows, seqs, group, block_size);
        most = std::max(most, 2 * (size_t)ctas_of(v, num_sms) * slot_floats(v) * sizeof(float));
    }
    return most;
}

cudaError_t launch_tree_attention(const TreeAttentionLaunch &p, int num_sms, cudaStream_t stream,
                                  const char **why)
{
    Args a{};
    static_cast<TreeAttentionLaunch &>(a) = p;
    a.scale_log2 = p.scale * kLog2e;
    a.min_tiles = 4;
    // no unit has more tiles than a CTA takes at least: nothing to split or join
    if ((int64_t)p.table_width * p.block_size <= a.min_tiles * kKeyTile)
        a.partial = nullptr;
    const Variant v = variant_for(p.rows, p.seqs, p.group, p.block_size);
    const int ctas = ctas_of(v, num_sms);
    switch (v) {
    case kSmall16: return launch_small<1>(a, ctas, stream, why);
    case kSmall32: return launch_small<2>(a, ctas, stream, why);
    case kWide128: return launch_wide<1>(a, ctas, stream, why);
    default: return launch_wide<2>(a, ctas, stream, why);
    }
}

cudaError_t read_attention_faults(uint32_t *flags, bool clear)
{
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess)
        return e;
    unsigned int v = 0;
    e = cudaMemcpyFromSymbol(&v, g_attention_faults, sizeof v);
    if (e != cudaSuccess)
        return e;
    *flags = v;
    if (clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_attention_faults, &zero, sizeof zero);
    }
    return e;
}

}  // namespace rc
