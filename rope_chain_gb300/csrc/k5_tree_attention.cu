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

#include <algorithm>
#include <cmath>

namespace rc {

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

// The header of this CTA's part of a split unit: key tiles from k0 of kt, its
// first tile at `begin` of all units' tiles laid end to end.
template <int kRows>
__device__ void write_header(const Args &a, const Place &p, int k0, int kt, int64_t begin, int b, int unit,
                             bool unfinite) {
    Header h{0, b, unit, unfinite ? 1 : 0};
    if (k0 == 0) {
        int64_t last = (begin + kt - 1) * p.used / p.total;      // its range holds the unit's last tile
        while (p.total * (last + 1) / p.used < begin + kt)
            ++last;
        while (p.total * last / p.used >= begin + kt)
            --last;
        h.last = (int32_t)last;
    }
    *reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + (k0 == 0 ? 1 : 0))) = h;
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

__device__ __forceinline__ uint32_t smem_at(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
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
    const uint32_t ring = smem_at(smem) + (uint32_t)warp * (kStages * kChunkBytes);
    pdl_trigger();
    pdl_wait();

    const Place at = locate<kRows, kSmallThreads>(a, blockIdx.x, gridDim.x);
    if (a.partial != nullptr && threadIdx.x == 0)
        reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + 1))->last = 0;
    int64_t pos = at.lo, off = at.off;
    int b = at.b;
    while (pos < at.hi) {
        const Seq s = seq_of(a, b);
        const int kt = key_tiles(s), rt = row_tiles<kRows>(a, s);
        const int64_t seq_tiles = (int64_t)rt * a.kv_heads * kt;
        if (off >= seq_tiles) {                         // the next sequence with rows
            off -= seq_tiles;
            ++b;
            continue;
        }
        const int unit = (int)(off / kt), k0 = (int)(off - (int64_t)unit * kt);
        const int h = unit / rt, tile = unit - h * rt;
        int count = (int)min((int64_t)(kt - k0), at.hi - pos);
        const bool split_ok = a.partial != nullptr;
        if (!split_ok) {
            // without a workspace a unit belongs to the CTA of its first tile
            if (k0 != 0) {
                pos += count;
                off += count;
                continue;
            }
            count = kt;
        }

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
        const bool whole = k0 == 0 && count == kt;
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
                    write_header<kRows>(a, at, k0, kt, pos - k0, b, unit, unfinite);
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
        pos += count;
        off += count;
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

// Row tile of a call: 16 rows while the average unit fits them, else 32.
int tiles_for(int64_t rows, int32_t seqs, int32_t group) {
    const int64_t mean = (rows + seqs - 1) / seqs * group;
    return mean <= 16 ? 1 : 2;
}

int ctas_for(int tiles, int num_sms) { return tiles == 1 ? 2 * num_sms : num_sms; }

template <int kTiles>
cudaError_t launch_small(const Args &a, int num_sms, cudaStream_t stream, const char **why)
{
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(k5_small<kTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kSmallSmem<kTiles>);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            configured[dev] = true;
    }
    const int ctas = ctas_for(kTiles, num_sms);
    *why = "tree attention launch";
    e = launch_pdl(k5_small<kTiles>, dim3((unsigned)ctas), dim3(kSmallThreads), kSmallSmem<kTiles>, stream, 1, a);
    if (e != cudaSuccess || a.partial == nullptr)
        return e;
    *why = "tree attention join launch";
    return launch_pdl(k5_join<16 * kTiles>, dim3((unsigned)ctas, 16 * kTiles / kJoinRows), dim3(kJoinThreads), 0, stream, 1, a);
}

}  // namespace

size_t tree_attention_workspace(int64_t rows, int32_t seqs, int32_t group, int num_sms)
{
    const int tiles = tiles_for(rows, seqs, group);
    const size_t slot = tiles == 1 ? kSlotFloats<16> : kSlotFloats<32>;
    return 2 * (size_t)ctas_for(tiles, num_sms) * slot * sizeof(float);
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
    return tiles_for(p.rows, p.seqs, p.group) == 1 ? launch_small<1>(a, num_sms, stream, why)
                                                   : launch_small<2>(a, num_sms, stream, why);
}

}  // namespace rc
