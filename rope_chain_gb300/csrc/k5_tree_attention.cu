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
// as a batch does.  Where units are fewer than CTAs and that is no longer, each
// is cut into equal parts instead, so that no CTA has to go from one to another
// (6 trees of 8 over 700 to 1405 keys: 20.8 us, cut anywhere 23.3; 9 of 6 with 16
// heads a KV head over 1900 to 3855: 21.0, 24.8), and short ones are not cut (36
// trees of 12 over 136 keys: 15.6 us, in equal ranges 34.6).  A unit that is cut
// leaves FP32 partials (output, m, sum) in the workspace, which a second kernel
// joins in key order (no atomics: the result does not depend on timing).
#include "rc_draft.cuh"
#include "rc_tcgen05.cuh"

#include <algorithm>
#include <cmath>

namespace rc {

__device__ unsigned int g_attention_faults;

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kKeyTile = 128;          // keys per step of a CTA
constexpr float kGrow = 8.0f;          // log2: growth of a row's maximum at which its output is rescaled

struct Args : TreeAttentionLaunch {
    float scale_log2;                  // scale * log2 e
    int32_t min_tiles;                 // fewest key tiles a CTA is given
    bool whole;                        // units are not cut
    int32_t change;                    // going to another unit, in key tiles' time
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

// How the units are cut.  Their slots, laid end to end, are shared out evenly.
//   most >= 1: a slot is a part of at most so many key tiles, and a CTA gets one
//              (or, uncut, as many units as another)
//   most == 0: a unit's slots are its key tiles and then `change` empty ones, for
//              the time that the change to it takes
template <int kRows> __device__ __forceinline__ int64_t slots_of(const Args &a, int b, int32_t most) {
    const Seq s = seq_of(a, b);
    const int kt = key_tiles(s);
    return (int64_t)row_tiles<kRows>(a, s) * a.kv_heads * (most > 0 ? (kt - 1) / most + 1 : kt + a.change);
}

// A quotient; division of 64 bits is some 100 instructions, of 32 bits 20.
__device__ __forceinline__ int64_t quotient(int64_t x, int32_t y) {
    return (x >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

struct Place {
    int32_t most;                      // see slots_of
    int64_t total;                     // slots of all units
    int32_t used;                      // CTAs that have some
    int64_t each;                      // total / used and the remainder
    int32_t rest;
    int64_t lo, hi;                    // this CTA's range
    // where CTA c's range begins: total * c / used
    __device__ __forceinline__ int64_t begin_of(int32_t c) const {
        return each * c + (uint32_t)((uint32_t)rest * (uint32_t)c) / (uint32_t)used;
    }
    int32_t b;                         // the sequence of `at`
    int64_t off;                       // `at` within the sequence's slots
};

// How many key tiles a part has at most, 0: a cut wherever it falls (slots_of).
// Parts of `most` tiles are at most tiles / most + units.  They are taken where a
// CTA gets fewer tiles so than slots otherwise, or hardly more than a change.
__device__ __forceinline__ int32_t most_of(const Args &a, int64_t tiles, int64_t units, int ctas) {
    if (units >= ctas)
        return 0;
    const int32_t room = ctas - (int32_t)units;
    const int64_t most = max((int64_t)a.min_tiles, quotient(tiles + room - 1, room));
    return most <= a.change + 2 || most * ctas <= tiles + a.change * units ? (int32_t)min(most, (int64_t)INT32_MAX) : 0;
}

// The range of CTA c of `ctas`, and where its first slot lies.  Called by all
// kThreads threads.  kParts: cut into parts where that is better (not in the small
// kernel: its start would take 0.7 us longer, one token over 500 keys 7.9 instead
// of 7.2 us, and few calls have fewer units than CTAs, 4 tokens over 3000 keys 14.0
// and 12.4).  Up to 32 sequences a lane takes one, and each warp finds the range
// by itself (3 trees of 13: 16.6 us, by the block 17.0); beyond, a thread takes a
// run of sequences, and the one whose run holds the slot walks it.
template <int kRows, int kThreads, bool kParts>
__device__ Place locate(const Args &a, int c, int ctas) {
    __shared__ int64_t warp_tiles[kParts ? kThreads / 32 : 1], warp_units[kParts ? kThreads / 32 : 1];
    __shared__ int64_t warp_sum[kThreads / 32];
    __shared__ int64_t found_off;
    __shared__ int32_t found_b;
    const bool alone = kParts && a.seqs <= 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int threads = alone ? 32 : kThreads, me = alone ? lane : (int)threadIdx.x;
    const int per = (a.seqs + threads - 1) / threads;
    const int b0 = min(me * per, a.seqs), b1 = min(b0 + per, a.seqs);
    Place p;
    p.most = a.whole ? INT32_MAX : 0;
    if (kParts && !a.whole && a.partial != nullptr) {
        int64_t tiles = 0, units = 0;
        for (int b = b0; b < b1; ++b) {
            const Seq s = seq_of(a, b);
            const int n = row_tiles<kRows>(a, s) * a.kv_heads;
            units += n;
            tiles += (int64_t)n * key_tiles(s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            tiles += __shfl_xor_sync(0xFFFFFFFFu, tiles, o);
            units += __shfl_xor_sync(0xFFFFFFFFu, units, o);
        }
        if (!alone) {
            if (lane == 0) {
                warp_tiles[kParts ? warp : 0] = tiles;
                warp_units[kParts ? warp : 0] = units;
            }
            __syncthreads();
            tiles = units = 0;
            for (int w = 0; w < kThreads / 32; ++w) {
                tiles += warp_tiles[kParts ? w : 0];
                units += warp_units[kParts ? w : 0];
            }
        }
        p.most = most_of(a, tiles, units, ctas);
    }
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += slots_of<kRows>(a, b, p.most);
    int64_t run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, run, o);
        if (lane >= o)
            run += v;
    }
    int64_t before = run - mine;
    if (alone) {
        p.total = __shfl_sync(0xFFFFFFFFu, run, 31);
    } else {
        if (lane == 31)
            warp_sum[warp] = run;
        __syncthreads();
        p.total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp)
                before += warp_sum[w];
            p.total += warp_sum[w];
        }
    }
    p.used = (int32_t)max((int64_t)1, min((int64_t)ctas, p.most > 0 ? p.total : quotient(p.total, a.min_tiles)));
    p.each = quotient(p.total, p.used);
    p.rest = (int32_t)(p.total - p.each * p.used);               // rest * c < used^2 < 2^32
    p.lo = c < p.used ? p.begin_of(c) : p.total;
    p.hi = c < p.used ? p.begin_of(c + 1) : p.total;
    p.b = 0;
    p.off = 0;
    if (p.lo >= p.hi)
        return p;                      // uniform
    const bool here = p.lo >= before && p.lo < before + mine;
    if (alone) {
        const int src = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
        p.b = src;
        p.off = p.lo - __shfl_sync(0xFFFFFFFFu, before, src);
        return p;
    }
    if (here) {
        int64_t off = p.lo - before;
        int b = b0;
        for (int64_t t; off >= (t = slots_of<kRows>(a, b, p.most)); ++b)
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
    int32_t parts;                     // of the unit, where it is cut into such
    int64_t begin;                     // the unit's first slot
    __device__ bool whole() const { return k0 == 0 && count == kt; }
};

// The pieces of a CTA's range, in order.
template <int kRows> struct Walk {
    int64_t pos, off, hi;
    int32_t b, most;
    __device__ explicit Walk(const Place &p) : pos(p.lo), off(p.off), hi(p.hi), b(p.b), most(p.most) {}
    __device__ bool next(const Args &a, Piece &u) {
        while (pos < hi) {
            u.s = seq_of(a, b);
            u.kt = key_tiles(u.s);
            const int rt = row_tiles<kRows>(a, u.s);
            u.parts = most > 0 ? (u.kt - 1) / most + 1 : 0;
            const int32_t slots = most > 0 ? u.parts : u.kt + a.change;
            const int64_t all = (int64_t)rt * a.kv_heads * slots;
            if (off >= all) {                           // the next sequence with rows
                off -= all;
                ++b;
                continue;
            }
            u.b = b;
            u.unit = (int32_t)quotient(off, slots);
            const int32_t slot = (int32_t)(off - (int64_t)u.unit * slots);
            u.h = u.unit / rt;
            u.tile = u.unit - u.h * rt;
            u.begin = pos - slot;
            if (most > 0) {
                u.k0 = (int32_t)quotient((int64_t)u.kt * slot, u.parts);
                u.count = (int32_t)quotient((int64_t)u.kt * (slot + 1), u.parts) - u.k0;
                ++pos;
                ++off;
                return true;
            }
            const int32_t here = (int32_t)min((int64_t)(slots - slot), hi - pos);
            u.k0 = slot;
            u.count = min(u.kt - slot, here);
            pos += here;
            off += here;
            if (u.count <= 0)
                continue;                               // empty slots only
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

// Logical key p's block, as the table has it, and with it the element offset of
// the key's row in the cache (-1 without a valid block).
__device__ __forceinline__ int32_t block_of(const Args &a, int b, int p) {
    return __ldg(a.block_table + b * a.table_stride + (uint32_t)p / (uint32_t)a.block_size);
}
__device__ __forceinline__ int64_t offset_in(const Args &a, int32_t blk, int h, int p) {
    const uint32_t bs = (uint32_t)a.block_size;
    if (blk < 0 || blk >= a.num_blocks)
        return -1;
    return (((int64_t)blk * a.kv_heads + h) * bs + (uint32_t)p % bs) * (2 * kHeadDim);
}

// The header of this CTA's part of a split unit.
template <int kRows>
__device__ void write_header(const Args &a, const Place &p, const Piece &u, bool unfinite) {
    Header h{0, u.b, u.unit, unfinite ? 1 : 0};
    if (u.k0 == 0 && p.most > 0) {
        h.last = (int32_t)blockIdx.x + u.parts - 1;
    } else if (u.k0 == 0) {
        const int64_t end = u.begin + u.kt;
        // the CTA of the unit's last tile, from an estimate
        int32_t last = min(p.used - 1, (int32_t)__fdividef((float)end * (float)p.used, (float)p.total));
        while (last + 1 < p.used && p.begin_of(last + 1) < end)
            ++last;
        while (p.begin_of(last) >= end)
            --last;
        h.last = last;
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
        const int64_t o = offset_in(a, block_of(a, b, s.ctx + j), h, s.ctx + j);
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
// Measured: one token over 131071 keys (8 KV heads, 268 MB) 51 us with the join,
// 5.2 TB/s; 64 tokens over 1025 to 2049 keys (204 MB) 43 us, 4.7 TB/s; the
// loads alone, without the products, 50 and 44 us before the changes of unit
// were counted.  One token over 500 keys 7.3 us: launch, lengths, Q and block
// numbers, then four tiles, one after the other.  Eight warps and two CTAs an SM
// (one token of 131071 keys 52.1 us; four warps and four CTAs 55.2).

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

// kRuns: blocks hold a multiple of 16 keys, so a chunk is 4 KiB in a row.
template <int kTiles, bool kRuns>
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

    const Place at = locate<kRows, kSmallThreads, false>(a, blockIdx.x, gridDim.x);
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
        // ref, limit: as in the wide kernel (a row's reference moves when a score
        // passes it by 2^8)
        float o[kTiles][8][4], ref[kTiles][2], limit[kTiles][2], sum[kTiles][2];
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                limit[m][e] = -INFINITY;
                ref[m][e] = sum[m][e] = 0.0f;
            }
#pragma unroll
            for (int n = 0; n < 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[m][n][e] = 0.0f;
        }
        bool unfinite = false;

        // Where chunks lie.  Block numbers are loaded well before they are looked
        // at (a warp that looks waits): with kRuns a lane has chunk j & ~31 +
        // lane, 32 chunks ahead, else a key of the next chunk.
        const int lane_key = kRuns ? lane * kKeyTile : lane & 15;
        auto first_key = [&](int j) { return (k0 + j) * kKeyTile + warp * kChunk; };
        auto table_entry = [&](int j) -> int32_t {          // for this lane's key at or after chunk j
            const int p = first_key(j) + lane_key;
            return j + (kRuns ? lane : 0) < count && p < s.keys ? block_of(a, b, p) : -1;
        };
        int32_t entry = table_entry(0);
        int64_t from = -1;
        auto place = [&](int j) {                           // this lane's row from `entry`
            const int p = first_key(j) + lane_key;
            const bool there = j + (kRuns ? lane : 0) < count && p < s.keys;
            from = there ? offset_in(a, entry, h, p) : -1;
            // once per block that is out of range: at its first key
            if (there && from < 0 && (kRuns || lane < 16) && unit == 0 && p % a.block_size == 0 && a.err != nullptr)
                atomicAdd(a.err, 1);
        };
        const uint32_t lane_at = ((lane >> 3) & 1) * (kChunkBytes / 2) + (lane >> 4) * 128;
        uint32_t swizzled[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            swizzled[i] = lane_at + i * 256 + (((lane & 7) ^ ((2 * i + (lane >> 4)) & 7)) << 4);
        auto issue = [&](int j, int st) {
            const uint32_t at = ring + st * kChunkBytes;
            if (kRuns) {
                if ((j & 31) == 0) {
                    place(j);
                    entry = table_entry(j + 32);
                }
                const int64_t first = __shfl_sync(0xFFFFFFFFu, from, j & 31);
                const int keys = first < 0 ? 0 : min(kChunk, s.keys - first_key(j));
                if (lane == 0)
                    s_real[warp][st] = (1u << keys) - 1u;
                const uint16_t *src = a.cache + (first < 0 ? 0 : first) + 8 * lane;
                if (keys == kChunk) {
#pragma unroll
                    for (int i = 0; i < kChunk / 2; ++i)
                        copy16_real(at + swizzled[i & 3] + (i >> 2) * 1024, src + i * (4 * kHeadDim));
                } else {
#pragma unroll
                    for (int i = 0; i < kChunk / 2; ++i)
                        copy16(at + swizzled[i & 3] + (i >> 2) * 1024, src + i * (4 * kHeadDim),
                               2 * i + (lane >> 4) < keys);
                }
            } else {
                place(j);
                entry = table_entry(j + 1);
                const uint32_t real = __ballot_sync(0xFFFFFFFFu, from >= 0) & 0xFFFFu;
                if (lane == 0)
                    s_real[warp][st] = real;
#pragma unroll
                for (int i = 0; i < kChunk / 2; ++i) {
                    const int64_t row = __shfl_sync(0xFFFFFFFFu, from, 2 * i + (lane >> 4));
                    copy16(at + swizzled[i & 3] + (i >> 2) * 1024,
                           a.cache + (row >= 0 ? row + 8 * (lane & 15) : 0), row >= 0);
                }
            }
        };
        // ldmatrix addresses within a stage: K by halves of 8 keys, V transposed
        uint32_t k_lane[4], v_lane[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int kr = (lane >> 4) * 8 + (lane & 7), vr = ((lane >> 3) & 1) * 8 + (lane & 7);
            k_lane[k] = ring + kr * 128 + (((2 * k + ((lane >> 3) & 1)) ^ (kr & 7)) << 4);
            v_lane[k] = ring + kChunkBytes / 2 + vr * 128 + (((2 * k + (lane >> 4)) ^ (vr & 7)) << 4);
        }
#pragma unroll
        for (int j = 0; j < kStages - 1; ++j) {
            if (j < count)
                issue(j, j);
            copy_commit();
        }
        int st = 0, st_in = kStages - 1;                    // stages of chunks j and j + kStages - 1
        for (int j = 0; j < count; ++j) {
            copy_wait<kStages - 2>();
            __syncwarp();
            if (j + kStages - 1 < count)
                issue(j + kStages - 1, st_in);
            copy_commit();
            st_in = st;
            const uint32_t at = st * kChunkBytes;
            const int p0 = first_key(j);
            const uint32_t real = s_real[warp][st];
            st = st + 1 == kStages ? 0 : st + 1;
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
                load4(kf, k_lane[k] + at);
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
                    now[m][e] = fmaxf(fmaxf(t[m][0][2 * e], t[m][0][2 * e + 1]),
                                      fmaxf(t[m][1][2 * e], t[m][1][2 * e + 1])) * a.scale_log2;
                    grew |= now[m][e] > limit[m][e];
                }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = now[m][e];
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
                        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
                        if (x > limit[m][e]) {
                            const float shrink = limit[m][e] == -INFINITY ? 0.0f : ex2(-ref[m][e] - x);
                            ref[m][e] = -x;
                            limit[m][e] = x + kGrow;
                            sum[m][e] *= shrink;
#pragma unroll
                            for (int n = 0; n < 8; ++n) {
                                o[m][n][2 * e] *= shrink;
                                o[m][n][2 * e + 1] *= shrink;
                            }
                        }
                    }
            }
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float part0 = 0.0f, part1 = 0.0f;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float &x0 = t[m][n][2 * e], &x1 = t[m][n][2 * e + 1];
                        fma2_rn(x0, x1, a.scale_log2, a.scale_log2, ref[m][e], ref[m][e]);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        add2_rn(part0, part1, x0, x1);
                    }
                    sum[m][e] += part0 + part1;
                }
                pf[m][0] = pack_bf16x2(t[m][0][0], t[m][0][1]);
                pf[m][1] = pack_bf16x2(t[m][0][2], t[m][0][3]);
                pf[m][2] = pack_bf16x2(t[m][1][0], t[m][1][1]);
                pf[m][3] = pack_bf16x2(t[m][1][2], t[m][1][3]);
            }
#pragma unroll
            for (int n = 0; n < 8; n += 2) {
                uint32_t vf[4];
                load4_t(vf, v_lane[n / 2] + at);
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
                    s_max[warp][r] = limit[m][e] == -INFINITY ? -INFINITY : -ref[m][e];
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
                const float f = limit[m][e] == -INFINITY ? 0.0f : ex2(-ref[m][e] - now);
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
// From 33 rows per unit on the products are the bound, and the work goes
// to tcgen05: kQ row tiles of 128 rows share each key tile of 128 keys.  A row
// tile's S = Q K^T lands in TMEM (128 columns), the weights go back to TMEM as
// bf16 (64 columns), from where they are the A operand of O += P V, and O stays
// in TMEM (64 columns): 256 columns per row tile, two row tiles per SM (kQ = 2,
// or two CTAs of kQ = 1).  Eight softmax warps per row tile, each with 16 of
// its rows and whole key tiles (a quad of lanes per row, as in m16n8 tiles:
// the maximum takes two shuffles): 16 warps per SM hide one another's
// latencies, where 8 warps of a row per thread ran at a third of the issue
// rate.  A row's reference (what its maximum is in a running softmax) is that of
// an earlier tile until a score passes it by more than 2^8: weights above 1 are
// harmless, FP32 and bf16 having the range.  So a tile's maximum needs no
// shuffles, only a vote on whether a lane saw more, and O is rescaled rarely, by
// the rows' own warp.
//   kQ loader warps  K and V tiles of 16 KiB by TMA, in boxes of the largest
//                    power of two of keys that divides a block (8 to 128),
//                    each box's block looked up in the table by its own lane
//   kQ MMA warps     one per row tile: the next S as soon as the softmax has
//                    the last one in registers, then O when the weights are
//                    there.  One warp for both tiles was the bottleneck: some
//                    100 cycles per product to issue, 1200 per tile and round
// Per 256 rows x 128 keys the exponentials need 1024 cycles of an SM (32 per
// cycle), the products as many at full rate; products of 64 columns (O) run at
// about half of it, 1536 in all.
// Measured: 8 trees of 64 tokens over 32768 keys (64 query and 8 KV heads, 273
// GFLOP) 290 to 307 us by the box, 0.89 to 0.94 PFLOP/s, 2700 cycles per 256 x 128
// (in blocks of 16 keys; 273 us in blocks of 128): the steps of the two row tiles,
// products, softmax and weights, one after the other; tensor pipe 42 %, issue slots
// 60 %.  16 trees of 16 over 8192 keys (273 MB) 71 us, 3.8 TB/s: 44 us at 6.2 TB/s
// between a start of 9 us (launch, lengths, Q, first tile) and changes of unit and
// the join of 18.  Two CTAs an SM leave kQ = 1 96 registers a thread, of which it
// spills 51 (204 bytes stored, 572 loaded); kQ = 2 spills three.
// Key tiles that hold drafted keys, or the end, take a masked path; there the
// V rows past the end are zeroed and what is infinite or NaN in a drafted one
// is taken out (see add_unfinite).  Every wait is bounded; on timeout a sticky
// fault bit is raised and all roles leave.

enum : unsigned { kFaultLoad = 1u, kFaultMma = 2u, kFaultSoftmax = 4u, kFaultDrain = 8u };

constexpr uint32_t kTileBytes = kKeyTile * kHeadDim * 2;           // K or V of a step, Q of a tile: 16 KiB
template <int kQ> constexpr int kSoftmaxWarps = 8 * kQ;
// A warp's boxes are issued one by one, at some 130 cycles each.  With two row
// tiles one warp loads K and another V: 293 us instead of 323 for 8 trees of 64
// tokens over 32768 keys (512 rows a KV head, blocks of 16).  With one row tile a
// single warp loads both, as an eleventh warp would cost the SM its second CTA:
// 16 trees of 16 over 8192 keys take 73 us, with two loaders 84.
template <int kQ> constexpr int kLoaders = kQ;
template <int kQ> constexpr int kWideThreads = 32 * (kSoftmaxWarps<kQ> + kQ + kLoaders<kQ>);
template <int kQ> constexpr int kWideStages = kQ == 1 ? 3 : 5;
template <int kQ> constexpr uint32_t kTmemCols = 256u * kQ;        // per row tile: S 128, P 64, O 64 columns
constexpr uint32_t kPCol = 128u, kOCol = 192u;
template <int kQ> constexpr size_t kWideSmem = kQ * kTileBytes + kWideStages<kQ> * 2 * kTileBytes;

// Keeps x in local memory: what is read at a piece's ends only would otherwise
// crowd the scores out of the registers.  Used with two row tiles (8 trees of 64
// tokens over 32768 keys in blocks of 128: 273 us, without 291; in blocks of 16,
// where the loads bound, 293 either way), not with one (16 trees of 16 over 8192
// keys: 73 us, with it 76).
template <typename T> __device__ __forceinline__ void in_memory(T &x) { asm volatile("" ::"l"(&x) : "memory"); }

// The slow half of a wait: up to kWaitNs from its first look at the timer, or
// until a fault has been raised; raises `fault` if the phase does not complete.
__device__ __noinline__ bool wait_slowly(uint32_t bar, uint32_t parity, unsigned fault) {
    const unsigned long long t0 = globaltimer();
    for (uint32_t it = 0;; ++it) {
        if (mbar_try(bar, parity))
            return true;
        if ((it & 31u) == 31u &&
            (*reinterpret_cast<volatile unsigned int *>(&g_attention_faults) != 0u || globaltimer() - t0 > kWaitNs)) {
            atomicOr(&g_attention_faults, fault);
            return false;
        }
    }
}
// Wait for a phase: a few tries in line (each suspended by the hardware for a
// while), then slowly; false once it has timed out or a fault has been raised.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, unsigned fault) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b32 i;\n\t"
                 "mov.b32 i, 0;\n"
                 "again_%=:\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
                 "@p bra done_%=;\n\t"
                 "add.u32 i, i, 1;\n\t"
                 "setp.lt.u32 q, i, 64;\n\t"
                 "@q bra again_%=;\n"
                 "done_%=:\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0u || wait_slowly(bar, parity, fault);
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int col, int off, int h, int blk,
                                        uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(off), "r"(h), "r"(blk), "r"(bar)
                 : "memory");
}
// Shared-memory descriptors (smem_desc_sw128) as their low words, so that the
// next 16 columns or keys are one addition away; the high word is a constant.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) {
    return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
// D[tmem] (+)= A[smem] x B[smem], and with A in TMEM
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alow, uint32_t blow, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
                 ::"r"(d), "r"(alow), "r"(blow), "r"(idesc), "r"(acc), "r"(kDescHigh) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t blow, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "mov.b64 b, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "r"(blow), "r"(idesc), "r"(acc), "r"(kDescHigh) : "memory");
}
// 64 columns of 16 lanes (FP32): lane l's values of rows l / 4 (r[4c], r[4c + 1])
// and l / 4 + 8 (r[4c + 2], r[4c + 3]) are columns 8c + 2 (l % 4) and the next.
// Complete after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld_rows(uint32_t at, float *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]),
          "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]),
          "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]),
          "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
        : "r"(at));
}
// 16 columns of the same kind, load and store.
__device__ __forceinline__ void tmem_ld_rows16(uint32_t at, float *r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(at));
}
__device__ __forceinline__ void tmem_st_rows16(uint32_t at, const float *r) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(at), "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}
// 32 columns of 16 lanes: w[2c] row l / 4, w[2c + 1] row l / 4 + 8, column
// 4c + l % 4 (pairs of bf16: columns 8c + 2 (l % 4) and the next of P).
__device__ __forceinline__ void tmem_st_pairs(uint32_t at, const uint32_t *w) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
        "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The values of a load, to be used no earlier than here (after the wait).
__device__ __forceinline__ void loaded8(float *r) {
    asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

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
    constexpr int kMmaWarp = kSoftmaxWarps<kQ>, kLoadWarp = kMmaWarp + kQ;
    extern __shared__ __align__(1024) uint8_t smem_wide[];
    const uint32_t sQ = smem_u32(smem_wide), sK = sQ + kQ * kTileBytes;     // a stage: K, then V
    __shared__ uint64_t bars[2 * kStages + 6 * kQ];
    // by piece modulo 8: a row tile is never more than kStages + 1 pieces ahead
    // of another, whose products free its stages
    __shared__ uint32_t s_tmem, s_skip, s_bad[kStages], s_unfinite[8];
    static_assert(kStages + 1 < 8, "pieces in flight");
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * kStages, q_ready0 = empty0 + 8u * kStages;
    const uint32_t s_full0 = q_ready0 + 8u * kQ, s_free0 = s_full0 + 8u * kQ, p_ready0 = s_free0 + 8u * kQ;
    const uint32_t o_done0 = p_ready0 + 8u * kQ, drain0 = o_done0 + 8u * kQ;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full0 + 8u * i, kLoaders<kQ>);
            mbar_init(empty0 + 8u * i, kQ);
        }
        for (int t = 0; t < kQ; ++t) {
            mbar_init(q_ready0 + 8u * t, 256);
            mbar_init(s_full0 + 8u * t, 1);
            mbar_init(s_free0 + 8u * t, 8);
            mbar_init(p_ready0 + 8u * t, 256);
            mbar_init(o_done0 + 8u * t, 1);
            mbar_init(drain0 + 8u * t, 1);
        }
        for (int i = 0; i < 8; ++i)
            s_unfinite[i] = 0u;
        // one decision for the CTA: a raised fault skips the work
        s_skip = *reinterpret_cast<volatile unsigned int *>(&g_attention_faults);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_tensormap(&map);
    }
    pdl_wait();
    // TMEM only now: two CTAs (kQ = 1) fit on an SM, and one that held its columns
    // while it waited for the previous kernel could keep them from a CTA of that
    // kernel which has still to allocate.  (The lengths are read meanwhile.)
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&s_tmem)), "r"(kTmemCols<kQ>) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    Place at = locate<kRows, kThreads, true>(a, blockIdx.x, gridDim.x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;                       // row tile t: S, P, O from column 256 t
    if (a.partial != nullptr && threadIdx.x == 0)
        reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + 1))->last = 0;
    Walk<kRows> walk(at);
    if (s_skip != 0u)
        walk.hi = walk.pos;
    Piece u;
    if constexpr (kQ == 2) {
        in_memory(at);
        in_memory(walk);
        in_memory(u);
    }
    uint32_t n = 0;                                     // key tiles of earlier pieces
    uint32_t piece = 0;

    if (warp >= kLoadWarp) {
        const bool keys = warp == kLoadWarp, values = kLoaders<kQ> == 1 || !keys;
        const int boxes = kKeyTile / box;               // <= 16
        bool fine = true;
        while (fine && walk.next(a, u)) {
            const Seq &s = u.s;
            // this lane's box of tile j: its block
            auto look_up = [&](int j) -> int {
                const int p = (u.k0 + j) * kKeyTile + lane * box;
                return j < u.count && lane < boxes && p < s.keys
                           ? block_of(a, u.b, p) : 0;
            };
            int blk = look_up(0);
            for (int j = 0; j < u.count; ++j, ++n) {
                const uint32_t st = n % kStages, full = full0 + 8u * st;
                const int p = (u.k0 + j) * kKeyTile + lane * box;
                const bool mine = lane < boxes && p < s.keys;
                const int off = mine ? (int)((uint32_t)p % (uint32_t)a.block_size) : 0;
                const bool bad = mine && (blk < 0 || blk >= a.num_blocks);
                if (bad && keys && u.unit == 0 && off == 0 && a.err != nullptr)
                    atomicAdd(a.err, 1);                // once per block: at its first key
                fine = wait_phase(empty0 + 8u * st, ((n / kStages) & 1u) ^ 1u, kFaultLoad);
                fine = __all_sync(0xFFFFFFFFu, fine);
                if (!fine)
                    break;
                const uint32_t bads = __ballot_sync(0xFFFFFFFFu, bad), loads = __ballot_sync(0xFFFFFFFFu, mine);
                if (lane == 0) {
                    if (keys)
                        s_bad[st] = bads;
                    mbar_expect_tx(full, (uint32_t)__popc(loads) * box * (256u / kLoaders<kQ>));
                }
                __syncwarp();
                if (mine) {
                    // a block out of range reads zeros: one past the last
                    const int from = bad ? a.num_blocks : blk;
                    const uint32_t dst = sK + st * (2 * kTileBytes) + (uint32_t)(lane * box) * 128u;
                    if (keys)
                        tma_box(dst, &map, 0, off, u.h, from, full);
                    if (values)
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
    } else if (warp >= kMmaWarp) {
        if (lane == 0) {
            const int t = warp - kMmaWarp;
            constexpr uint32_t idesc_s = make_idesc(128, kKeyTile, false), idesc_o = make_idesc(128, kHeadDim, true);
            const uint32_t tS = tmem + 256u * t, tP = tS + kPCol, tO = tS + kOCol;
            const uint32_t q = desc_low(sQ + t * kTileBytes, 16u);
            const uint32_t k0 = desc_low(sK, 16u), v0 = desc_low(sK + kTileBytes, 8192u);
            const uint32_t s_full = s_full0 + 8u * t, s_free = s_free0 + 8u * t, p_ready = p_ready0 + 8u * t;
            const uint32_t o_done = o_done0 + 8u * t;
            // the scores of key tile i, once their columns are free
            auto scores = [&](uint32_t i) {
                const uint32_t st = i % kStages;
                if (!wait_phase(full0 + 8u * st, (i / kStages) & 1u, kFaultMma) ||
                    (i > 0 && !wait_phase(s_free, (i - 1) & 1u, kFaultMma)))
                    return false;
                tc_fence_after();
                const uint32_t k = k0 + st * (2 * kTileBytes >> 4);
#pragma unroll
                for (uint32_t kk = 0; kk < kHeadDim / 16; ++kk)
                    mma_ss(tS, q + 2u * kk, k + 2u * kk, idesc_s, kk);
                mma_commit(s_full);
                return true;
            };
            bool fine = true;
            while (fine && walk.next(a, u)) {
                fine = wait_phase(q_ready0 + 8u * t, piece & 1u, kFaultMma) && scores(n);
                for (int j = 0; j < u.count && fine; ++j, ++n) {
                    if (j + 1 < u.count)
                        fine = scores(n + 1);
                    fine = fine && wait_phase(p_ready, n & 1u, kFaultMma);
                    if (!fine)
                        break;
                    tc_fence_after();
                    const uint32_t st = n % kStages, v = v0 + st * (2 * kTileBytes >> 4);
                    mma_ts(tO, tP, v, idesc_o, j != 0);
#pragma unroll
                    for (uint32_t kk = 1; kk < kKeyTile / 16; ++kk)
                        mma_ts(tO, tP + 8u * kk, v + kk * (2048u >> 4), idesc_o, 1u);
                    mma_commit(o_done);
                    mma_commit(empty0 + 8u * st);
                }
                ++piece;
            }
            mma_commit(drain0 + 8u * t);
            if (!mbar_wait_own(drain0 + 8u * t, 0u))
                atomicOr(&g_attention_faults, kFaultDrain);
        }
        __syncwarp();
    } else {
        // warp w of a row tile: rows 32 (w % 4) + 16 (w / 4) .. + 15 (a warp
        // reaches the TMEM lanes of its number modulo 4); this lane's are
        // l / 4 and l / 4 + 8 of them
        const int t = warp >> 3, w8 = warp & 7;
        const int first = 32 * (w8 & 3) + 16 * (w8 >> 2);
        const uint32_t lanes = (uint32_t)first << 16;
        const uint32_t tS = tmem + lanes + 256u * t, tP = tS + kPCol, tO = tS + kOCol;
        const uint32_t s_full = s_full0 + 8u * t, p_ready = p_ready0 + 8u * t, o_done = o_done0 + 8u * t;
        // (a wait that fails has raised a fault: the tiles are gone through all
        // the same, so that every barrier sees its arrivals)
        while (walk.next(a, u)) {
            const Seq &s = u.s;
            {
                // Q: thread i of the tile's 256 takes half of row i / 2
                const int i = threadIdx.x & 255, r = i >> 1, half = i & 1;
                const int row = u.tile * kRows + 128 * t + r, node = row / a.group;
                const uint4 *src = reinterpret_cast<const uint4 *>(
                    a.q + (int64_t)(s.r0 + node) * a.q_row_stride + (u.h * a.group + row - node * a.group) * kHeadDim) + 4 * half;
                const uint32_t dst = sQ + (uint32_t)t * kTileBytes + (uint32_t)r * 128u;
                uint4 w[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    w[c] = node < s.n ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    st_shared_v4(dst + (uint32_t)(((4 * half + c) ^ (r & 7)) << 4), w[c]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive_local(q_ready0 + 8u * t);
            }
            int node[2];
            // of each row: minus the reference (log2), the maximum that asks for
            // another (-inf: none seen yet), this lane's sum
            float ref[2], limit[2], sum[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = (u.tile * kRows + 128 * t + first + (lane >> 2) + 8 * e) / a.group;
                node[e] = i < s.n ? i : -1;
                ref[e] = sum[e] = 0.0f;
                limit[e] = -INFINITY;
            }
            const int count = u.count, ctx = s.ctx;
            int p0 = u.k0 * kKeyTile;
            for (int j = 0; j < count; ++j, ++n, p0 += kKeyTile) {
                wait_phase(s_full, n & 1u, kFaultSoftmax);
                __syncwarp();
                tc_fence_after();
                const uint32_t st = n % kStages;
                const uint32_t bads = *reinterpret_cast<volatile uint32_t *>(&s_bad[st]);
                // y[32h + 4c + 2e + f]: row e, key 64h + 8c + 2 (l % 4) + f
                float y[64];
                tmem_ld_rows(tS, y);
                tmem_ld_rows(tS + 64u, y + 32);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    loaded8(y + 8 * c);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_local(s_free0 + 8u * t);
                if (p0 + kKeyTile > ctx || bads != 0u) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t out = 0u;              // keys of blocks out of range
                        for (int k = 0; bads != 0u && k < 32; ++k)
                            out |= ((bads >> ((32 * c + k) / box)) & 1u) << k;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t see = (seen32(a, s, node[e], p0 + 32 * c) & ~out) >> (2 * (lane & 3));
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int f = 0; f < 2; ++f)
                                    if (!((see >> (8 * k + f)) & 1u))
                                        y[4 * (4 * c + k) + 2 * e + f] = -INFINITY;
                        }
                    }
                    // the tile's V: zeros past the end, and in place of what is
                    // not finite in drafted keys.  Every row tile looks at all
                    // of it; one that finds such a value says so (the number of
                    // the piece) before it takes it out, so that the others,
                    // who may see the zero, see the word too.
                    wait_phase(full0 + 8u * st, (n / kStages) & 1u, kFaultSoftmax);    // complete: seen through S
                    const uint32_t v = sK + st * (2 * kTileBytes) + kTileBytes;
                    for (int i = threadIdx.x & 255; i < kKeyTile * 8; i += 256) {
                        const int key = p0 + (i >> 3);
                        if (key < s.ctx)
                            continue;
                        const uint32_t chunk = v + 16u * i;
                        uint4 w = make_uint4(0, 0, 0, 0);
                        bool write = true;
                        if (key < s.keys) {
                            w = ld_shared_v4(chunk);
                            write = finite_only(w.x, true, true);
                            write |= finite_only(w.y, true, true);
                            write |= finite_only(w.z, true, true);
                            write |= finite_only(w.w, true, true);
                            if (write) {
                                *reinterpret_cast<volatile uint32_t *>(&s_unfinite[piece & 7u]) = piece + 1u;
                                __threadfence_block();
                            }
                        }
                        if (write)
                            st_shared_v4(chunk, w);
                    }
                    __threadfence_block();
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                // this lane's maxima: past a row's reference by more than 2^8
                // (or the first that it sees), the row takes a new one
                float m[2];
                bool grew = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float m0 = fmaxf(y[2 * e], y[2 * e + 1]), m1 = fmaxf(y[4 + 2 * e], y[5 + 2 * e]);
#pragma unroll
                    for (int c = 2; c < 16; c += 2) {
                        m0 = max3(m0, y[4 * c + 2 * e], y[4 * c + 2 * e + 1]);
                        m1 = max3(m1, y[4 * c + 4 + 2 * e], y[4 * c + 5 + 2 * e]);
                    }
                    m[e] = fmaxf(m0, m1) * a.scale_log2;
                    grew |= m[e] > limit[e];
                }
                if (__any_sync(0xFFFFFFFFu, grew)) {
                    if (n > 0)                          // O holds the products of the tiles before
                        wait_phase(o_done, (n - 1) & 1u, kFaultSoftmax);
                    tc_fence_after();
                    float shrink[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        m[e] = fmaxf(m[e], __shfl_xor_sync(0xFFFFFFFFu, m[e], 1));
                        m[e] = fmaxf(m[e], __shfl_xor_sync(0xFFFFFFFFu, m[e], 2));
                        shrink[e] = 1.0f;
                        if (m[e] > limit[e]) {
                            shrink[e] = limit[e] == -INFINITY ? 0.0f : ex2(-ref[e] - m[e]);
                            sum[e] *= shrink[e];
                            ref[e] = -m[e];
                            limit[e] = m[e] + kGrow;
                        }
                    }
                    if (j > 0) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
                            float o[8];
                            tmem_ld_rows16(tO + 16u * c, o);
                            tmem_wait_ld();
                            loaded8(o);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                o[k] *= shrink[(k >> 1) & 1];
                            tmem_st_rows16(tO + 16u * c, o);
                        }
                    }
                }
                float part[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[16];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float e0 = y[32 * h + 4 * c + 2 * e], e1 = y[32 * h + 4 * c + 2 * e + 1];
                            fma2_rn(e0, e1, a.scale_log2, a.scale_log2, ref[e], ref[e]);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            add2_rn(part[e][0], part[e][1], e0, e1);
                            w[2 * c + e] = pack_bf16x2(e0, e1);
                        }
                    if (h == 0 && n > 0) {
                        // the products of the last tile have read P
                        wait_phase(o_done, (n - 1) & 1u, kFaultSoftmax);
                        tc_fence_after();
                    }
                    tmem_st_pairs(tP + 32u * h, w);
                }
                sum[0] += part[0][0] + part[0][1];
                sum[1] += part[1][0] + part[1][1];
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive_local(p_ready);
            }
            // the rows' outputs
            wait_phase(o_done, (n - 1) & 1u, kFaultSoftmax);
            __syncwarp();
            tc_fence_after();
            float o[32];                                // o[4c + 2e + f]: row e, column 8c + 2 (l % 4) + f
            tmem_ld_rows(tO, o);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 4; ++c)
                loaded8(o + 8 * c);
            tc_fence_before();
            const bool unfinite = *reinterpret_cast<volatile uint32_t *>(&s_unfinite[piece & 7u]) == piece + 1u;
            const bool whole = u.whole();
            float *slot = whole ? nullptr : slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + (u.k0 == 0 ? 1 : 0));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 128 * t + first + (lane >> 2) + 8 * e, row = u.tile * kRows + r, i = node[e];
                float total = sum[e];
                total += __shfl_xor_sync(0xFFFFFFFFu, total, 1);
                total += __shfl_xor_sync(0xFFFFFFFFu, total, 2);
                const float top = limit[e] == -INFINITY ? -INFINITY : -ref[e];
                if (!whole) {
                    float *dst = slot + kSlotOut<kRows> + r * kHeadDim + 2 * (lane & 3);
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<float2 *>(dst + 8 * c) = make_float2(o[4 * c + 2 * e], o[4 * c + 2 * e + 1]);
                    if ((lane & 3) == 0) {
                        slot[kSlotMax<kRows> + r] = top;
                        slot[kSlotSum<kRows> + r] = total;
                    }
                } else if (i >= 0) {
                    const int head = u.h * a.group + row - i * a.group, col = 2 * (lane & 3);
                    const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
                    uint16_t *dst = a.out + (int64_t)(s.r0 + i) * a.out_row_stride + head * kHeadDim + col;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        float lo = o[4 * c + 2 * e], hi = o[4 * c + 2 * e + 1];
                        if (unfinite) {
                            lo = add_unfinite(a, s, u.b, u.h, i, 8 * c + col, lo);
                            hi = add_unfinite(a, s, u.b, u.h, i, 8 * c + col + 1, hi);
                        }
                        *reinterpret_cast<uint32_t *>(dst + 8 * c) = pack_bf16x2(lo * inv, hi * inv);
                    }
                    if ((lane & 3) == 0 && a.lse != nullptr)
                        a.lse[(int64_t)(s.r0 + i) * (a.kv_heads * a.group) + head] =
                            total == 0.0f ? -INFINITY : __fmaf_rn(top, kLn2, logf(total));
                }
            }
            if (threadIdx.x == 0) {
                if (!whole)
                    write_header<kRows>(a, at, u, unfinite);
                else if (u.unit == 0 && a.err != nullptr && (int64_t)max(__ldg(a.context_len + u.b), 0) + s.n > s.keys)
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
// Block (c, y) joins rows of the unit that CTA c began and did not end: its own
// part and those of the CTAs after it, in key order.  A thread has four columns
// of a row; with few rows (kRows <= 32: units cut into many parts) four groups
// of threads take every fourth part each and are joined in order at the end.  A
// thread loads eight parts' maxima, sums and columns at once, so that the few
// parts of a unit of many rows cost one latency (one part at a time: 27 us for 16
// trees of 16 tokens, 42 for 8 of 64; now about 5 behind the kernel that wrote
// them, of which launch and headers are 1.3).
constexpr int kJoinThreads = 256;
template <int kRows> constexpr int kJoinRows = kRows <= 32 ? 4 : 16;

template <int kRows>
__global__ void __launch_bounds__(kJoinThreads)
k5_join(const __grid_constant__ Args a)
{
    constexpr int kGroups = kJoinThreads / (16 * kJoinRows<kRows>), kBatch = 8;
    __shared__ float4 s_out[kGroups][16 * kJoinRows<kRows>];
    __shared__ float s_top[kGroups][kJoinRows<kRows>], s_sum[kGroups][kJoinRows<kRows>];
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
    const int r0 = blockIdx.y * kJoinRows<kRows>, parts = hd.last - c + 1;
    if (threadIdx.x == 0 && blockIdx.y == 0 && hd.unit == 0 && a.err != nullptr &&
        (int64_t)max(__ldg(a.context_len + hd.b), 0) + s.n > s.keys)
        atomicAdd(a.err, 1);
    if (tile * kRows + r0 >= s.n * a.group)
        return;
    const int group = threadIdx.x / (16 * kJoinRows<kRows>), col = (threadIdx.x & 15) * 4;
    const int r = (threadIdx.x >> 4) % kJoinRows<kRows>;
    int unfinite = 0;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float top = -INFINITY, total = 0.0f;
    for (int k0 = group; k0 < parts; k0 += kBatch * kGroups) {
        float m[kBatch], l[kBatch];
        float4 y[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = k0 + i * kGroups;
            m[i] = -INFINITY;
            l[i] = 0.0f;
            y[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (k < parts) {
                const float *part = k == 0 ? own : slot_of<kRows>(a, 2 * (int64_t)(c + k));
                m[i] = part[kSlotMax<kRows> + r0 + r];
                l[i] = part[kSlotSum<kRows> + r0 + r];
                y[i] = *reinterpret_cast<const float4 *>(part + kSlotOut<kRows> + (r0 + r) * kHeadDim + col);
                unfinite |= reinterpret_cast<const Header *>(part)->unfinite;
            }
        }
        float now = top;
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            now = fmaxf(now, m[i]);
        const float ref = now == -INFINITY ? 0.0f : now, shrink = ex2(top - ref);
        top = now;
        total *= shrink;
        x.x *= shrink;
        x.y *= shrink;
        x.z *= shrink;
        x.w *= shrink;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (k0 + i * kGroups >= parts)
                break;
            const float f = ex2(m[i] - ref);
            total = __fmaf_rn(l[i], f, total);
            x.x = __fmaf_rn(y[i].x, f, x.x);
            x.y = __fmaf_rn(y[i].y, f, x.y);
            x.z = __fmaf_rn(y[i].z, f, x.z);
            x.w = __fmaf_rn(y[i].w, f, x.w);
        }
    }
    if (kGroups > 1) {
        s_out[group][threadIdx.x % (16 * kJoinRows<kRows>)] = x;
        if (col == 0) {
            s_top[group][r] = top;
            s_sum[group][r] = total;
        }
        unfinite = __syncthreads_or(unfinite);
        if (group > 0)
            return;
        float now = top;
#pragma unroll
        for (int g = 1; g < kGroups; ++g)
            now = fmaxf(now, s_top[g][r]);
        const float ref = now == -INFINITY ? 0.0f : now, f0 = ex2(top - ref);
        top = now;
        total *= f0;
        x.x *= f0;
        x.y *= f0;
        x.z *= f0;
        x.w *= f0;
#pragma unroll
        for (int g = 1; g < kGroups; ++g) {
            const float f = ex2(s_top[g][r] - ref);
            const float4 y = s_out[g][threadIdx.x];
            total = __fmaf_rn(s_sum[g][r], f, total);
            x.x = __fmaf_rn(y.x, f, x.x);
            x.y = __fmaf_rn(y.y, f, x.y);
            x.z = __fmaf_rn(y.z, f, x.z);
            x.w = __fmaf_rn(y.w, f, x.w);
        }
    }
    const int row = tile * kRows + r0 + r, i = row / a.group;
    if (i >= s.n)
        return;
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
// known on the host; any kernel is right for any unit).  8 sequences over 4096
// keys, us:
//   up to 16 rows   k5_small<1>: 21.2 at 16 rows, k5_small<2> 23.5
//   up to 32        k5_small<2>: 26.5 at 32, k5_wide<1> 29.6; at 40 31.3 and 29.5
//   up to 128       k5_wide<1>: 32.5 at 128, k5_wide<2> 38.5; at 160 44.1 and 40.1
//   beyond          k5_wide<2>: two row tiles share each key tile
// Batches that mix them: 63 single tokens and a tree of 64 over 2000 keys 57 us (64
// single tokens 51, the tree alone 25).
// The wide kernel's TMA boxes need blocks of a multiple of 8 keys; other block
// sizes stay with k5_small<2>.
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
    return launch_pdl(k5_join<kRows>, dim3((unsigned)ctas, kRows / kJoinRows<kRows>), dim3(kJoinThreads), 0, stream, 1, a);
}

template <int kTiles, bool kRuns>
cudaError_t launch_small(const Args &a, int ctas, cudaStream_t stream, const char **why)
{
    static bool configured[64] = {};
    cudaError_t e = allow_smem(k5_small<kTiles, kRuns>, kSmallSmem<kTiles>, configured);
    if (e != cudaSuccess)
        return e;
    *why = "tree attention launch";
    e = launch_pdl(k5_small<kTiles, kRuns>, dim3((unsigned)ctas), dim3(kSmallThreads), kSmallSmem<kTiles>, stream, 1, a);
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
    // For whichever block size the cache has (a multiple of 8 gives the variant of
    // most rows) and for any call of fewer rows or more sequences: the variants of
    // smaller tiles have twice the CTAs, and so may take a few headers more.
    const Variant last = variant_for(rows, seqs, group, 8);
    size_t most = 0;
    for (const Variant v : {kSmall16, kSmall32, kWide128, kWide256})
        if (v <= last)
            most = std::max(most, 2 * (size_t)ctas_of(v, num_sms) * slot_floats(v) * sizeof(float));
    return most;
}

cudaError_t launch_tree_attention(const TreeAttentionLaunch &p, int num_sms, cudaStream_t stream,
                                  const char **why)
{
    Args a{};
    static_cast<TreeAttentionLaunch &>(a) = p;
    a.scale_log2 = p.scale * kLog2e;
    const Variant v = variant_for(p.rows, p.seqs, p.group, p.block_size);
    // (3 trees of 13 over 1500 keys, in equal ranges: 15.3 us with two tiles a CTA at
    // least, 19.9 with four, 18.3 with one)
    a.min_tiles = 2;
    const int64_t unit_rows = v == kSmall16 ? 16 : v == kSmall32 ? 32 : v == kWide128 ? 128 : 256;
    const int64_t units = (p.rows * p.group / unit_rows + p.seqs) * p.kv_heads;      // at most
    // Units of at most so many tiles are not worth a cut and a join: one token over
    // 300 keys 6.9 us (cut 11.2), 30 single tokens over 450 to 900 15.0 (19.2); a
    // tile of many rows takes longer, 16 trees of 16 over 480 15.7 (23.2), but 3 of
    // 13 over 900 17.6 whole and 16.1 cut.  With several units a CTA equal ranges
    // of tiles spread ragged lengths better (256 tokens over 450 to 900: 77.4 whole,
    // 73.5 cut; 64 25.9 and 27.8).
    const int whole = v == kWide128 || v == kWide256 || units > 3 * ctas_of(v, num_sms) ? 4 : 8;
    if ((int64_t)p.table_width * p.block_size <= whole * kKeyTile) {
        a.partial = nullptr;
        a.whole = true;
    }
    // as many CTAs as fill the GPU, or as the block table lets have work
    const int64_t tiles = std::max<int64_t>(1, ((int64_t)p.table_width * p.block_size + kKeyTile - 1) / kKeyTile);
    const int ctas = (int)std::min<int64_t>(ctas_of(v, num_sms), std::max<int64_t>(1, a.whole ? units : units * tiles / a.min_tiles));
    // A CTA that goes from one unit to another loses some 10 us while the cache is
    // streamed, six key tiles' time; counted as such, 64 sequences of 1025 to 2050
    // keys take 43 us instead of 46, 16 trees of 16 over 8192 71.2, 74.5.  In
    // the small kernel, with few tiles a CTA, the ranges had better begin with the
    // units.
    const bool wide = v == kWide128 || v == kWide256;
    a.change = wide || units * tiles >= 8 * ctas ? 6 : 0;
    switch (v) {
    case kSmall16: return p.block_size % kChunk == 0 ? launch_small<1, true>(a, ctas, stream, why)
                                                     : launch_small<1, false>(a, ctas, stream, why);
    case kSmall32: return p.block_size % kChunk == 0 ? launch_small<2, true>(a, ctas, stream, why)
                                                     : launch_small<2, false>(a, ctas, stream, why);
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
