// What the attention kernels over paged caches (k5 in bf16, k11 in 4 bits) share: how
// the work is cut over the CTAs, which keys a row sees, and how parts are joined.
#pragma once
#include "rc_paged.cuh"

#include <algorithm>
#include <type_traits>

namespace rc {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kKeyTile = 128;          // keys per step of a CTA
// Fewest key tiles a CTA is given (3 trees of 13 over 1500 keys, in equal ranges: 15.3 us
// with two, 19.9 with four, 18.3 with one).
constexpr int32_t kMinTiles = 2;
constexpr float kGrow = 8.0f;          // log2: growth of a row's maximum at which its output is rescaled

struct Args : TreeAttentionLaunch {
    float scale_log2;                  // scale * log2 e
    float grow;                        // kGrow / scale_log2: in scores before that factor
    bool whole;                        // units are not cut
    int32_t change;                    // going to another unit, in key tiles' time
    int32_t join;                      // and joining parts; 0: units are cut in any case
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
// With a window: of the keys that a row sees, in order (the context, then the nodes
// that its mask row names), the first `sinks` and the last `window` count.  So a row
// that sees m nodes has the context keys below `sinks` and from ctx + m - window on;
// which of the others a unit's rows have depends on m, 0 <= m <= nodes.
struct WindowSeq : Seq {
    int32_t lo;                        // below it, and not below sinks: of no row
    int32_t hi;                        // from it on of every row
    int32_t sink_tiles, skip;          // key tiles of the first keys; tiles of no row that follow them
};
template <bool kWindow> using SeqOf = std::conditional_t<kWindow, WindowSeq, Seq>;

template <bool kWindow> __device__ __forceinline__ SeqOf<kWindow> seq_of(const Args &a, int b) {
    SeqOf<kWindow> s;
    s.r0 = (int32_t)max((int64_t)0, min((int64_t)__ldg(a.row_start + b), a.rows));
    const int32_t r1 = (int32_t)max((int64_t)s.r0, min((int64_t)__ldg(a.row_start + b + 1), a.rows));
    s.n = r1 - s.r0;
    const int64_t ctx = max(__ldg(a.context_len + b), 0);
    const int64_t room = (int64_t)a.table_width * a.block_size;
    s.keys = (int32_t)min(ctx + s.n, room);
    s.ctx = (int32_t)min(ctx, (int64_t)s.keys);
    if constexpr (kWindow) {
        s.lo = max(0, s.ctx - a.window);
        s.hi = s.keys - a.window;      // the nodes that exist: keys - ctx at most
        s.sink_tiles = (min(a.sinks, s.ctx) + kKeyTile - 1) / kKeyTile;
        s.skip = max(0, s.lo / kKeyTile - s.sink_tiles);
    }
    return s;
}

template <int kRows> __device__ __forceinline__ int row_tiles(const Args &a, const Seq &s) {
    return (s.n * a.group + kRows - 1) / kRows;
}
// Key tiles that are gone through, and the number of the k-th of them.
__device__ __forceinline__ int key_tiles(const Seq &s) { return max(1, (s.keys + kKeyTile - 1) / kKeyTile); }
__device__ __forceinline__ int key_tiles(const WindowSeq &s) {
    return max(1, (s.keys + kKeyTile - 1) / kKeyTile) - s.skip;
}
__device__ __forceinline__ int tile_at(const Seq &, int k) { return k; }
__device__ __forceinline__ int tile_at(const WindowSeq &s, int k) { return k < s.sink_tiles ? k : k + s.skip; }

// How the units are cut.  Their slots, laid end to end, are shared out evenly.
//   most >= 1: a slot is a part of at most so many key tiles, and a CTA gets one
//              (or, uncut, as many units as another)
//   most == 0: a unit's slots are its key tiles and then `change` empty ones, for
//              the time that the change to it takes
template <int kRows, bool kWindow>
__device__ __forceinline__ int64_t slots_of(const Args &a, int b, int32_t most) {
    const SeqOf<kWindow> s = seq_of<kWindow>(a, b);
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
    const int64_t most = max((int64_t)kMinTiles, quotient(tiles + room - 1, room));
    return most <= a.change + 2 || most * ctas <= tiles + a.change * units ? (int32_t)min(most, (int64_t)INT32_MAX) : 0;
}

// The range of CTA c of `ctas`, and where its first slot lies.  Called by all
// kThreads threads.  kParts: cut into parts where that is better (not in the small
// kernel: its start would take 0.7 us longer, one token over 500 keys 7.9 instead
// of 7.2 us, and few calls have fewer units than CTAs, 4 tokens over 3000 keys 14.0
// and 12.4).  Up to 32 sequences a lane takes one, and each warp finds the range
// by itself (3 trees of 13: 16.6 us, by the block 17.0); beyond, a thread takes a
// run of sequences, and the one whose run holds the slot walks it.
template <int kRows, int kThreads, bool kParts, bool kWindow>
__device__ Place locate(const Args &a, int c, int ctas) {
    __shared__ int64_t warp_tiles[kParts ? kThreads / 32 : 1], warp_units[kParts ? kThreads / 32 : 1];
    __shared__ int32_t warp_longest[kParts ? kThreads / 32 : 1];
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
        int32_t longest = 0;
        for (int b = b0; b < b1; ++b) {
            const SeqOf<kWindow> s = seq_of<kWindow>(a, b);
            const int n = row_tiles<kRows>(a, s) * a.kv_heads, kt = key_tiles(s);
            units += n;
            tiles += (int64_t)n * kt;
            longest = max(longest, n > 0 ? kt : 0);
        }
        longest = __reduce_max_sync(0xFFFFFFFFu, longest);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            tiles += __shfl_xor_sync(0xFFFFFFFFu, tiles, o);
            units += __shfl_xor_sync(0xFFFFFFFFu, units, o);
        }
        if (!alone) {
            if (lane == 0) {
                warp_tiles[kParts ? warp : 0] = tiles;
                warp_units[kParts ? warp : 0] = units;
                warp_longest[kParts ? warp : 0] = longest;
            }
            __syncthreads();
            tiles = units = 0;
            for (int w = 0; w < kThreads / 32; ++w) {
                tiles += warp_tiles[kParts ? w : 0];
                units += warp_units[kParts ? w : 0];
                longest = max(longest, warp_longest[kParts ? w : 0]);
            }
        }
        p.most = most_of(a, tiles, units, ctas);
        if (p.most == 0 && a.join > 0 &&
            quotient(units + ctas - 1, ctas) * longest * ctas <= tiles + a.change * units + (int64_t)a.join * ctas)
            p.most = INT32_MAX;
    }
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += slots_of<kRows, kWindow>(a, b, p.most);
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
    p.used = (int32_t)max((int64_t)1, min((int64_t)ctas, p.most > 0 ? p.total : quotient(p.total, kMinTiles)));
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
        for (int64_t t; off >= (t = slots_of<kRows, kWindow>(a, b, p.most)); ++b)
            off -= t;
        found_b = b;
        found_off = off;
    }
    __syncthreads();
    p.b = found_b;
    p.off = found_off;
    return p;
}

// One piece of a unit: key tiles k0 .. k0 + count - 1 of its kt (tile_at).
template <bool kWindow> struct Piece {
    SeqOf<kWindow> s;
    int32_t b, unit, h, tile;          // sequence, unit within it, its KV head and row tile
    int32_t k0, count, kt;
    int32_t parts;                     // of the unit, where it is cut into such
    int64_t begin;                     // the unit's first slot
    __device__ bool whole() const { return k0 == 0 && count == kt; }
};

// The pieces of a CTA's range, in order.
template <int kRows, bool kWindow> struct Walk {
    int64_t pos, off, hi;
    int32_t b, most;
    __device__ explicit Walk(const Place &p) : pos(p.lo), off(p.off), hi(p.hi), b(p.b), most(p.most) {}
    __device__ bool next(const Args &a, Piece<kWindow> &u) {
        while (pos < hi) {
            u.s = seq_of<kWindow>(a, b);
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

// Whether node i's row sees node j.
__device__ __forceinline__ bool sees(const Args &a, const Seq &s, int i, int j) {
    if (a.tree_mask == nullptr)
        return j <= i;
    return (j >> 6) < a.mask_words &&
           ((__ldg(a.tree_mask + (int64_t)(s.r0 + i) * a.mask_words + (j >> 6)) >> (j & 63)) & 1u) != 0u;
}
// How many of the first n nodes node i's row sees.
__device__ __forceinline__ int seen_before(const Args &a, const Seq &s, int i, int n) {
    if (a.tree_mask == nullptr)
        return min(i + 1, n);
    const uint64_t *row = a.tree_mask + (int64_t)(s.r0 + i) * a.mask_words;
    int count = 0;
    for (int w = 0; w < a.mask_words && 64 * w < n; ++w) {
        const uint64_t v = __ldg(row + w);
        count += __popcll(n - 64 * w >= 64 ? v : v & ((1ull << (n - 64 * w)) - 1ull));
    }
    return count;
}
// The window's begin in the order of what node i's row sees: of its keys from place
// `sinks` on, those before it do not count (i < 0, a row that does not exist: all do).
__device__ __forceinline__ int32_t begin_of_window(const Args &a, const WindowSeq &s, int i) {
    return i < 0 ? 0 : max(0, s.ctx + seen_before(a, s, i, s.keys - s.ctx) - a.window);
}
// Whether logical key p reaches node i's row (whose window begins at `begin`).
__device__ __forceinline__ bool sees_key(const Args &a, const Seq &s, int i, int p, int32_t) {
    return p < s.ctx || (i >= 0 && sees(a, s, i, p - s.ctx));
}
__device__ __forceinline__ bool sees_key(const Args &a, const WindowSeq &s, int i, int p, int32_t begin) {
    if (p < s.ctx)
        return p < a.sinks || p >= begin;
    if (i < 0 || !sees(a, s, i, p - s.ctx))
        return false;
    if (begin <= s.ctx)
        return true;
    const int place = s.ctx + seen_before(a, s, i, p - s.ctx);
    return place < a.sinks || place >= begin;
}
// Whether key p is one that some row of the sequence may not see: a drafted one, or
// one at the window's begin; and whether there is such a key from p to p + n - 1.
__device__ __forceinline__ bool partly_seen(const Args &, const Seq &s, int p) { return p >= s.ctx; }
__device__ __forceinline__ bool partly_seen(const Args &a, const WindowSeq &s, int p) {
    return p >= s.ctx || (p >= a.sinks && p < s.hi);
}
__device__ __forceinline__ bool some_partly_seen(const Args &, const Seq &s, int p, int n) { return p + n > s.ctx; }
__device__ __forceinline__ bool some_partly_seen(const Args &a, const WindowSeq &s, int p, int n) {
    return p + n > s.ctx || (p + n > a.sinks && p < s.hi);
}
// Whether a row may see one of the keys p .. p + n - 1 of a context (or they are
// drafted); what no row sees is not loaded.
__device__ __forceinline__ bool some_seen(const Args &, const Seq &, int, int) { return true; }
__device__ __forceinline__ bool some_seen(const Args &a, const WindowSeq &s, int p, int n) {
    return p < a.sinks || p + n > s.lo;
}
// Whether the first key of its block that is needed is one of p .. p + n - 1 (which
// lie in one block): there a block out of range is counted, once.
__device__ __forceinline__ bool first_needed(const Args &a, const Seq &, int p, int) {
    return (uint32_t)p % (uint32_t)a.block_size == 0u;
}
__device__ __forceinline__ bool first_needed(const Args &a, const WindowSeq &s, int p, int n) {
    const int begin = p - (int)((uint32_t)p % (uint32_t)a.block_size);
    // (a row that sees itself does not see key ctx - window)
    const int first = begin < a.sinks ? begin : max(begin, s.ctx + 1 - a.window);
    return first >= p && first < p + n;
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
template <int kRows, bool kWindow>
__device__ void write_header(const Args &a, const Place &p, const Piece<kWindow> &u, bool unfinite) {
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

// A V row that is infinite or NaN must not reach rows that do not see it (0 * inf in
// the matrix product), so the products take zeros in its place where some row may not
// (partly_seen), and the rows that see it get it added here.  Rare: only where the
// flag of a unit is set.
template <typename S>
__device__ __noinline__ float add_unfinite(const Args &a, const S &s, int b, int h, int i, int d, float x) {
    auto add = [&](int p) {
        const int64_t o = offset_in(a, block_of(a, b, p), h, p);
        const uint32_t v = o < 0 ? 0u : (uint32_t)a.cache[o + kHeadDim + d] << 16;
        if ((v & 0x7F800000u) == 0x7F800000u)
            x += __uint_as_float(v);
    };
    int32_t begin = 0;
    if constexpr (std::is_same_v<S, WindowSeq>) {
        begin = begin_of_window(a, s, i);
        for (int p = max(max(begin, s.lo), a.sinks); p < min(s.hi, s.ctx); ++p)
            add(p);
    }
    for (int p = s.ctx; p < s.keys; ++p)
        if (sees_key(a, s, i, p, begin))
            add(p);
    return x;
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

template <int kRows, bool kWindow, bool kCache4>
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
    const SeqOf<kWindow> s = seq_of<kWindow>(a, hd.b);
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
    if (!kCache4 && unfinite) {
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

template <int kRows, bool kWindow, bool kCache4>
cudaError_t launch_join(const Args &a, int ctas, cudaStream_t stream, const char **why) {
    if (a.partial == nullptr)
        return cudaSuccess;
    *why = "attention join launch";
    return launch_pdl(k5_join<kRows, kWindow, kCache4>, dim3((unsigned)ctas, kRows / kJoinRows<kRows>), dim3(kJoinThreads), 0,
                      stream, 1, a);
}

// The keys of a unit that the block table, and the window, let be, at most: that of the
// first keys, those of the window, which may begin and end inside a tile, and of the
// nodes, of which a mask names so many (an estimate: others cost time only).
inline int64_t most_keys(const TreeAttentionLaunch &a)
{
    const int64_t keys = (int64_t)a.table_width * a.block_size;
    if (a.window == 0)
        return keys;
    const int64_t nodes = a.tree_mask != nullptr ? std::min<int64_t>(a.rows, 64 * (int64_t)a.mask_words) : a.rows;
    return std::min<int64_t>(keys, (((int64_t)a.sinks + kKeyTile - 1) / kKeyTile + 1) * kKeyTile + a.window + nodes);
}

// How a call is cut (Args' whole, change, join, partial), for units of
// `unit_rows` rows and at most `most` CTAs at once; returns the CTAs.
inline int plan(Args &a, int64_t unit_rows, bool wide, int most)
{
    const int64_t units = (a.rows * a.group / unit_rows + a.seqs) * a.kv_heads;      // at most
    const int64_t keys = most_keys(a);
    // Units of at most so many tiles are not worth a cut and a join: one token over
    // 300 keys 6.9 us (cut 11.2), 30 single tokens over 450 to 900 15.0 (19.2); a
    // tile of many rows takes longer, 16 trees of 16 over 480 15.7 (23.2), but 3 of
    // 13 over 900 17.6 whole and 16.1 cut.  With several units a CTA equal ranges
    // of tiles spread ragged lengths better (256 tokens over 450 to 900: 77.4 whole,
    // 73.5 cut; 64 25.9 and 27.8).
    const int whole = wide || units > 3 * most ? 4 : 8;
    if (keys <= whole * kKeyTile) {
        a.partial = nullptr;
        a.whole = true;
    }
    // as many CTAs as fill the GPU, or as the block table lets have work
    const int64_t tiles = std::max<int64_t>(1, (keys + kKeyTile - 1) / kKeyTile);
    const int ctas = (int)std::min<int64_t>(most, std::max<int64_t>(1, a.whole ? units : units * tiles / kMinTiles));
    // A CTA that goes from one unit to another loses some 10 us while the cache is
    // streamed, six key tiles' time; counted as such, 64 sequences of 1025 to 2050
    // keys take 43 us instead of 46, 16 trees of 16 over 8192 71.2, 74.5.  In
    // the small kernel, with few tiles a CTA, the ranges had better begin with the
    // units.
    a.change = wide || units * tiles >= 8 * ctas ? 6 : 0;
    // Units that come out even are not cut where the longest of their rounds takes no
    // more than the cut and some tiles' time for the join (in 4 bits a tile takes
    // longer): 8 trees of 64 over a window of 1024 28.7 us, cut 38.3, of 8192 97.4, 100;
    // 32 of 16 over 1024 in 4 bits 39.5, 47.9.  (Calls that have neither keep their cuts
    // and with them the last bit of their results.)
    a.join = a.cache4 != nullptr ? 4 : (a.window > 0 ? 6 : 0);
    return ctas;
}

}  // namespace

}  // namespace rc
