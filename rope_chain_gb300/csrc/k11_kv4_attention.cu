// K11: attention of drafted tokens over a paged cache in 4 bits (rc_kv4.cuh has the
// format, k5_tree_attention.cu the formulas; the cut over the CTAs and the join are
// those of rc_attention.cuh).
//
// A row of 64 bytes and four scales is read where the bf16 caches have 256 bytes, so
// the arithmetic that makes bf16 numbers of it comes near to being the bound: per 16
// keys some 100 instructions of a warp, 11 for every eight values.  Two things keep it
// down.  The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, with the
// keys as the 16 rows of m16n8k16 and eight query rows as its columns: a group of
// eight query heads and one token fills them, and what is made of a key is used by
// every column.  And the elements of the heads' 64 go to the products' inner index in
// the order in which the half-bytes of a word come apart, (i, i + 4) in one register:
// any order will do as long as Q has it too, and O's rows are put back on the way
// out.
//   K: a lane (g = lane / 4, c = lane % 4) has keys g and g + 8, elements 16c to
//      16c + 15, eight bytes each, all of one scale
//   V: keys 2c, 2c + 1, 2c + 8 and 2c + 9, elements 8g to 8g + 7, a word each; the low
//      halves of two keys' words in one register come apart into pairs of keys
// Every value is an exact bf16 number, so nothing is rounded but the weights (to bf16,
// for the products with V) and the output.  No value is infinite or NaN, so what a row
// does not see stays away by a weight of 0.
//
// Every warp streams its own 16 of a tile's 128 keys from the cache, into registers
// kAhead chunks ahead or through a ring in shared memory, with a running maximum, sum and
// output of its own; the warps' parts are joined at a unit's end.
// Measured: 64 tokens over 4100 to 8200 keys (8 query heads a KV head, 229 MB) 74 us,
// 3.1 TB/s (tree attention over bf16 reads 3.6 times as much); one token over 131071 keys
// (75 MB) 29 us with the join; 32 trees of 2 over 4000 to 8000 52, 16 of 4 47; one token
// over 500 keys 6.5.  Memory does not bound it (with every block in L2 the first took 74 of
// then 77): some 210 instructions of a warp per chunk, half of them on the integer pipe, at
// 2.3 an SM's cycle, and some 20 us of starts, changes of unit and the join.  Tried and no
// faster: chunks in pairs (80), three blocks an SM (80 to 93), four-warp blocks (85 to 96),
// shifts as products on the other pipe (79 to 81), the scores' products in 8 bits (80).
#include "rc_attention.cuh"
#include "rc_kv4.cuh"
#include "rc_tcgen05.cuh"

namespace rc {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps, kChunk = 16;
constexpr int kStride = kHeadDim + 8;  // floats of a row in shared memory

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D = A B
__device__ __forceinline__ void mma16816_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
// The transpose of an 8 x 8 matrix of 16-bit elements (lane l: row l / 4, columns
// 2 (l % 4) and the next).
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// What a lane has of a chunk of 16 keys.
struct Chunk {
    uint2 k[2];                        // keys g, g + 8
    uint32_t v[4];                     // keys 2c, 2c + 1, 2c + 8, 2c + 9
    uint2 scale;                       // lanes 0 to 15: of key `lane`, K's two and V's two
    int32_t at;                        // kRuns: its number in the cache, -1 without a block; else which keys exist
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// kShared: the chunks come through a ring in shared memory instead.  With two row tiles
// that leaves the registers for two blocks an SM (32 trees of 2 over 4000 to 8000 keys: 52
// us for 58); with one it is better over long contexts (64 tokens over 4100 to 8200 keys:
// 74 for 77), not over short ones (256 tokens over 350 to 700: 56 for 52; 64 tokens over a
// window of 512 of 8192 keys 29.5 for 22.4, of 2048 39.2 for 40.3).  There a
// chunk is the K of its rows, 32 bytes each; their V, the rows in the
// order 0 2 4 6 1 3 5 7, so that what a warp reads at once lies in all banks; their
// scales.
constexpr int kRing = 4;               // stages
constexpr uint32_t kChunkV = 512, kChunkScales = 1024, kChunkBytes = 1024 + 128;
template <bool kShared> constexpr uint32_t kSmem = kShared ? kWarps * kRing * kChunkBytes : 0;
constexpr int64_t kLongContext = 2048; // keys that the block table and the window must let be

// Chunks in flight beside the one that is worked on (64 tokens over 4100 to 8200 keys: 82
// us with two, 78 with three), and CTAs on an SM (three, at 80 registers a thread: 93 us).
template <int kTiles> constexpr int kAhead = kTiles == 4 ? 2 : 3;
template <int kTiles> constexpr int kPerSm = kTiles <= 2 ? 2 : 1;

// kTiles: tiles of eight rows.  kRuns: blocks hold a multiple of 16 keys, so a chunk
// is 1 KiB in a row.
template <int kTiles, bool kShared, bool kRuns, bool kWindow>
__global__ void __launch_bounds__(kThreads, kPerSm<kTiles>)
k11_attention(const __grid_constant__ Args a)
{
    constexpr int kRows = 8 * kTiles;
    __shared__ float s_max[kWarps][kRows], s_sum[kWarps][kRows];
    __shared__ __align__(16) float s_out[kWarps][8 * kStride];
    extern __shared__ __align__(128) uint8_t s_ring[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_trigger();
    pdl_wait();

    const Place at = locate<kRows, kThreads, false, kWindow>(a, blockIdx.x, gridDim.x);
    if (a.partial != nullptr && threadIdx.x == 0)
        reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + 1))->last = 0;
    Walk<kRows, kWindow> walk(at);
    Piece<kWindow> u;
    while (walk.next(a, u)) {
        const SeqOf<kWindow> &s = u.s;
        const int b = u.b, h = u.h, tile = u.tile, unit = u.unit, k0 = u.k0, count = u.count;

        // Q: row g of each tile, elements 16c to 16c + 15 as (i, i + 4), for each run of eight
        uint32_t qf[kTiles][4][2];
        // the rows whose scores this lane has: 2c and 2c + 1 of each tile
        int node[kTiles][2];
        int32_t begin[kTiles][2];
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
            const int r = tile * kRows + 8 * m + g, i = r / a.group;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                a.q + (int64_t)(s.r0 + i) * a.q_row_stride + (h * a.group + r - i * a.group) * kHeadDim) + 2 * c;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint4 x = i < s.n ? __ldg(src + w) : make_uint4(0, 0, 0, 0);
                qf[m][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);
                qf[m][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);
                qf[m][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);
                qf[m][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);
            }
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int n = (tile * kRows + 8 * m + 2 * c + f) / a.group;
                node[m][f] = n < s.n ? n : -1;
                if constexpr (kWindow)
                    begin[m][f] = begin_of_window(a, s, node[m][f]);
            }
        }
        // o[m][t][2e + f]: row 2c + f, element 8g + 2t + e.  ref as in k5_small; limit is of
        // the scores before their factor
        float o[kTiles][4][4], ref[kTiles][2], limit[kTiles][2], sum[kTiles][2];
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                limit[m][f] = -INFINITY;
                ref[m][f] = sum[m][f] = 0.0f;
            }
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[m][t][e] = 0.0f;
        }

        // Where chunks lie, as in k5_small: with kRuns a lane has chunk (j & ~31) +
        // lane, else a key of chunk j; block numbers are loaded one round before.
        auto first_key = [&](int j) { return tile_at(s, k0 + j) * kKeyTile + warp * kChunk; };
        auto lane_key = [&](int j) { return kRuns ? first_key(j + lane) : first_key(j) + (lane & 15); };
        auto table_entry = [&](int j) -> int32_t {
            const int p = lane_key(j);
            return j + (kRuns ? lane : 0) < count && p < s.keys ? block_of(a, b, p) : -1;
        };
        int32_t entry = table_entry(0);
        // kRuns: the number of this lane's chunk of 16 rows (a cache holds fewer than
        // 2^31 of them: it would be 2 TB); else the row of its key
        using Where = std::conditional_t<kRuns, int32_t, int64_t>;
        Where from = -1;
        auto place = [&](int j) {
            const int p = lane_key(j);
            const bool wanted = j + (kRuns ? lane : 0) < count && p < s.keys && some_seen(a, s, p, kRuns ? kChunk : 1);
            const bool there = wanted && entry >= 0 && entry < a.num_blocks;
            const uint32_t bs = (uint32_t)a.block_size;
            const int64_t row = ((int64_t)entry * a.kv_heads + h) * bs + (uint32_t)p % bs;
            from = there ? (Where)(kRuns ? row / kChunk : row) : (Where)-1;
            if (wanted && !there && (kRuns || lane < 16) && unit == 0 && a.err != nullptr &&
                first_needed(a, s, p, kRuns ? min(kChunk, s.keys - p) : 1))
                atomicAdd(a.err, 1);
        };
        // (rows that do not exist are read from row 0, or lie in a block that does:
        // their values are finite whatever is there, their weights 0)
        const uint8_t *const k_at = a.cache4 + g * kKv4Row + 8 * c, *const v_at = a.cache4 + 2 * c * kKv4Row + 32 + 4 * g;
        const uint16_t *const scale_at = a.scales + (lane & 15) * kKv4Scales;
        auto load = [&](int j, Chunk &x) {
            if constexpr (kRuns) {
                if ((j & 31) == 0) {
                    place(j);
                    entry = table_entry(j + 32);
                }
                x.at = __shfl_sync(0xFFFFFFFFu, from, j & 31);
                const uint32_t i = (uint32_t)max(x.at, 0);
                const uint8_t *const k = k_at + (uint64_t)i * (kChunk * kKv4Row), *const v = v_at + (uint64_t)i * (kChunk * kKv4Row);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    x.k[e] = __ldg(reinterpret_cast<const uint2 *>(k + 8 * e * kKv4Row));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x.v[e] = __ldg(reinterpret_cast<const uint32_t *>(v + ((e & 1) + 8 * (e >> 1)) * kKv4Row));
                x.scale = __ldg(reinterpret_cast<const uint2 *>(scale_at + (uint64_t)i * (kChunk * kKv4Scales)));
            } else {
                place(j);
                entry = table_entry(j + 1);
                x.at = (int32_t)(__ballot_sync(0xFFFFFFFFu, from >= 0) & 0xFFFFu);
                const int64_t row = max(from, (int64_t)0);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    x.k[e] = __ldg(reinterpret_cast<const uint2 *>(
                                       a.cache4 + __shfl_sync(0xFFFFFFFFu, row, g + 8 * e) * kKv4Row) + c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x.v[e] = __ldg(reinterpret_cast<const uint32_t *>(
                                       a.cache4 + __shfl_sync(0xFFFFFFFFu, row, 2 * c + (e & 1) + 8 * (e >> 1)) * kKv4Row) + 8 + g);
                x.scale = __ldg(reinterpret_cast<const uint2 *>(a.scales + row * kKv4Scales));
            }
        };
        // (v_word(e): x.v[e], asked for late)
        auto work = [&](int j, const Chunk &x, const auto &v_word) {
            const int p0 = first_key(j);
            // scales: of this lane's two keys of K, twice each; of its pairs of keys of V
            const uint32_t ks = kv4_scales(x.scale.x), vs = kv4_scales(x.scale.y);
            uint32_t k_scale[2], v_scale[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                k_scale[e] = __byte_perm(__shfl_sync(0xFFFFFFFFu, ks, g + 8 * e), 0u, c < 2 ? 0x1010 : 0x3232);
                v_scale[e] = __byte_perm(__shfl_sync(0xFFFFFFFFu, vs, 2 * c + 8 * e), __shfl_sync(0xFFFFFFFFu, vs, 2 * c + 1 + 8 * e),
                                         g < 4 ? 0x5410 : 0x7632);
            }
            float t[kTiles][4];                         // keys g, g, g + 8, g + 8; rows 2c, 2c + 1
            const uint32_t ko[2] = {kv4_offsets(k_scale[0]), kv4_offsets(k_scale[1])};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t kf[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    kf[e] = fma_bf16x2(kv4_pair(k < 2 ? x.k[e & 1].x : x.k[e & 1].y, 2 * (k & 1) + (e >> 1)), k_scale[e & 1], ko[e & 1]);
#pragma unroll
                for (int m = 0; m < kTiles; ++m) {
                    if (k == 0)
                        mma16816_new(t[m], kf, qf[m][k][0], qf[m][k][1]);
                    else
                        mma16816(t[m], kf, qf[m][k][0], qf[m][k][1]);
                }
            }
            if ((kRuns ? x.at < 0 : x.at != 0xFFFF) || some_partly_seen(a, s, p0, kChunk)) {
                const uint32_t real = !kRuns ? (uint32_t)x.at : x.at < 0 ? 0u : (1u << max(0, min(kChunk, s.keys - p0))) - 1u;
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int in = g + 8 * (e >> 1);
                        if (!((real >> in) & 1u) || !sees_key(a, s, node[m][e & 1], p0 + in, kWindow ? begin[m][e & 1] : 0))
                            t[m][e] = -INFINITY;
                    }
            }
            bool grew = false;
            float now[kTiles][2];
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    now[m][f] = fmaxf(t[m][f], t[m][2 + f]);
                    grew |= now[m][f] > limit[m][f];
                }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        float y = now[m][f];
                        y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4));
                        y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 8));
                        y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 16));
                        if (y > limit[m][f]) {
                            const float top = y * a.scale_log2;
                            const float shrink = limit[m][f] == -INFINITY ? 0.0f : ex2(-ref[m][f] - top);
                            ref[m][f] = -top;
                            limit[m][f] = y + a.grow;
                            sum[m][f] *= shrink;
#pragma unroll
                            for (int n = 0; n < 4; ++n) {
                                o[m][n][f] *= shrink;
                                o[m][n][2 + f] *= shrink;
                            }
                        }
                    }
            }
            uint32_t pf[kTiles][2];
#pragma unroll
            for (int m = 0; m < kTiles; ++m) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x0 = t[m][2 * e], &x1 = t[m][2 * e + 1];
                    fma2_rn(x0, x1, a.scale_log2, a.scale_log2, ref[m][0], ref[m][1]);
                    x0 = ex2(x0);
                    x1 = ex2(x1);
                    pf[m][e] = transposed(pack_bf16x2(x0, x1));
                }
                add2_rn(t[m][0], t[m][1], t[m][2], t[m][3]);
                add2_rn(sum[m][0], sum[m][1], t[m][0], t[m][1]);
            }
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = v_word(e);
            const uint32_t vo[2] = {kv4_offsets(v_scale[0]), kv4_offsets(v_scale[1])};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                uint32_t vf[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    // element 2n + (e & 1) of keys 2c, 2c + 1 (and + 8): from the low or
                    // the high halves of their words
                    const uint32_t two = __byte_perm(v[2 * (e >> 1)], v[2 * (e >> 1) + 1], n < 2 ? 0x5410 : 0x7632);
                    vf[e] = fma_bf16x2(kv4_pair(two, 2 * (n & 1) + (e & 1)), v_scale[e >> 1], vo[e >> 1]);
                }
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
                    mma16816(o[m][n], vf, pf[m][0], pf[m][1]);
            }
        };
        if constexpr (kShared) {
            const uint32_t ring = smem_u32(s_ring) + (uint32_t)warp * (kRing * kChunkBytes);
            const int row_of = lane >> 1, half = 16 * (lane & 1);
            const uint32_t to_k = ring + 16u * lane;
            const uint32_t to_v = ring + kChunkV + 32u * (((row_of >> 1) & 3) | (row_of & 1) << 2 | (row_of & 8)) + half;
            const uint32_t to_scales = ring + kChunkScales + 4u * lane;
            const uint8_t *const from4 = a.cache4 + row_of * kKv4Row + half;
            const uint16_t *const from_scales = a.scales + 2 * lane;
            // kRuns: which of the 32 chunks that `from` is of, and of the 32 before, are not
            // there; else which keys of a stage's chunk are
            uint32_t lost = 0u, lost_before = 0u, there[kRing];
#pragma unroll
            for (int i = 0; i < kRing; ++i)
                there[i] = 0u;
            auto issue = [&](int j, int st) {
                const uint32_t at = st * kChunkBytes;
                if constexpr (kRuns) {
                    if ((j & 31) == 0) {
                        place(j);
                        entry = table_entry(j + 32);
                        lost_before = lost;
                        lost = __ballot_sync(0xFFFFFFFFu, from < 0);
                    }
                    const uint64_t i = (uint32_t)max(__shfl_sync(0xFFFFFFFFu, from, j & 31), 0);
                    const uint8_t *const src = from4 + i * (kChunk * kKv4Row);
                    copy16(to_k + at, src);
                    copy16(to_v + at, src + 32);
                    copy4(to_scales + at, from_scales + i * (kChunk * kKv4Scales));
                } else {
                    place(j);
                    entry = table_entry(j + 1);
                    there[st] = __ballot_sync(0xFFFFFFFFu, from >= 0) & 0xFFFFu;
                    const int64_t row = __shfl_sync(0xFFFFFFFFu, max(from, (int64_t)0), row_of);
                    const uint8_t *const src = from4 + (row - row_of) * kKv4Row;
                    copy16(to_k + at, src);
                    copy16(to_v + at, src + 32);
                    copy4(to_scales + at, a.scales + row * kKv4Scales + 2 * (lane & 1));
                }
            };
            const uint8_t *const own = s_ring + warp * (kRing * kChunkBytes);
            const uint8_t *const k_from = own + 32 * g + 8 * c, *const v_from = own + kChunkV + 32 * c + 4 * g;
            const uint8_t *const scale_from = own + kChunkScales + 8 * (lane & 15);
#pragma unroll
            for (int j = 0; j < kRing - 1; ++j) {
                if (j < count)
                    issue(j, j);
                copy_commit();
            }
            for (int j0 = 0; j0 < count; j0 += kRing) {
#pragma unroll
                for (int i = 0; i < kRing; ++i) {
                    const int j = j0 + i;
                    if (j >= count)
                        break;
                    copy_wait<kRing - 2>();
                    __syncwarp();
                    // (into the stage of chunk j - 1, which every lane has read)
                    if (j + kRing - 1 < count)
                        issue(j + kRing - 1, (i + kRing - 1) % kRing);
                    copy_commit();
                    Chunk now;
                    const uint32_t at = i * kChunkBytes;
                    now.scale = *reinterpret_cast<const uint2 *>(scale_from + at);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        now.k[e] = *reinterpret_cast<const uint2 *>(k_from + at + 256u * e);
                    // (`lost` is of the 32 that the chunk issued last is one of)
                    const uint32_t gone = ((min(j + kRing - 1, count - 1) ^ j) & ~31) != 0 ? lost_before : lost;
                    now.at = !kRuns ? (int32_t)there[i] : (gone >> (j & 31)) & 1u ? -1 : 0;
                    work(j, now, [&](int e) { return *reinterpret_cast<const volatile uint32_t *>(v_from + at + 128u * e); });
                }
            }
            copy_wait<0>();
        }
        constexpr int kBuffers = kAhead<kTiles> + 1;
        Chunk ring[kBuffers];
        const int streamed = kShared ? 0 : count;       // straight into registers
#pragma unroll
        for (int i = 0; i < kAhead<kTiles>; ++i)
            if (i < streamed)
                load(i, ring[i]);
        for (int j = 0; j < streamed; j += kBuffers) {
#pragma unroll
            for (int i = 0; i < kBuffers; ++i) {
                if (j + i >= streamed)
                    break;
                if (j + i + kAhead<kTiles> < streamed)
                    load(j + i + kAhead<kTiles>, ring[(i + kAhead<kTiles>) % kBuffers]);
                work(j + i, ring[i], [&](int e) { return ring[i].v[e]; });
            }
        }

        // The warps' parts, joined.
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                float x = sum[m][f];
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
                x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
                if (g == 0) {
                    s_max[warp][8 * m + 2 * c + f] = limit[m][f] == -INFINITY ? -INFINITY : -ref[m][f];
                    s_sum[warp][8 * m + 2 * c + f] = x;
                }
            }
        __syncthreads();
        const bool whole = u.whole();
        float *slot = whole ? nullptr : slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + (k0 == 0 ? 1 : 0));
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int r = 2 * c + f;
                float now = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    now = fmaxf(now, s_max[w][8 * m + r]);
                const float y = limit[m][f] == -INFINITY ? 0.0f : ex2(-ref[m][f] - now);
                float4 *dst = reinterpret_cast<float4 *>(&s_out[warp][r * kStride + 8 * g]);
                dst[0] = make_float4(o[m][0][f] * y, o[m][0][2 + f] * y, o[m][1][f] * y, o[m][1][2 + f] * y);
                dst[1] = make_float4(o[m][2][f] * y, o[m][2][2 + f] * y, o[m][3][f] * y, o[m][3][2 + f] * y);
            }
            __syncthreads();
            // 8 rows of 64: a warp has a row, a lane two columns
            const int r = warp, col = 2 * lane;
            float x0 = 0.0f, x1 = 0.0f, now = -INFINITY, total = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                now = fmaxf(now, s_max[w][8 * m + r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 y = *reinterpret_cast<const float2 *>(&s_out[w][r * kStride + col]);
                x0 += y.x;
                x1 += y.y;
                total = __fmaf_rn(s_sum[w][8 * m + r], ex2(s_max[w][8 * m + r] - (now == -INFINITY ? 0.0f : now)), total);
            }
            const int row = tile * kRows + 8 * m + r, i = row / a.group;
            if (!whole) {
                *reinterpret_cast<float2 *>(slot + kSlotOut<kRows> + (8 * m + r) * kHeadDim + col) = make_float2(x0, x1);
                if (lane == 0) {
                    slot[kSlotMax<kRows> + 8 * m + r] = now;
                    slot[kSlotSum<kRows> + 8 * m + r] = total;
                }
                if (threadIdx.x == 0 && m == 0)
                    write_header<kRows, kWindow>(a, at, u, false);
            } else if (i < s.n) {
                const int head = h * a.group + row - i * a.group;
                const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
                *reinterpret_cast<uint32_t *>(a.out + (int64_t)(s.r0 + i) * a.out_row_stride + head * kHeadDim + col) =
                    pack_bf16x2(x0 * inv, x1 * inv);
                if (lane == 0 && a.lse != nullptr)
                    a.lse[(int64_t)(s.r0 + i) * (a.kv_heads * a.group) + head] =
                        total == 0.0f ? -INFINITY : __fmaf_rn(now, kLn2, logf(total));
            }
            if (whole && threadIdx.x == 0 && m == 0 && unit == 0 && s.n > 0 && a.err != nullptr &&
                (int64_t)max(__ldg(a.context_len + b), 0) + s.n > s.keys)
                atomicAdd(a.err, 1);
            __syncthreads();
        }
    }
}

// By the average rows of a unit; any kernel is right for any unit.  From 33 rows on
// the products are the bound, and k5_wide takes the call (blocks of a multiple of 8
// keys; other block sizes stay here).  8 sequences over 4096 keys, and 32, us:
//   up to 8 rows    one tile: 14.4 and 31.8 at 8 rows, two tiles 16.6 and 39.5; at 16 17.2 and 42.9
//   up to 16        two: 17.3 and 40.9 at 16, four 23.1 and 60.2
//   up to 32        four: 25.1 and 64.0 at 32, two 25.9 and 70.0, k5_wide<1> 31.4 and 88.0; at
//                   24 23.9 and 62.1, two 21.9 and 55.0
//   up to 128       k5_wide<1>: 31.5 and 87.8 at 40 rows, four 31.2 and 89.7; at 128 33.8 and
//                   90.3, k5_wide<2> 39.0 and 120
//   beyond          k5_wide<2>: 40.0 and 122 at 160, k5_wide<1> 50.1 and 160
enum Variant { kRows8, kRows16, kRows32, kRows128, kRows256 };
Variant variant_for(int64_t rows, int32_t seqs, int32_t group, int32_t block_size) {
    const int64_t mean = (rows + seqs - 1) / seqs * group;
    if (mean <= 16)
        return mean <= 8 ? kRows8 : kRows16;
    if (mean <= 32 || block_size % 8 != 0)
        return kRows32;
    return mean <= 128 ? kRows128 : kRows256;
}
int tiles_of(Variant v) { return v == kRows8 ? 1 : v == kRows16 ? 2 : 4; }
int ctas_of(Variant v, int num_sms) {
    return num_sms * (v == kRows8 ? kPerSm<1> : v == kRows16 ? kPerSm<2> : kPerSm<4>);
}
size_t workspace_of(Variant v, int num_sms) {
    if (v >= kRows128)
        return kv4_wide_workspace(v == kRows256, num_sms);
    const size_t floats = v == kRows8 ? kSlotFloats<8> : v == kRows16 ? kSlotFloats<16> : kSlotFloats<32>;
    return 2 * (size_t)ctas_of(v, num_sms) * floats * sizeof(float);
}

template <int kTiles, bool kShared, bool kRuns, bool kWindow>
cudaError_t launch_tiles(const Args &a, int ctas, cudaStream_t stream, const char **why)
{
    static bool configured[64] = {};
    cudaError_t e = kShared ? allow_smem(k11_attention<kTiles, kShared, kRuns, kWindow>, kSmem<kShared>, configured) : cudaSuccess;
    if (e != cudaSuccess)
        return e;
    *why = "attention launch";
    e = launch_pdl(k11_attention<kTiles, kShared, kRuns, kWindow>, dim3((unsigned)ctas), dim3(kThreads), kSmem<kShared>, stream, 1, a);
    return e != cudaSuccess ? e : launch_join<8 * kTiles, kWindow, true>(a, ctas, stream, why);
}

template <bool kRuns, bool kWindow>
cudaError_t launch_variant(Variant v, const Args &a, int ctas, cudaStream_t stream, const char **why)
{
    switch (v) {
    case kRows8:
        return most_keys(a) >= kLongContext
                   ? launch_tiles<1, true, kRuns, kWindow>(a, ctas, stream, why)
                   : launch_tiles<1, false, kRuns, kWindow>(a, ctas, stream, why);
    case kRows16: return launch_tiles<2, true, kRuns, kWindow>(a, ctas, stream, why);
    default: return launch_tiles<4, false, kRuns, kWindow>(a, ctas, stream, why);
    }
}

}  // namespace

size_t kv4_attention_workspace(int64_t rows, int32_t seqs, int32_t group, int num_sms)
{
    // for whichever block size, and for any call of fewer rows or more sequences too
    const Variant last = variant_for(rows, seqs, group, 8);
    size_t most = 0;
    for (const Variant v : {kRows8, kRows16, kRows32, kRows128, kRows256})
        if (v <= last)
            most = std::max(most, workspace_of(v, num_sms));
    return most;
}

cudaError_t launch_kv4_attention(const TreeAttentionLaunch &p, int num_sms, cudaStream_t stream, const char **why)
{
    Args a{};
    static_cast<TreeAttentionLaunch &>(a) = p;
    a.scale_log2 = p.scale * kLog2e;
    a.grow = kGrow / a.scale_log2;
    const Variant v = variant_for(p.rows, p.seqs, p.group, p.block_size);
    if (v >= kRows128)
        return launch_kv4_wide(p, v == kRows256, num_sms, stream, why);
    const int ctas = plan(a, 8 * tiles_of(v), false, ctas_of(v, num_sms));
    if (p.block_size % kChunk == 0)
        return p.window > 0 ? launch_variant<true, true>(v, a, ctas, stream, why)
                            : launch_variant<true, false>(v, a, ctas, stream, why);
    return p.window > 0 ? launch_variant<false, true>(v, a, ctas, stream, why)
                        : launch_variant<false, false>(v, a, ctas, stream, why);
}

}  // namespace rc
