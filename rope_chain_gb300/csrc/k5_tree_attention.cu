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
#include "rc_attention.cuh"
#include "rc_kv4.cuh"
#include "rc_tcgen05.cuh"

#include <cmath>

namespace rc {

__device__ unsigned int g_attention_faults;

namespace {

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
// With a window (kWindow) only the key tiles that some row may see are gone through: 64
// tokens over a window of 4096 + 16 of 8192 to 16384 keys (537 MB) 95 us, 5.7 TB/s; one
// token over one of 1024 + 4 of 131071 keys 12, where ten tiles are cut and joined.
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
// are such as a row may not see (lo, hi); true if there was one.
__device__ __forceinline__ bool finite_only(uint32_t &w, bool lo, bool hi) {
    const bool x = lo && (w & 0x00007F80u) == 0x00007F80u, y = hi && (w & 0x7F800000u) == 0x7F800000u;
    if (x)
        w &= 0xFFFF0000u;
    if (y)
        w &= 0x0000FFFFu;
    return x || y;
}

// kRuns: blocks hold a multiple of 16 keys, so a chunk is 4 KiB in a row.
template <int kTiles, bool kRuns, bool kWindow>
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

    const Place at = locate<kRows, kSmallThreads, false, kWindow>(a, blockIdx.x, gridDim.x);
    if (a.partial != nullptr && threadIdx.x == 0)
        reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + 1))->last = 0;
    Walk<kRows, kWindow> walk(at);
    Piece<kWindow> u;
    while (walk.next(a, u)) {
        const SeqOf<kWindow> &s = u.s;
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
        int32_t begin[kTiles][2];                       // of the rows' windows
        if constexpr (kWindow) {
#pragma unroll
            for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    begin[m][e] = begin_of_window(a, s, node[m][e]);
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
        auto first_key = [&](int j) { return tile_at(s, k0 + j) * kKeyTile + warp * kChunk; };
        auto lane_key = [&](int j) { return kRuns ? first_key(j + lane) : first_key(j) + (lane & 15); };
        auto table_entry = [&](int j) -> int32_t {          // for this lane's key at or after chunk j
            const int p = lane_key(j);
            return j + (kRuns ? lane : 0) < count && p < s.keys ? block_of(a, b, p) : -1;
        };
        int32_t entry = table_entry(0);
        int64_t from = -1;
        auto place = [&](int j) {                           // this lane's row from `entry`
            const int p = lane_key(j);
            const bool there = j + (kRuns ? lane : 0) < count && p < s.keys;
            const bool wanted = there && some_seen(a, s, p, kRuns ? kChunk : 1);
            from = wanted ? offset_in(a, entry, h, p) : -1;
            // once per block that is out of range: at the first of its keys that is needed
            if (wanted && from < 0 && (kRuns || lane < 16) && unit == 0 && a.err != nullptr &&
                first_needed(a, s, p, kRuns ? min(kChunk, s.keys - p) : 1))
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
            const bool partly = some_partly_seen(a, s, p0, kChunk);
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
            if (real != 0xFFFFu || partly) {
#pragma unroll
                for (int m = 0; m < kTiles; ++m)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int in = 8 * n + 2 * (lane & 3) + (e & 1);
                            if (!((real >> in) & 1u) ||
                                !sees_key(a, s, node[m][e >> 1], p0 + in, kWindow ? begin[m][e >> 1] : 0))
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
                if (partly) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int p = p0 + 8 * (q & 1) + 2 * (lane & 3);
                        unfinite |= finite_only(vf[q], partly_seen(a, s, p), partly_seen(a, s, p + 1));
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
                    write_header<kRows, kWindow>(a, at, u, unfinite);
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
// GFLOP) 274 us, 1.0 PFLOP/s, some 2500 cycles per 256 x 128
// (in blocks of 16 keys; 264 us in blocks of 128): the steps of the two row tiles,
// products, softmax and weights, one after the other; tensor pipe 43 %, issue slots
// 64 %.  16 trees of 16 over 8192 keys (273 MB) 69.5 us, 3.9 TB/s: 44 us at 6.2 TB/s
// between a start of 9 us (launch, lengths, Q, first tile) and changes of unit and
// the join of 17.  Two CTAs an SM leave kQ = 1 96 registers a thread, of which it
// spills 51 (204 bytes stored, 676 loaded; with a window one); kQ = 2 spills one.
// Key tiles that hold drafted keys, the end, or a window's begin, take a masked path; there the
// V rows past the end are zeroed and what is infinite or NaN in a drafted one
// is taken out (see add_unfinite).  Every wait is bounded; on timeout a sticky
// fault bit is raised and all roles leave.

enum : unsigned { kFaultLoad = 1u, kFaultMma = 2u, kFaultSoftmax = 4u, kFaultDrain = 8u };

constexpr uint32_t kTileBytes = kKeyTile * kHeadDim * 2;           // K or V of a step, Q of a tile: 16 KiB
template <int kQ> constexpr int kSoftmaxWarps = 8 * kQ;
// A warp's boxes are issued one by one, at some 130 cycles each.  With two row
// tiles one warp loads K and another V: 274 us instead of 323 for 8 trees of 64
// tokens over 32768 keys (512 rows a KV head, blocks of 16; of 128 264 either way).
// With one row tile a single warp loads both, as an eleventh warp would leave 88
// registers a thread for two CTAs an SM: 16 trees of 16 over 8192 keys take 70 us,
// with two loaders 76.
//
// kFour: over a cache in 4 bits the loaders make bf16 numbers of the rows in shared
// memory, in place of the boxes: 32 elements and their scale to a lane.  That is some
// 1000 instructions a tile, more than one warp (or two for two row tiles) issues beside
// the softmax: 16 trees of 16 over a window of 6000 keys 103 us with one loader, with two
// 79, with three, as many as fit at 80 registers a thread, 68; 8 trees of 64 over 32768
// keys 538 with two, with four 380 (bf16: 65 and 274).  The loaders cost the softmax warps
// registers, 80 a thread instead of 96.  A branch between a loader's boxes keeps it from
// working on several at once: 380 us would be 460.
constexpr int kTileBoxes = 16;         // of eight keys
template <int kQ, bool kFour> constexpr int kLoaders = kFour ? (kQ == 1 ? 3 : 4) : kQ;
template <int kQ, bool kFour> constexpr int kWideThreads = 32 * (kSoftmaxWarps<kQ> + kQ + kLoaders<kQ, kFour>);
template <int kQ> constexpr int kWideStages = kQ == 1 ? 3 : 5;
template <int kQ> constexpr uint32_t kTmemCols = 256u * kQ;        // per row tile: S 128, P 64, O 64 columns
constexpr uint32_t kPCol = 128u, kOCol = 192u;
template <int kQ> constexpr size_t kWideSmem = kQ * kTileBytes + kWideStages<kQ> * 2 * kTileBytes;

// Keeps x in local memory: what is read at a piece's ends only would otherwise
// crowd the scores out of the registers.  Used with two row tiles (8 trees of 64
// tokens over 32768 keys: 274 us, without 288; in blocks of 128 265 and 288), with a
// window (8 trees of 64 over one of 8192 98 and 100 us, with one row tile 64 and 63) and
// in 4 bits, not with one row tile over bf16 (16 trees of 16 over 8192 keys: 69.7 us,
// with it 70.4).
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
// One lane of a warp whose lanes are all here; the compiler knows it for one (the
// products' operands otherwise go through a loop over lanes: 8 trees of 64 tokens over a
// window of 8192 102 us, so 100).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0u;
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
// i < 0: none of the drafted ones.  `begin`: of the row's window.
template <bool kWindow> __device__ uint32_t seen32(const Args &a, const SeqOf<kWindow> &s, int i, int base, int32_t begin) {
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
    if constexpr (kWindow) {
        uint32_t seen = (ctx & (below(a.sinks - base) | ~below(begin - base))) | (drafted & ~ctx);
        if (i >= 0 && begin > s.ctx && base + 32 > s.ctx) {
            // nodes that the window has left behind, by their place in the row's order
            int place = s.ctx + seen_before(a, s, i, max(0, base - s.ctx));
            for (uint32_t rest = drafted & ~ctx; rest != 0u && place < begin; rest &= rest - 1u, ++place)
                if (place >= a.sinks)
                    seen &= ~(rest & (0u - rest));
        }
        return seen & below(s.keys - base);
    }
    return (ctx | (drafted & ~ctx)) & below(s.keys - base);
}

template <int kQ, bool kWindow, bool kFour>
__global__ void __launch_bounds__(kWideThreads<kQ, kFour>, kQ == 1 ? 2 : 1)
k5_wide(const __grid_constant__ CUtensorMap map, const __grid_constant__ Args a, int box)
{
    constexpr int kRows = 128 * kQ, kStages = kWideStages<kQ>, kThreads = kWideThreads<kQ, kFour>;
    constexpr int kMmaWarp = kSoftmaxWarps<kQ>, kLoadWarp = kMmaWarp + kQ;
    extern __shared__ __align__(1024) uint8_t smem_wide[];
    const uint32_t sQ = smem_u32(smem_wide), sK = sQ + kQ * kTileBytes;     // a stage: K, then V
    __shared__ uint64_t bars[2 * kStages + 6 * kQ];
    // by piece modulo 8: a row tile is never more than kStages + 1 pieces ahead
    // of another, whose products free its stages
    __shared__ uint32_t s_tmem, s_skip, s_bad[kStages], s_unfinite[8];
    __shared__ __align__(16) uint16_t s_gone[kFour ? kStages : 1][8];  // kFour: such of each loader
    static_assert(kStages + 1 < 8, "pieces in flight");
    const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * kStages, q_ready0 = empty0 + 8u * kStages;
    const uint32_t s_full0 = q_ready0 + 8u * kQ, s_free0 = s_full0 + 8u * kQ, p_ready0 = s_free0 + 8u * kQ;
    const uint32_t o_done0 = p_ready0 + 8u * kQ, drain0 = o_done0 + 8u * kQ;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    pdl_trigger();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full0 + 8u * i, kLoaders<kQ, kFour>);
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
        for (int i = 0; kFour && i < 8 * kStages; ++i)
            s_gone[i / 8][i % 8] = 0;
        // one decision for the CTA: a raised fault skips the work
        s_skip = *reinterpret_cast<volatile unsigned int *>(&g_attention_faults);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (!kFour)
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
    Place at = locate<kRows, kThreads, true, kWindow>(a, blockIdx.x, gridDim.x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;                       // row tile t: S, P, O from column 256 t
    if (a.partial != nullptr && threadIdx.x == 0)
        reinterpret_cast<Header *>(slot_of<kRows>(a, 2 * (int64_t)blockIdx.x + 1))->last = 0;
    Walk<kRows, kWindow> walk(at);
    if (s_skip != 0u)
        walk.hi = walk.pos;
    Piece<kWindow> u;
    if constexpr ((kQ == 2 || kWindow) && !kFour) {
        in_memory(at);
        in_memory(walk);
        in_memory(u);
    }
    uint32_t n = 0;                                     // key tiles of earlier pieces
    uint32_t piece = 0;

    if constexpr (kFour) {
        in_memory(at);
        in_memory(walk);
        in_memory(u);
    }
    if (kFour && warp >= kLoadWarp) {
        // A tile's 16 boxes of eight keys, kOwn to a warp (with three warps two boxes are
        // done twice, as a branch around them would part their arithmetic).  Lane 4r + q has key r of a box
        // and of its 64 bytes the q-th 16, K's two halves and V's two: a group of 32
        // elements with one scale.  A box's registers are loaded again, for the next
        // kOwn boxes, as soon as they are used.  In a word the elements come apart as
        // (i, i + 4): the heads' elements are in that order in shared memory, Q's too, and
        // O's columns are put back at the end.  V's lanes take their words in the order
        // 2 3 0 1, so that the eight lanes of a store's phase write to all banks.
        constexpr int kWarps = kLoaders<kQ, kFour>, kOwn = 2 * ((kTileBoxes / 2 + kWarps - 1) / kWarps);
        constexpr int kAtOnce = 32 / kOwn;              // tiles whose boxes are looked up at once, a lane each
        const int first_box = min((warp - kLoadWarp) * kOwn, kTileBoxes - kOwn), r = lane >> 2, q = lane & 3;
        const uint32_t first_word = (q & 2) ? 2u : 0u;
        // where this lane's words of box 0 go: word i, chunk 4 (q % 2) + i of the row
        const uint32_t row_at = sK + (q >> 1) * kTileBytes + (uint32_t)(8 * first_box + r) * 128u;
        uint32_t chunk_at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            chunk_at[i] = row_at + (((4u * (q & 1) + (i ^ first_word)) ^ (uint32_t)r) << 4);
        const uint8_t *const from4 = a.cache4 + r * kKv4Row + 16 * q + 4 * first_word;
        const int other = first_word != 0u ? -1 : 1;    // from the first two words to the others
        const uint16_t *const from_scales = a.scales + r * kKv4Scales + q;
        bool fine = true;
        while (fine && walk.next(a, u)) {
            const SeqOf<kWindow> &s = u.s;
            uint2 word[kOwn][2];
            uint32_t scale[kOwn];
            // this lane's box, of tile j + lane / kOwn: its table entry, then the number of
            // its eight rows in the cache (negative: none)
            auto key_of = [&](int j) { return tile_at(s, u.k0 + j + lane / kOwn) * kKeyTile + (first_box + lane % kOwn) * 8; };
            const bool has_box = lane < kAtOnce * kOwn;
            auto look_up = [&](int j) -> int {
                const int p = key_of(j);
                return has_box && j + lane / kOwn < u.count && p < s.keys ? block_of(a, u.b, p) : 0;
            };
            auto place = [&](int j, int blk) -> int32_t {
                const int p = key_of(j);
                const bool mine = has_box && j + lane / kOwn < u.count && p < s.keys && some_seen(a, s, p, 8);
                const bool lost = mine && (blk < 0 || blk >= a.num_blocks);
                if (lost && u.unit == 0 && a.err != nullptr && first_box + lane % kOwn >= (warp - kLoadWarp) * kOwn &&
                    first_needed(a, s, p, min(8, s.keys - p)))
                    atomicAdd(a.err, 1);
                if (!mine || lost)
                    return lost ? -1 : -2;              // (-2: hidden by the rows' masks anyway)
                const uint32_t bs = (uint32_t)a.block_size;
                return (int32_t)((((int64_t)blk * a.kv_heads + u.h) * bs + (uint32_t)p % bs) / 8);
            };
            auto load = [&](int32_t at, int lane_of, int k) {
                const uint64_t i = (uint32_t)max(__shfl_sync(0xFFFFFFFFu, at, lane_of), 0);
                const uint2 *src = reinterpret_cast<const uint2 *>(from4 + i * (8 * kKv4Row));
                word[k][0] = __ldg(src);
                word[k][1] = __ldg(src + other);
                scale[k] = __ldg(from_scales + i * (8 * kKv4Scales));
            };
            int32_t at = place(0, look_up(0));
            int blk = look_up(kAtOnce);
            uint32_t gone = __ballot_sync(0xFFFFFFFFu, at == -1);   // of the tiles that are worked on
            uint32_t gone_next = gone;
            int next_lane = 0;                          // of the boxes that are loaded next
#pragma unroll
            for (int k = 0; k < kOwn; ++k)
                load(at, next_lane + k, k);
            next_lane += kOwn;
            for (int j = 0; j < u.count; ++j, ++n) {
                const uint32_t st = n % kStages;
                if (j % kAtOnce == 0)
                    gone = gone_next;
                fine = wait_phase(empty0 + 8u * st, ((n / kStages) & 1u) ^ 1u, kFaultLoad);
                fine = __all_sync(0xFFFFFFFFu, fine);
                if (!fine)
                    break;
                if (lane == 0)
                    s_gone[kFour ? st : 0][warp - kLoadWarp] =
                        (uint16_t)((gone >> (j % kAtOnce * kOwn) & ((1u << kOwn) - 1u)) << first_box);
                const uint32_t to = st * (2 * kTileBytes);
                if (next_lane == kAtOnce * kOwn) {      // the next boxes are those of tile j + 1
                    next_lane = 0;
                    at = place(j + 1, blk);
                    blk = look_up(j + 1 + kAtOnce);
                    gone_next = __ballot_sync(0xFFFFFFFFu, at == -1);
                }
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
                    const uint32_t sc = kv4_scales(scale[k] * 0x10001u), off = kv4_offsets(sc);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t w = c & 1 ? word[k][c >> 1].y : word[k][c >> 1].x;
                        st_shared_v4(chunk_at[c] + to + 1024u * k,
                                     make_uint4(fma_bf16x2(kv4_pair(w, 0), sc, off), fma_bf16x2(kv4_pair(w, 1), sc, off),
                                                fma_bf16x2(kv4_pair(w, 2), sc, off), fma_bf16x2(kv4_pair(w, 3), sc, off)));
                    }
                    load(at, next_lane + k, k);         // (past the last tile: row 0)
                }
                next_lane += kOwn;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_local(full0 + 8u * st);
            }
        }
    } else if (warp >= kLoadWarp) {
        const bool keys = warp == kLoadWarp, values = kLoaders<kQ, kFour> == 1 || !keys;
        const int boxes = kKeyTile / box;               // <= 16
        bool fine = true;
        while (fine && walk.next(a, u)) {
            const SeqOf<kWindow> &s = u.s;
            // this lane's box of tile j: its block
            auto look_up = [&](int j) -> int {
                const int p = tile_at(s, u.k0 + j) * kKeyTile + lane * box;
                return j < u.count && lane < boxes && p < s.keys
                           ? block_of(a, u.b, p) : 0;
            };
            int blk = look_up(0);
            for (int j = 0; j < u.count; ++j, ++n) {
                const uint32_t st = n % kStages, full = full0 + 8u * st;
                const int p = tile_at(s, u.k0 + j) * kKeyTile + lane * box;
                const bool mine = lane < boxes && p < s.keys;
                const int off = mine ? (int)((uint32_t)p % (uint32_t)a.block_size) : 0;
                const bool lost = mine && (blk < 0 || blk >= a.num_blocks);
                const bool bad = lost || (mine && !some_seen(a, s, p, box));
                if (lost && keys && u.unit == 0 && a.err != nullptr && first_needed(a, s, p, min(box, s.keys - p)))
                    atomicAdd(a.err, 1);                // once per block: at the first key that is needed
                fine = wait_phase(empty0 + 8u * st, ((n / kStages) & 1u) ^ 1u, kFaultLoad);
                fine = __all_sync(0xFFFFFFFFu, fine);
                if (!fine)
                    break;
                const uint32_t bads = __ballot_sync(0xFFFFFFFFu, lost), loads = __ballot_sync(0xFFFFFFFFu, mine);
                if (lane == 0) {
                    if (keys)
                        s_bad[st] = bads;
                    mbar_expect_tx(full, (uint32_t)__popc(loads) * box * (256u / kLoaders<kQ, kFour>));
                }
                __syncwarp();
                if (mine) {
                    // a block out of range, or of no row, reads zeros: one past the last
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
        if (elect_one()) {
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
            const SeqOf<kWindow> &s = u.s;
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
                for (int c = 0; c < 4; ++c) {
                    if constexpr (kFour)                // elements in the order of the loaders
                        w[c] = make_uint4(__byte_perm(w[c].x, w[c].z, 0x5410), __byte_perm(w[c].x, w[c].z, 0x7632),
                                          __byte_perm(w[c].y, w[c].w, 0x5410), __byte_perm(w[c].y, w[c].w, 0x7632));
                    st_shared_v4(dst + (uint32_t)(((4 * half + c) ^ (r & 7)) << 4), w[c]);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive_local(q_ready0 + 8u * t);
            }
            int node[2];
            int32_t begin[2];                           // of the rows' windows
            // of each row: minus the reference (log2), the maximum that asks for
            // another (-inf: none seen yet), this lane's sum
            float ref[2], limit[2], sum[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = (u.tile * kRows + 128 * t + first + (lane >> 2) + 8 * e) / a.group;
                node[e] = i < s.n ? i : -1;
                if constexpr (kWindow)
                    begin[e] = begin_of_window(a, s, node[e]);
                ref[e] = sum[e] = 0.0f;
                limit[e] = -INFINITY;
            }
            if constexpr (kWindow || kFour) {
                in_memory(node);
                in_memory(begin);
            }
            const int count = u.count, ctx = s.ctx;
            int p0 = u.k0 * kKeyTile;
            for (int j = 0; j < count; ++j, ++n, p0 += kKeyTile) {
                if constexpr (kWindow)
                    p0 = tile_at(s, u.k0 + j) * kKeyTile;
                wait_phase(s_full, n & 1u, kFaultSoftmax);
                __syncwarp();
                tc_fence_after();
                const uint32_t st = n % kStages;
                uint32_t bads;                          // boxes without keys
                if constexpr (kFour) {
                    const uint4 gone = ld_shared_v4(smem_u32(s_gone[st]));
                    bads = gone.x | gone.y | gone.z | gone.w;
                    bads = (bads | bads >> 16) & 0xFFFFu;
                } else {
                    bads = *reinterpret_cast<volatile uint32_t *>(&s_bad[st]);
                }
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
                if ((kWindow ? some_partly_seen(a, s, p0, kKeyTile) : p0 + kKeyTile > ctx) || bads != 0u) {
                    // of the four lanes of a row each finds 32 of the keys
                    uint32_t own[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        own[e] = seen32<kWindow>(a, s, node[e], p0 + 32 * (lane & 3), kWindow ? begin[e] : 0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t out = 0u;              // keys of blocks out of range
#pragma unroll 1
                        for (int k = 0; bads != 0u && k < 32; k += 8)   // (boxes of 8 keys at least)
                            out |= ((bads >> ((32 * c + k) / box)) & 1u ? 0xFFu : 0u) << k;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t see =
                                (__shfl_sync(0xFFFFFFFFu, own[e], (lane & 28) | c) & ~out) >> (2 * (lane & 3));
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int f = 0; f < 2; ++f)
                                    if (!((see >> (8 * k + f)) & 1u))
                                        y[4 * (4 * c + k) + 2 * e + f] = -INFINITY;
                        }
                    }
                    // (in 4 bits no value is infinite or NaN, nor is what lies past the end)
                    if constexpr (!kFour) {
                        // the tile's V: zeros past the end, and in place of what is
                        // not finite in keys that a row may not see.  Every row tile looks at all
                        // of it; one that finds such a value says so (the number of
                        // the piece) before it takes it out, so that the others,
                        // who may see the zero, see the word too.
                        wait_phase(full0 + 8u * st, (n / kStages) & 1u, kFaultSoftmax);    // complete: seen through S
                        const uint32_t v = sK + st * (2 * kTileBytes) + kTileBytes;
                        for (int i = threadIdx.x & 255; i < kKeyTile * 8; i += 256) {
                            const int key = p0 + (i >> 3);
                            if (!partly_seen(a, s, key))
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
            if constexpr (kFour) {
                // columns 2i and 2i + 1 of eight are elements i and i + 4
                const int from = (lane & 28) | ((2 * lane) & 3);
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const float a0 = __shfl_sync(0xFFFFFFFFu, o[k], from), a1 = __shfl_sync(0xFFFFFFFFu, o[k + 1], from);
                    const float b0 = __shfl_sync(0xFFFFFFFFu, o[k], from + 1), b1 = __shfl_sync(0xFFFFFFFFu, o[k + 1], from + 1);
                    o[k] = (lane & 2) ? a1 : a0;
                    o[k + 1] = (lane & 2) ? b1 : b0;
                }
            }
            const bool unfinite = !kFour && *reinterpret_cast<volatile uint32_t *>(&s_unfinite[piece & 7u]) == piece + 1u;
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
                        if (!kFour && unfinite) {
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
                    write_header<kRows, kWindow>(a, at, u, unfinite);
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

// Which kernel takes a call, by the average rows of a unit (only the totals are
// known on the host; any kernel is right for any unit).  8 sequences over 4096
// keys, us:
//   up to 16 rows   k5_small<1>: 16.8 at 16 rows, k5_small<2> 20.3
//   up to 32        k5_small<2>: 23.0 at 32, k5_wide<1> 25.3; at 40 28.5 and 25.6
//   up to 128       k5_wide<1>: 28.7 at 128, k5_wide<2> 35.1; at 160 39.9 and 36.3
//   beyond          k5_wide<2>
// Batches that mix them: 63 single tokens and a tree of 64 over 2000 keys 56 us (64
// single tokens 51, the tree alone 24).
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

template <int kTiles, bool kRuns, bool kWindow>
cudaError_t launch_small(const Args &a, int ctas, cudaStream_t stream, const char **why)
{
    static bool configured[64] = {};
    cudaError_t e = allow_smem(k5_small<kTiles, kRuns, kWindow>, kSmallSmem<kTiles>, configured);
    if (e != cudaSuccess)
        return e;
    *why = "attention launch";
    e = launch_pdl(k5_small<kTiles, kRuns, kWindow>, dim3((unsigned)ctas), dim3(kSmallThreads), kSmallSmem<kTiles>, stream, 1, a);
    return e != cudaSuccess ? e : launch_join<16 * kTiles, kWindow, false>(a, ctas, stream, why);
}

template <int kQ, bool kWindow, bool kFour>
cudaError_t launch_wide(const Args &a, int ctas, cudaStream_t stream, const char **why)
{
    static bool configured[64] = {};
    cudaError_t e = allow_smem(k5_wide<kQ, kWindow, kFour>, kWideSmem<kQ>, configured);
    if (e != cudaSuccess)
        return e;
    // the cache as [num_blocks, kv_heads, block_size, 128], boxes of 64 columns
    // (K or V) and the largest power of two of keys, at most a tile, in a block
    const int box = kFour ? 8 : std::min(kKeyTile, a.block_size & -a.block_size);
    CUtensorMap map = {};
    if (!kFour) {
        const uint64_t row = 2 * kHeadDim * 2;
        const cuuint64_t dims[4] = {2 * kHeadDim, (cuuint64_t)a.block_size, (cuuint64_t)a.kv_heads, (cuuint64_t)a.num_blocks};
        const cuuint64_t strides[3] = {row, row * a.block_size, row * a.block_size * a.kv_heads};
        const cuuint32_t boxes[4] = {kHeadDim, (cuuint32_t)box, 1, 1}, ones[4] = {1, 1, 1, 1};
        const EncodeTiledFn enc = encode_fn();
        *why = "tensor map of the cache could not be encoded";
        if (!enc || enc(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint16_t *>(a.cache), dims, strides, boxes,
                        ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    *why = "attention launch";
    e = launch_pdl(k5_wide<kQ, kWindow, kFour>, dim3((unsigned)ctas), dim3(kWideThreads<kQ, kFour>), kWideSmem<kQ>, stream,
                   1, map, a, box);
    return e != cudaSuccess ? e : launch_join<128 * kQ, kWindow, kFour>(a, ctas, stream, why);
}

template <bool kWindow>
cudaError_t launch_variant(Variant v, const Args &a, int ctas, cudaStream_t stream, const char **why)
{
    const bool runs = a.block_size % kChunk == 0;
    switch (v) {
    case kSmall16: return runs ? launch_small<1, true, kWindow>(a, ctas, stream, why)
                               : launch_small<1, false, kWindow>(a, ctas, stream, why);
    case kSmall32: return runs ? launch_small<2, true, kWindow>(a, ctas, stream, why)
                               : launch_small<2, false, kWindow>(a, ctas, stream, why);
    case kWide128: return launch_wide<1, kWindow, false>(a, ctas, stream, why);
    default: return launch_wide<2, kWindow, false>(a, ctas, stream, why);
    }
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
    const bool wide = v == kWide128 || v == kWide256;
    const int64_t unit_rows = v == kSmall16 ? 16 : v == kSmall32 ? 32 : v == kWide128 ? 128 : 256;
    const int ctas = plan(a, unit_rows, wide, ctas_of(v, num_sms));
    return p.window > 0 ? launch_variant<true>(v, a, ctas, stream, why) : launch_variant<false>(v, a, ctas, stream, why);
}

size_t kv4_wide_workspace(bool two, int num_sms)
{
    const Variant v = two ? kWide256 : kWide128;
    return 2 * (size_t)ctas_of(v, num_sms) * slot_floats(v) * sizeof(float);
}

cudaError_t launch_kv4_wide(const TreeAttentionLaunch &p, bool two, int num_sms, cudaStream_t stream, const char **why)
{
    Args a{};
    static_cast<TreeAttentionLaunch &>(a) = p;
    a.scale_log2 = p.scale * kLog2e;
    const int ctas = plan(a, two ? 256 : 128, true, ctas_of(two ? kWide256 : kWide128, num_sms));
    if (two)
        return p.window > 0 ? launch_wide<2, true, true>(a, ctas, stream, why) : launch_wide<2, false, true>(a, ctas, stream, why);
    return p.window > 0 ? launch_wide<1, true, true>(a, ctas, stream, why) : launch_wide<1, false, true>(a, ctas, stream, why);
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
