// K10: the accepted nodes' rows of a verified tree, moved to follow the context in
// every cache.
//
//   row(context + k) <- row(context + path[k]),  path increasing, so path[k] >= k
//
// A thread has the same 16 (or 8) bytes of every row of a path, and takes them in
// order: what it writes at k is never read later (later sources are past k), so the
// move needs no other memory and no word between threads.  Few bytes: what counts is
// the chain of loads, lengths with path, block numbers, rows: 3 trees of 13 in five
// caches 2.9 us, 64 of 64 with paths up to 12 in eight caches of 8 heads 6.1 (17 MB).
#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kThreads = 128;          // rows of a path looked up at once, too
constexpr int kBatch = 8;              // rows whose loads are in flight

template <typename V>
__device__ __forceinline__ void move_rows(const CompactLaunch &a, const int32_t *s_src, const int32_t *s_dst, int rows) {
    const int cols = a.row_bytes[blockIdx.y] / (int)sizeof(V);
    const uint32_t bs = (uint32_t)a.block_size;
    V *cache = static_cast<V *>(a.caches[blockIdx.y]);
    for (int e = threadIdx.x; e < a.heads * cols; e += kThreads) {
        const int h = e / cols, col = e - h * cols;
        auto at = [&](int32_t slot) {
            const uint32_t blk = (uint32_t)slot / bs;
            return cache + (((int64_t)blk * a.heads + h) * bs + ((uint32_t)slot - blk * bs)) * cols + col;
        };
        for (int k0 = 0; k0 < rows; k0 += kBatch) {
            V v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (k0 + i < rows && s_src[k0 + i] != s_dst[k0 + i])
                    v[i] = *at(s_src[k0 + i]);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (k0 + i < rows && s_src[k0 + i] != s_dst[k0 + i])
                    *at(s_dst[k0 + i]) = v[i];
        }
    }
}

__global__ void __launch_bounds__(kThreads)
k10_compact(const __grid_constant__ CompactLaunch a)
{
    __shared__ int32_t s_src[kThreads], s_dst[kThreads];
    __shared__ int32_t s_rows;
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x;
    const int64_t r0 = max((int64_t)0, min((int64_t)__ldg(a.row_start + b), a.rows));
    const int64_t r1 = max(r0, min((int64_t)__ldg(a.row_start + b + 1), a.rows));
    const int64_t ctx = max(__ldg(a.context_len + b), 0);
    const int len = max(0, min(__ldg(a.path_len + b), a.path_width)), nodes = (int)(r1 - r0);
    const int64_t keys = (int64_t)a.table_width * a.block_size;
    const uint32_t bs = (uint32_t)a.block_size;
    const int32_t *path = a.path + b * a.path_stride, *table = a.block_table + b * a.table_stride;
    // where logical key p lies, or -1
    auto slot_of = [&](int64_t p) -> int32_t {
        if (p >= keys)
            return -1;
        const uint32_t i = (uint32_t)p / bs;
        const int32_t blk = __ldg(table + i);
        return blk >= 0 && blk < a.num_blocks ? (int32_t)((uint32_t)blk * bs + ((uint32_t)p - i * bs)) : -1;
    };
    int done = 0;
    for (bool more = true; more && done < len;) {
        const int k = done + threadIdx.x;
        if (threadIdx.x == 0)
            s_rows = min(kThreads, len - done);
        __syncthreads();
        if (k < len) {
            const int node = __ldg(path + k), before = k > 0 ? __ldg(path + k - 1) : -1;
            int32_t src = -1, dst = -1;
            if (node > before && node >= 0 && node < nodes) {
                src = slot_of(ctx + node);
                dst = slot_of(ctx + k);
            }
            s_src[threadIdx.x] = src;
            s_dst[threadIdx.x] = dst;
            if (src < 0 || dst < 0)
                atomicMin(&s_rows, (int)threadIdx.x);
        }
        __syncthreads();
        const int rows = s_rows;
        if (a.row_bytes[blockIdx.y] % 16 == 0)
            move_rows<uint4>(a, s_src, s_dst, rows);
        else
            move_rows<uint2>(a, s_src, s_dst, rows);
        more = rows == min(kThreads, len - done);
        done += rows;
        __syncthreads();
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        if (a.new_len != nullptr)
            a.new_len[b] = (int32_t)ctx + done;
        if (done < len && a.err != nullptr)
            atomicAdd(a.err, 1);
    }
}

}  // namespace

cudaError_t launch_kv_compact(const CompactLaunch &a, cudaStream_t stream)
{
    return launch_pdl(k10_compact, dim3((unsigned)a.seqs, (unsigned)a.count), dim3(kThreads), 0, stream, 1, a);
}

}  // namespace rc
