// K9: rows into and out of a cache in 4 bits (rc_kv4.cuh has the format).
//
//   scale = max |x| / 7 to four significant bits,  c = 8 + x / scale to the nearest
//
// Bound by memory: 256 bytes of a row's head in, 72 out, and the other way round.
// The store's arithmetic has to stay under some 14 instructions an element for that: a
// lane has a whole group of 32 elements, so a scale's division is made once; the largest
// size is a maximum of 15-bit numbers in pairs; an element is unpacked, multiplied and
// added in one go so that 8 + x / scale stands in the low bits of an FP32 number, and
// joined to its word by one integer multiply-add.  Measured, 131072 rows of 8 heads: the
// store 52 us, 6.6 TB/s (eight elements a lane, four lanes to a group: 102), the load 57,
// 6.1 TB/s; 39 rows 1.8 and 1.5.
#include "rc_kv4.cuh"
#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 8;              // of a row's head that is loaded: 16 elements each

// The largest size that is kept, 7 * 2^100, as bf16.
constexpr uint32_t kMostValue = 0x72E0u;

// An element of a row with NaN, infinities or larger sizes, as it is stored.
__device__ __forceinline__ uint32_t tamed(uint32_t half) {
    const uint32_t size = half & 0x7FFFu;
    return size > 0x7F80u ? 0u : size > kMostValue ? (half & 0x8000u) | kMostValue : half;
}

constexpr int kGroups = 4;             // of a row's head: K's two and V's two, a lane each

__global__ void __launch_bounds__(kThreads)
k9_store(const __grid_constant__ Kv4StoreLaunch a)
{
    pdl_trigger();
    pdl_wait();
    const int q = threadIdx.x & (kGroups - 1);
    const uint32_t items = (uint32_t)a.T * (uint32_t)a.heads;
    const uint32_t item = blockIdx.x * (uint32_t)(kThreads / kGroups) + threadIdx.x / kGroups;
    const uint32_t t = item < items ? item / (uint32_t)a.heads : 0u, head = item - t * (uint32_t)a.heads;
    uint32_t w[16];
    int64_t slot = -1;
    if (item < items) {
        slot = __ldg(a.slots + t);
        const uint16_t *const src = (q >= 2 ? a.v : a.k) + 32 * (q & 1);
        const int64_t row_stride = q >= 2 ? a.v_row_stride : a.k_row_stride;
        const int64_t head_stride = q >= 2 ? a.v_head_stride : a.k_head_stride;
        const uint4 *from = reinterpret_cast<const uint4 *>(src + t * row_stride + head * head_stride);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 x = __ldg(from + j);
            w[4 * j] = x.x;
            w[4 * j + 1] = x.y;
            w[4 * j + 2] = x.z;
            w[4 * j + 3] = x.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            w[j] = 0u;
    }
    auto largest = [&] {
        uint32_t most[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 16; ++j)
            most[j & 1] = __vmaxu2(most[j & 1], w[j] & 0x7FFF7FFFu);
        most[0] = __vmaxu2(most[0], most[1]);
        return max(most[0] & 0xFFFFu, most[0] >> 16);
    };
    uint32_t most = largest();
    const uint32_t odd = __ballot_sync(0xFFFFFFFFu, most >= 0x7F80u);
    if (most > kMostValue) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
            w[j] = tamed(w[j] & 0xFFFFu) | tamed(w[j] >> 16) << 16;
        most = largest();
    }
    // to four significant bits, ties to even
    uint32_t bits = __float_as_uint(__fdiv_rn(__uint_as_float(most << 16), 7.0f));
    bits = (bits + 0x7FFFFu + ((bits >> 20) & 1u)) & 0xFFF00000u;
    if (bits < 0x0D800000u)                              // 2^-100
        bits = 0u;
    // 1 / scale, less 2^-14 of it: a quotient that lies between two whole numbers goes
    // toward zero, any other is 2^-10 away from such a tie at least (eight bits over four)
    const float per = bits == 0u ? 0.0f : __fmul_rn(__frcp_rn(__uint_as_float(bits)), 1.0f - 0x1p-14f);
    // 1.5 * 2^23 + 8: the sum's unit is 1, so its bits are those of 1.5 * 2^23 plus 8 + the
    // whole number; what 16 times and add leaves of the former is taken off
    constexpr uint32_t kOnes = 0x11111111u * 0x4B400000u;
    uint32_t word[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t sum = 0u;
#pragma unroll
        for (int e = 3; e >= 0; --e) {
            float lo = bf16_lo(w[4 * j + e]), hi = bf16_hi(w[4 * j + e]);
            fma2_rn(lo, hi, per, per, 12582920.0f, 12582920.0f);
            sum = sum * 16u + __float_as_uint(hi);
            sum = sum * 16u + __float_as_uint(lo);
        }
        word[j] = sum - kOnes;
    }
    // the row's four scales in one lane
    const uint32_t two = (bits >> 16) | (__shfl_down_sync(0xFFFFFFFFu, bits, 1) & 0xFFFF0000u);
    const uint32_t far = __shfl_down_sync(0xFFFFFFFFu, two, 2);
    if (slot < 0)
        return;
    if (slot >= a.capacity) {
        if (q == 0 && head == 0 && a.err != nullptr)
            atomicAdd(a.err, 1);
        return;
    }
    const uint32_t s = (uint32_t)slot, blk = s / (uint32_t)a.block_size;         // capacity < 2^31
    const int64_t row = ((int64_t)blk * a.heads + head) * a.block_size + (s - blk * (uint32_t)a.block_size);
    reinterpret_cast<uint4 *>(a.cache4)[row * kGroups + q] = make_uint4(word[0], word[1], word[2], word[3]);
    if (q == 0) {
        *reinterpret_cast<uint2 *>(a.scales + row * kKv4Scales) = make_uint2(two, far);
        if (((odd >> (threadIdx.x & 28)) & 15u) != 0u && a.err != nullptr)
            atomicAdd(a.err, 1);
    }
}

// kWhole: 32 bytes of a row are stored at once, whole sectors (131072 rows of 8 heads,
// 344 MB: 57 us, 6.1 TB/s; in two stores of 16 bytes 69 us).
template <int kItems, bool kWhole>
__global__ void __launch_bounds__(kThreads)
k9_load(const __grid_constant__ Kv4LoadLaunch a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & (kLanes - 1);
    const uint32_t items = (uint32_t)a.T * (uint32_t)a.heads;
    const uint32_t first = blockIdx.x * (uint32_t)(kThreads / kLanes * kItems) + threadIdx.x / kLanes;
    uint2 word[kItems];
    uint32_t scale[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t item = first + i * (kThreads / kLanes);
        word[i] = make_uint2(0u, 0u);
        scale[i] = 0u;
        if (item >= items)
            continue;
        const uint32_t t = item / (uint32_t)a.heads, head = item - t * (uint32_t)a.heads;
        const int64_t slot = __ldg(a.slots + t);
        if (slot >= a.capacity && lane == 0 && head == 0 && a.err != nullptr)
            atomicAdd(a.err, 1);
        if (slot < 0 || slot >= a.capacity)
            continue;
        const uint32_t s = (uint32_t)slot, blk = s / (uint32_t)a.block_size;
        const int64_t row = ((int64_t)blk * a.heads + head) * a.block_size + (s - blk * (uint32_t)a.block_size);
        word[i] = __ldg(reinterpret_cast<const uint2 *>(a.cache4) + row * (kKv4Row / 8) + lane);
        scale[i] = __ldg(a.scales + row * kKv4Scales + (lane >> 1));
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t item = first + i * (kThreads / kLanes);
        if (item >= items)
            break;
        const uint32_t s = kv4_scales(scale[i] * 0x10001u), o = kv4_offsets(s);
        uint32_t y[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v[4];                               // elements (i, i + 4)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = fma_bf16x2(kv4_pair(h ? word[i].y : word[i].x, j), s, o);
            y[4 * h] = __byte_perm(v[0], v[1], 0x5410);
            y[4 * h + 1] = __byte_perm(v[2], v[3], 0x5410);
            y[4 * h + 2] = __byte_perm(v[0], v[1], 0x7632);
            y[4 * h + 3] = __byte_perm(v[2], v[3], 0x7632);
        }
        uint4 *to = reinterpret_cast<uint4 *>(a.out) + ((int64_t)item * kLanes + lane) * 2;
        if constexpr (kWhole) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                         ::"l"(to), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                         : "memory");
        } else {
            to[0] = make_uint4(y[0], y[1], y[2], y[3]);
            to[1] = make_uint4(y[4], y[5], y[6], y[7]);
        }
    }
}

// Four rows a thread where they fill the GPU; else one, for latency.
template <bool kWhole> cudaError_t launch_load(const Kv4LoadLaunch &a, int num_sms, cudaStream_t stream)
{
    constexpr int kRows = kThreads / kLanes, kMany = 4;
    const int64_t items = a.T * a.heads;
    const bool more = items >= (int64_t)num_sms * 8 * kRows * kMany;
    const int64_t per = kRows * (more ? kMany : 1);
    return launch_pdl(more ? k9_load<kMany, kWhole> : k9_load<1, kWhole>, dim3((unsigned)((items + per - 1) / per)), dim3(kThreads), 0,
                      stream, 1, a);
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4StoreLaunch &a, cudaStream_t stream)
{
    constexpr int kRows = kThreads / kGroups;
    return launch_pdl(k9_store, dim3((unsigned)((a.T * a.heads + kRows - 1) / kRows)), dim3(kThreads), 0, stream, 1, a);
}

cudaError_t launch_kv4_load(const Kv4LoadLaunch &a, int num_sms, cudaStream_t stream)
{
    return reinterpret_cast<uintptr_t>(a.out) % 32 != 0 ? launch_load<false>(a, num_sms, stream)
                                                        : launch_load<true>(a, num_sms, stream);
}

}  // namespace rc
