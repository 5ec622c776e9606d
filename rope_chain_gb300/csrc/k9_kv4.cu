// K9: rows into and out of a cache in 4 bits (rc_kv4.cuh has the format).
//
//   scale = max |x| / 7 to four significant bits,  c = 8 + x / scale to the nearest
//
// Bound by memory: 256 bytes of a row's head in, 72 out, and the other way round.
// The arithmetic has to stay under some 20 instructions an element for that, hence
// the largest size as a maximum of 15-bit numbers in pairs, and one multiply-add per
// element that leaves 8 + x / scale in the low bits of an FP32 number.
#include "rc_kv4.cuh"
#include "rc_paged.cuh"

namespace rc {

namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;             // of a row's head: 8 elements each, four to a group of 32

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// The largest size that is kept, 7 * 2^100, as bf16.
constexpr uint32_t kMostValue = 0x72E0u;

// An element of a row with NaN, infinities or larger sizes, as it is stored.
__device__ __forceinline__ uint32_t tamed(uint32_t half) {
    const uint32_t size = half & 0x7FFFu;
    return size > 0x7F80u ? 0u : size > kMostValue ? (half & 0x8000u) | kMostValue : half;
}

template <int kItems>
__global__ void __launch_bounds__(kThreads)
k9_store(const __grid_constant__ Kv4StoreLaunch a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & (kLanes - 1);
    const uint32_t items = (uint32_t)a.T * (uint32_t)a.heads;
    const uint32_t first = blockIdx.x * (uint32_t)(kThreads / kLanes * kItems) + threadIdx.x / kLanes;
    const bool value = lane >= kLanes / 2;
    const uint16_t *src = value ? a.v : a.k;
    const int64_t row_stride = value ? a.v_row_stride : a.k_row_stride;
    const int64_t head_stride = value ? a.v_head_stride : a.k_head_stride;
    uint4 x[kItems];
    int64_t slot[kItems];
    uint32_t head[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t item = first + i * (kThreads / kLanes);
        const uint32_t t = item < items ? item / (uint32_t)a.heads : 0u;
        head[i] = item - t * (uint32_t)a.heads;
        slot[i] = -1;
        x[i] = make_uint4(0, 0, 0, 0);
        if (item < items) {
            slot[i] = __ldg(a.slots + t);
            x[i] = __ldcs(reinterpret_cast<const uint4 *>(src + t * row_stride + head[i] * head_stride) + (lane & 7));
        }
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        auto largest = [&] {
            uint32_t most = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                most = max_u16x2(most, w[j] & 0x7FFF7FFFu);
            return max(most & 0xFFFFu, most >> 16);
        };
        uint32_t most = largest();
        const uint32_t odd = __ballot_sync(0xFFFFFFFFu, most >= 0x7F80u);
        if (most > kMostValue) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = tamed(w[j] & 0xFFFFu) | tamed(w[j] >> 16) << 16;
            most = largest();
        }
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        // to four significant bits, ties to even
        uint32_t bits = __float_as_uint(__fdiv_rn(__uint_as_float(most << 16), 7.0f));
        bits = (bits + 0x7FFFFu + ((bits >> 20) & 1u)) & 0xFFF00000u;
        if (bits < 0x0D800000u)                          // 2^-100
            bits = 0u;
        // 1 / scale, less 2^-14 of it: a quotient that lies between two whole
        // numbers goes toward zero, any other is 2^-10 away from such a tie at least
        // (eight bits over four)
        const float per = bits == 0u ? 0.0f : __fmul_rn(__frcp_rn(__uint_as_float(bits)), 1.0f - 0x1p-14f);
        uint32_t word = 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // 1.5 * 2^23 + 8: the sum's unit is 1, its low bits 8 + the whole number
            const uint32_t lo = __float_as_uint(__fmaf_rn(bf16_lo(w[j]), per, 12582920.0f));
            const uint32_t hi = __float_as_uint(__fmaf_rn(bf16_hi(w[j]), per, 12582920.0f));
            word |= (lo & 15u) << (8 * j) | (hi & 15u) << (8 * j + 4);
        }
        // the row's four scales in one lane
        const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, bits, 4);
        const uint32_t two = (bits >> 16) | (next & 0xFFFF0000u);
        const uint32_t far = __shfl_down_sync(0xFFFFFFFFu, two, 8);
        if (slot[i] < 0)
            continue;
        if (slot[i] >= a.capacity) {
            if (lane == 0 && head[i] == 0 && a.err != nullptr)
                atomicAdd(a.err, 1);
            continue;
        }
        const uint32_t s = (uint32_t)slot[i], blk = s / (uint32_t)a.block_size;      // capacity < 2^31
        const int64_t row = ((int64_t)blk * a.heads + head[i]) * a.block_size + (s - blk * (uint32_t)a.block_size);
        reinterpret_cast<uint32_t *>(a.cache4)[row * (kKv4Row / 4) + lane] = word;
        if (lane == 0) {
            *reinterpret_cast<uint2 *>(a.scales + row * kKv4Scales) = make_uint2(two, far);
            if (((odd >> (threadIdx.x & 16)) & 0xFFFFu) != 0u && a.err != nullptr)
                atomicAdd(a.err, 1);
        }
    }
}

template <int kItems>
__global__ void __launch_bounds__(kThreads)
k9_load(const __grid_constant__ Kv4LoadLaunch a)
{
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & (kLanes - 1);
    const uint32_t items = (uint32_t)a.T * (uint32_t)a.heads;
    const uint32_t first = blockIdx.x * (uint32_t)(kThreads / kLanes * kItems) + threadIdx.x / kLanes;
    uint32_t word[kItems], scale[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t item = first + i * (kThreads / kLanes);
        word[i] = scale[i] = 0u;
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
        word[i] = __ldg(reinterpret_cast<const uint32_t *>(a.cache4) + row * (kKv4Row / 4) + lane);
        scale[i] = __ldg(a.scales + row * kKv4Scales + (lane >> 2));
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t item = first + i * (kThreads / kLanes);
        if (item >= items)
            break;
        const uint32_t s = kv4_scales(scale[i] | scale[i] << 16), o = kv4_offsets(s);
        uint32_t v[4];                                   // elements (i, i + 4)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            v[j] = fma_bf16x2(kv4_pair(word[i], j), s, o);
        __stcs(reinterpret_cast<uint4 *>(a.out) + (int64_t)item * kLanes + lane,
               make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                          __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632)));
    }
}

// Several rows a thread where they fill the GPU; else one, for latency.
template <typename Launch>
cudaError_t launch_rows(void (*one)(Launch), void (*many)(Launch), const Launch &a, int num_sms, cudaStream_t stream)
{
    constexpr int kRows = kThreads / kLanes, kMany = 4;
    const int64_t items = a.T * a.heads;
    const bool more = items >= (int64_t)num_sms * 8 * kRows * kMany;
    const int64_t per = kRows * (more ? kMany : 1);
    return launch_pdl(more ? many : one, dim3((unsigned)((items + per - 1) / per)), dim3(kThreads), 0, stream, 1, a);
}

}  // namespace

cudaError_t launch_kv4_store(const Kv4StoreLaunch &a, int num_sms, cudaStream_t stream)
{
    return launch_rows<Kv4StoreLaunch>(k9_store<1>, k9_store<4>, a, num_sms, stream);
}

cudaError_t launch_kv4_load(const Kv4LoadLaunch &a, int num_sms, cudaStream_t stream)
{
    return launch_rows<Kv4LoadLaunch>(k9_load<1>, k9_load<4>, a, num_sms, stream);
}

}  // namespace rc
