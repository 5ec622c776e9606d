// K6: rotary positions -- the cos|sin table (scaled for long contexts) and
// its application to any heads, in interleaved pairs or halves, over all or
// the first part of a head, forward and transposed (the gradient).
//
//   (a, b) -> (a c - b s, b c + a s);  transposed: (a c + b s, b c - a s)
// in FP32 (the store's form: fma(a, c, -(b s)), fma(b, c, a s)), rounded once
// to the output's type; what lies past rot_dim is copied.
//
// Both kernels are bound by memory: one read and one write of every element
// (the table rows, shared by a token's heads, come from L1 and L2).
#include "rc_internal.cuh"

#include <algorithm>
#include <cmath>

namespace rc {

namespace {

constexpr int kThreads = 256;
constexpr int kIter = 4;               // heads per thread: loads in flight

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<uint16_t>(uint16_t v) {
    return __uint_as_float((uint32_t)v << 16);
}
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ uint16_t from_f<uint16_t>(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }

// kN elements of T; kWideOf<T> of them are the 16 bytes of one access, and the
// table's columns that go with them are 4 to 32 aligned bytes.
template <typename T, int kN>
struct alignas(sizeof(T) * kN < 16 ? sizeof(T) * kN : 16) Vec { T v[kN]; };
template <typename T> constexpr int kWideOf = 16 / (int)sizeof(T);

// kN consecutive elements, in one access (kOne) or one by one.
template <bool kOne, typename T, int kN>
__device__ __forceinline__ void get(Vec<T, kN> &d, const T *p) {
    if (kOne) {
        d = *reinterpret_cast<const Vec<T, kN> *>(p);
    } else {
#pragma unroll
        for (int j = 0; j < kN; ++j)
            d.v[j] = p[j];
    }
}
template <bool kOne, typename T, int kN>
__device__ __forceinline__ void put(T *p, const Vec<T, kN> &d) {
    if (kOne) {
        *reinterpret_cast<Vec<T, kN> *>(p) = d;
    } else {
#pragma unroll
        for (int j = 0; j < kN; ++j)
            p[j] = d.v[j];
    }
}

template <bool kInverse>
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    if (kInverse)
        s = -s;
    const float x = __fmaf_rn(a, c, -__fmul_rn(b, s));
    b = __fmaf_rn(b, c, __fmul_rn(a, s));
    a = x;
}

// One thread: one unit of kIter (token, head) rows.  A unit is kVec
// elements (pairs layout, and what is only copied) or kVec elements of each
// half (halves layout).  Consecutive threads take the units of a head, then
// the next head, so a warp reads whole rows.  kVec is 16 bytes' worth where
// every pointer, stride, width and rot_dim allows it, else one pair, element
// by element.  A narrow copied tail of odd width has kVec = 1 units, so pairs
// heads whose tail is odd are refused on the host.
template <typename T, typename C, bool kHalves, bool kInverse, int kVec>
__global__ void __launch_bounds__(kThreads)
k6_rope_apply(const RopeLaunch a)
{
    pdl_trigger();
    pdl_wait();
    constexpr bool kOne = kVec == kWideOf<T>;
    const uint32_t rotated = kHalves ? (uint32_t)a.rot / (2 * kVec) : (uint32_t)a.rot / kVec;
    const uint32_t units = rotated + (uint32_t)(a.width - a.rot) / kVec;
    const int half = a.rot / 2;
    const int64_t all = a.T * a.heads;
    const int64_t block0 = (int64_t)blockIdx.x * a.rows_per_block;
    const uint32_t lanes = (uint32_t)a.rows_per_block / kIter;       // rows side by side
    const T *x = static_cast<const T *>(a.x);
    T *out = static_cast<T *>(a.out);
    const C *table = static_cast<const C *>(a.table);
    // units of a row beyond the block's threads (wide heads) are walked
    for (uint32_t item = threadIdx.x; item < units * lanes; item += kThreads) {
        const uint32_t u = item % units, lane_row = item / units;
        const bool rot = u < rotated;
        const int at = rot ? (int)u * kVec : a.rot + (int)(u - rotated) * kVec;   // first element
        const int pair = kHalves ? at : at / 2;                                   // its table column
        Vec<T, kVec> v0[kIter], v1[kIter];
        int64_t pos[kIter], dst[kIter];
        bool live[kIter];
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            const int64_t row = block0 + lane_row + (int64_t)i * lanes;
            live[i] = row < all;
            if (!live[i])
                continue;
            // T * heads < 2^31 (checked on the host)
            const uint32_t t = (uint32_t)row / (uint32_t)a.heads, h = (uint32_t)row - t * (uint32_t)a.heads;
            const T *src = x + t * a.x_row_stride + h * a.x_head_stride + at;
            get<kOne>(v0[i], src);
            if (kHalves && rot)
                get<kOne>(v1[i], src + half);
            pos[i] = __ldg(a.positions + t);
            dst[i] = t * a.out_row_stride + h * a.out_head_stride + at;
            if (u == 0 && h == 0 && a.err != nullptr && (pos[i] < 0 || pos[i] >= a.max_position))
                atomicAdd(a.err, 1);
        }
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
            if (!live[i])
                continue;
            // a token without a table row passes through
            if (rot && pos[i] >= 0 && pos[i] < a.max_position) {
                const C *cs = table + pos[i] * a.rot + pair;
                if (kHalves) {
                    Vec<C, kVec> c, s;
                    get<kOne>(c, cs);
                    get<kOne>(s, cs + half);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        float p = to_f(v0[i].v[j]), q = to_f(v1[i].v[j]);
                        turn<kInverse>(p, q, to_f(c.v[j]), to_f(s.v[j]));
                        v0[i].v[j] = from_f<T>(p);
                        v1[i].v[j] = from_f<T>(q);
                    }
                } else {
                    constexpr int kPairs = kVec > 1 ? kVec / 2 : 1;
                    Vec<C, kPairs> c, s;
                    get<kOne>(c, cs);
                    get<kOne>(s, cs + half);
#pragma unroll
                    for (int j = 0; j + 1 < kVec; j += 2) {
                        float p = to_f(v0[i].v[j]), q = to_f(v0[i].v[j + 1]);
                        turn<kInverse>(p, q, to_f(c.v[j / 2]), to_f(s.v[j / 2]));
                        v0[i].v[j] = from_f<T>(p);
                        v0[i].v[j + 1] = from_f<T>(q);
                    }
                }
            }
            put<kOne>(out + dst[i], v0[i]);
            if (kHalves && rot)
                put<kOne>(out + dst[i] + half, v1[i]);
        }
    }
}

template <typename T, typename C, bool kHalves, bool kInverse>
cudaError_t launch_vec(RopeLaunch &a, bool wide, cudaStream_t stream)
{
    constexpr int kWide = kWideOf<T>;
    constexpr int kNarrow = kHalves ? 1 : 2;
    const int vec = wide ? kWide : kNarrow;
    const int units = (kHalves ? a.rot / (2 * vec) : a.rot / vec) + (a.width - a.rot) / vec;
    const int lanes = units >= kThreads ? 1 : kThreads / units;
    a.rows_per_block = lanes * kIter;
    const int64_t blocks = (a.T * a.heads + a.rows_per_block - 1) / a.rows_per_block;
    auto kernel = wide ? k6_rope_apply<T, C, kHalves, kInverse, kWide>
                       : k6_rope_apply<T, C, kHalves, kInverse, kNarrow>;
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, 1, a);
}

template <typename T, typename C>
cudaError_t launch_types(RopeLaunch &a, bool halves, bool inverse, bool wide, cudaStream_t stream)
{
    if (halves)
        return inverse ? launch_vec<T, C, true, true>(a, wide, stream)
                       : launch_vec<T, C, true, false>(a, wide, stream);
    return inverse ? launch_vec<T, C, false, true>(a, wide, stream)
                   : launch_vec<T, C, false, false>(a, wide, stream);
}

// ------------------------------------------------------------- the table
//
// Column j's angle is p * inv_j.  In turns that is p * (inv_j / 2 pi), of
// which only the fraction matters, so inv_j / 2 pi mod 1 is held as a 64-bit
// fixed-point fraction and p times it modulo 2^64 is exact integer
// arithmetic: its top 32 bits give the angle to 2^-32 turns at any position
// (the fraction's own rounding, 2^-65 turns times p < 2^31, stays below
// that), with no FP64 arithmetic on the GPU.
struct TableArgs {
    void *out;
    int64_t positions;
    int32_t half;                       // rot / 2
    float gain;                         // factor of every cos and sin
    uint64_t step[kMaxRotDim / 2];      // inv_j / 2 pi mod 1, times 2^64
};

template <typename C, int kVec>
__global__ void __launch_bounds__(kThreads)
k6_rope_table(const __grid_constant__ TableArgs a)
{
    pdl_trigger();
    pdl_wait();
    const uint32_t chunks = (uint32_t)a.half / kVec;
    const int64_t n = a.positions * chunks;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kThreads) {
        // positions * half < 2^31 * 256: the quotient by 64-bit division is
        // only needed past 2^32
        int64_t p;
        uint32_t c;
        if (n <= 0xFFFFFFFFll) {
            p = (uint32_t)i / chunks;
            c = (uint32_t)i - (uint32_t)p * chunks;
        } else {
            p = i / chunks;
            c = (uint32_t)(i - p * chunks);
        }
        Vec<C, kVec> co, si;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const uint64_t turns = (uint64_t)p * a.step[c * kVec + j];
            const float x = __fmul_rn((float)(int32_t)(turns >> 32), 0x1p-31f);    // half turns
            float s, k;
            sincospif(x, &s, &k);
            co.v[j] = from_f<C>(__fmul_rn(k, a.gain));
            si.v[j] = from_f<C>(__fmul_rn(s, a.gain));
        }
        C *row = static_cast<C *>(a.out) + p * 2 * a.half + c * kVec;
        put<kVec == kWideOf<C>>(row, co);
        put<kVec == kWideOf<C>>(row + a.half, si);
    }
}

}  // namespace

cudaError_t launch_rope_apply(RopeLaunch a, bool x_f32, bool table_f32, bool halves, bool inverse,
                              bool wide, cudaStream_t stream)
{
    if (x_f32)
        return table_f32 ? launch_types<float, float>(a, halves, inverse, wide, stream)
                         : launch_types<float, uint16_t>(a, halves, inverse, wide, stream);
    return table_f32 ? launch_types<uint16_t, float>(a, halves, inverse, wide, stream)
                     : launch_types<uint16_t, uint16_t>(a, halves, inverse, wide, stream);
}

cudaError_t launch_rope_table(void *out, bool f32, int64_t positions, int32_t rot, const double *inv,
                              float gain, int num_sms, cudaStream_t stream)
{
    TableArgs a{};
    a.out = out;
    a.positions = positions;
    a.half = rot / 2;
    a.gain = gain;
    for (int j = 0; j < rot / 2; ++j) {
        // inv / 2 pi in two doubles (the quotient and its remainder), so that
        // the 64-bit fraction is right to its last bits
        const double two_pi = 6.283185307179586476925, two_pi_lo = 2.4492935982947064e-16;
        const double q = inv[j] / two_pi;
        const double rest = (std::fma(-q, two_pi, inv[j]) - q * two_pi_lo) / two_pi;
        const double frac = q - std::floor(q);
        a.step[j] = (uint64_t)std::llround(std::ldexp(frac, 52)) << 12;
        // what ldexp(frac, 52) rounds off, and the remainder
        const double low = std::ldexp(frac, 52) - (double)std::llround(std::ldexp(frac, 52));
        a.step[j] += (uint64_t)(int64_t)std::llround(std::ldexp(low, 12) + std::ldexp(rest, 64));
    }
    const int half = rot / 2;
    const int size = f32 ? 4 : 2;
    const int vec = half * size % 16 == 0 ? 16 / size : 1;
    const int64_t n = positions * (half / vec);
    const int64_t blocks = std::min<int64_t>((n + kThreads - 1) / kThreads, (int64_t)num_sms * 64);
    auto kernel = f32 ? (vec > 1 ? k6_rope_table<float, 4> : k6_rope_table<float, 1>)
                      : (vec > 1 ? k6_rope_table<uint16_t, 8> : k6_rope_table<uint16_t, 1>);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, 1, a);
}

}  // namespace rc
