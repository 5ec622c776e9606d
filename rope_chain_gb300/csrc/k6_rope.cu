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
#include "rc_draft.cuh"

#include <algorithm>
#include <cmath>

namespace rc {

namespace {

constexpr int kThreads = 256;

// kN elements of T as 32-bit words (bf16 in pairs): 16 bytes at a time for
// kOne accesses (4 or 8 for the table columns that go with fewer elements),
// else element by element.
template <typename T> constexpr int kWideOf = 16 / (int)sizeof(T);

template <typename T, int kN> struct Run {
    static constexpr int kWords = (int)sizeof(T) * kN >= 4 ? (int)sizeof(T) * kN / 4 : 1;
    uint32_t w[kWords];

    template <bool kOne, bool kStream = false> __device__ __forceinline__ void get(const T *p) {
        if (kOne && kWords % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 *q = reinterpret_cast<const uint4 *>(p) + i, v = kStream ? __ldcs(q) : *q;
                w[4 * i] = v.x;
                w[(4 * i + 1) % kWords] = v.y;
                w[(4 * i + 2) % kWords] = v.z;
                w[(4 * i + 3) % kWords] = v.w;
            }
        } else if (kOne && kWords == 2) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x;
            w[kWords - 1] = v.y;
        } else if (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                w[i % kWords] = reinterpret_cast<const uint32_t *>(p)[i];
        } else {
#pragma unroll
            for (int i = 0; i < kN; i += 2)
                w[i / 2] = (uint32_t)reinterpret_cast<const uint16_t *>(p)[i] |
                           (i + 1 < kN ? (uint32_t)reinterpret_cast<const uint16_t *>(p)[i + 1] << 16 : 0u);
        }
    }
    template <bool kOne, bool kStream = false> __device__ __forceinline__ void put(T *p) const {
        if (kOne && kWords % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = make_uint4(w[4 * i], w[(4 * i + 1) % kWords], w[(4 * i + 2) % kWords],
                                           w[(4 * i + 3) % kWords]);
                if (kStream)
                    __stcs(reinterpret_cast<uint4 *>(p) + i, v);
                else
                    reinterpret_cast<uint4 *>(p)[i] = v;
            }
        } else if (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                reinterpret_cast<uint32_t *>(p)[i] = w[i % kWords];
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                reinterpret_cast<uint16_t *>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
        }
    }
    __device__ __forceinline__ float at(int i) const {
        if (sizeof(T) == 4)
            return __uint_as_float(w[i % kWords]);
        return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
    // Elements i and i + 1 (i even), or the only one.
    __device__ __forceinline__ void set2(int i, float lo, float hi) {
        if (sizeof(T) == 4) {
            w[i % kWords] = __float_as_uint(lo);
            if (kN > 1)
                w[(i + 1) % kWords] = __float_as_uint(hi);
        } else {
            w[i / 2] = pack_bf16x2(lo, hi);
        }
    }
};

template <bool kInverse>
__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    if (kInverse)
        s = -s;
    const float x = __fmaf_rn(a, c, -__fmul_rn(b, s));
    b = __fmaf_rn(b, c, __fmul_rn(a, s));
    a = x;
}

// One thread: one unit of kHeads consecutive heads of one token.  A unit is
// kVec elements (pairs layout, and what is only copied) or kVec elements of
// each half (halves layout), so its table columns are read once for all the
// heads.  Consecutive threads take the units of a head, then the next group of
// heads, then the next token.  Work of several heads per thread is larger than a
// few MB and passes the caches by (evict first), or it would drive its own table
// out: 32768 x 16 heads of 128, halves, forward and transposed, 105 us without
// the hints, 93 with them, 88 with five blocks on an SM instead of four (6.1 TB/s;
// the pairs' four loads per thread want the registers of four: 17.2 us for
// 32768 x 16 heads of 64, with five 18.3; FP32, 32768 x 16 heads of 128: 76.5 us a
// direction in either layout, 7.0 TB/s).  kVec is 16 bytes' worth where every pointer,
// stride, width and rot_dim allows it, else one pair, element by element (a
// copied tail of odd width in the pairs layout is refused on the host).
template <typename T, typename C, bool kHalves, bool kInverse, int kVec, int kHeads>
__global__ void __launch_bounds__(kThreads, kHalves && kHeads > 1 ? 5 : 4)
k6_rope_apply(const __grid_constant__ RopeLaunch a)
{
    pdl_trigger();
    pdl_wait();
    constexpr bool kOne = kVec == kWideOf<T>, kStream = kHeads > 1;
    const uint32_t rotated = kHalves ? (uint32_t)a.rot / (2 * kVec) : (uint32_t)a.rot / kVec;
    const uint32_t units = rotated + (uint32_t)(a.width - a.rot) / kVec;
    const uint32_t groups = ((uint32_t)a.heads + kHeads - 1) / kHeads;
    const int half = a.rot / 2;
    // a block's threads are `units` wide (heads of more units than threads are
    // walked) and take whole (token, group) items
    const uint32_t side = max(1u, kThreads / units);
    for (uint32_t i = threadIdx.x; i < units * side; i += kThreads) {
        const uint32_t u = i % units;
        const int64_t item = (int64_t)blockIdx.x * side + i / units;
        if (item >= a.T * groups)
            break;
        // T * heads < 2^31 (checked on the host)
        const uint32_t t = (uint32_t)item / groups, h0 = ((uint32_t)item - t * groups) * kHeads;
        const bool rot = u < rotated;
        const int at = rot ? (int)u * kVec : a.rot + (int)(u - rotated) * kVec;   // first element
        const int pair = kHalves ? at : at / 2;                                   // its table column
        const T *src = static_cast<const T *>(a.x) + t * a.x_row_stride + h0 * a.x_head_stride + at;
        T *dst = static_cast<T *>(a.out) + t * a.out_row_stride + h0 * a.out_head_stride + at;
        const int64_t pos = __ldg(a.positions + t);
        Run<T, kVec> v0[kHeads], v1[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
            if (h0 + k < (uint32_t)a.heads) {
                v0[k].template get<kOne, kStream>(src + k * a.x_head_stride);
                if (kHalves && rot)
                    v1[k].template get<kOne, kStream>(src + k * a.x_head_stride + half);
            }
        // a token without a table row passes through
        const bool bad = pos < 0 || pos >= a.max_position;
        if (bad && u == 0 && h0 == 0 && a.err != nullptr)
            atomicAdd(a.err, 1);
        if (rot && !bad) {
            constexpr int kPairs = kHalves ? kVec : (kVec > 1 ? kVec / 2 : 1);
            const C *cs = static_cast<const C *>(a.table) + pos * a.rot + pair;
            Run<C, kPairs> c, s;
            c.template get<kOne>(cs);
            s.template get<kOne>(cs + half);
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {
                if (kHalves) {
#pragma unroll
                    for (int j = 0; j < kVec; j += 2) {
                        const int j1 = kVec > 1 ? j + 1 : j;
                        float p0 = v0[k].at(j), q0 = v1[k].at(j), p1 = v0[k].at(j1), q1 = v1[k].at(j1);
                        turn<kInverse>(p0, q0, c.at(j), s.at(j));
                        turn<kInverse>(p1, q1, c.at(j1), s.at(j1));
                        v0[k].set2(j, p0, p1);
                        v1[k].set2(j, q0, q1);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j + 1 < kVec; j += 2) {
                        float p = v0[k].at(j), q = v0[k].at(j + 1);
                        turn<kInverse>(p, q, c.at(j / 2), s.at(j / 2));
                        v0[k].set2(j, p, q);
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
            if (h0 + k < (uint32_t)a.heads) {
                v0[k].template put<kOne, kStream>(dst + k * a.out_head_stride);
                if (kHalves && rot)
                    v1[k].template put<kOne, kStream>(dst + k * a.out_head_stride + half);
            }
    }
}

template <typename T, typename C, bool kHalves, bool kInverse>
cudaError_t launch_vec(const RopeLaunch &a, bool wide, int num_sms, cudaStream_t stream)
{
    constexpr int kWide = kWideOf<T>;
    constexpr int kNarrow = kHalves ? 1 : 2;
    const int vec = wide ? kWide : kNarrow;
    const int64_t units = (kHalves ? a.rot / (2 * vec) : a.rot / vec) + (a.width - a.rot) / vec;
    // four loads in flight per thread (the heads that share them share the
    // table's columns; eight for halves, in either number of blocks: 94 and 118
    // us in place of 88); with less work than fills the GPU that way, one head
    // per thread
    constexpr int kMany = kHalves ? 2 : 4;
    const bool many = wide && a.heads >= kMany && a.T * a.heads * units >= (int64_t)kMany * num_sms * 1024;
    const int64_t items = a.T * (many ? (a.heads + kMany - 1) / kMany : a.heads);
    const int64_t side = std::max<int64_t>(1, kThreads / units);
    auto kernel = many ? k6_rope_apply<T, C, kHalves, kInverse, kWide, kMany>
                       : (wide ? k6_rope_apply<T, C, kHalves, kInverse, kWide, 1>
                               : k6_rope_apply<T, C, kHalves, kInverse, kNarrow, 1>);
    return launch_pdl(kernel, dim3((unsigned)((items + side - 1) / side)), dim3(kThreads), 0, stream, 1, a);
}

template <typename T, typename C>
cudaError_t launch_types(const RopeLaunch &a, bool halves, bool inverse, bool wide, int num_sms,
                         cudaStream_t stream)
{
    if (halves)
        return inverse ? launch_vec<T, C, true, true>(a, wide, num_sms, stream)
                       : launch_vec<T, C, true, false>(a, wide, num_sms, stream);
    return inverse ? launch_vec<T, C, false, true>(a, wide, num_sms, stream)
                   : launch_vec<T, C, false, false>(a, wide, num_sms, stream);
}

// ------------------------------------------------------------- the table
//
// Column j's angle is p * inv_j.  In turns that is p * (inv_j / 2 pi), of
// which only the fraction matters, so inv_j / 2 pi mod 1 is held as a 64-bit
// fixed-point fraction and p times it modulo 2^64 is exact integer
// arithmetic: its top 32 bits give the angle to 2^-32 turns at any position
// (the fraction's own rounding, 2^-65 turns times p < 2^31, stays below
// that), with no FP64 arithmetic on the GPU.  As an FP32 number the angle is off
// by up to 2^-26 turns, 1.6 * 2^-24 of cos and sin: absolute, so near a zero of
// theirs the relative error is larger.
struct TableArgs {
    void *out;
    int64_t positions;
    int32_t half;                       // rot / 2
    float gain;                         // factor of every cos and sin
    uint64_t step[kMaxRotDim / 2];      // inv_j / 2 pi mod 1, times 2^64
};

// cos and sin of p times column j's angle.
__device__ __forceinline__ void cos_sin_at(uint64_t step, uint64_t p, float &c, float &s) {
    sincospif(__fmul_rn((float)(int32_t)((p * step) >> 32), 0x1p-31f), &s, &c);     // of half turns
}

// FP32 tables: every entry from its own angle (131072 positions of 64 columns, 34
// MB: 10.9 us, 3.1 TB/s, bound by that arithmetic), within 2^-21 times the gain.
template <int kVec>
__global__ void __launch_bounds__(kThreads)
k6_rope_table_f32(const __grid_constant__ TableArgs a)
{
    pdl_trigger();
    pdl_wait();
    const uint32_t chunks = (uint32_t)a.half / kVec;
    const int64_t n = a.positions * chunks;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t p = n <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / chunks) : i / chunks;
        const uint32_t c = (uint32_t)(i - p * chunks);
        Run<float, kVec> co, si;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            float k, s;
            cos_sin_at(a.step[c * kVec + j], (uint64_t)p, k, s);
            co.w[j] = __float_as_uint(__fmul_rn(k, a.gain));
            si.w[j] = __float_as_uint(__fmul_rn(s, a.gain));
        }
        float *row = static_cast<float *>(a.out) + p * 2 * a.half + c * kVec;
        co.template put<kVec == kWideOf<float>>(row);
        si.template put<kVec == kWideOf<float>>(row + a.half);
    }
}

// bf16 tables: a sine and cosine of its own take a thread some 40 instructions,
// four times what the stores allow, so a thread makes them for one of kStep
// positions and turns that one by the block's table of the first kStep - 1
// steps (cos(x + y) = cos x cos y - sin x sin y): each entry has two angles' errors
// and two more FP32 roundings, within 2^-20 times the gain together, against
// bf16's 2^-8 of the entry.  131072 positions of 64 columns (17 MB):
// 5.0 us, 3.3 TB/s with the launch, every entry from its own angle 7.4.
constexpr int kStep = 4;
template <int kVec>
__global__ void __launch_bounds__(kThreads)
k6_rope_table_bf16(const __grid_constant__ TableArgs a)
{
    extern __shared__ float s_turn[];                   // [kStep][2][half]: cos and sin of k steps, without the gain
    for (int i = threadIdx.x; i < a.half * kStep; i += kThreads) {
        const int k = i / a.half, j = i - k * a.half;
        cos_sin_at(a.step[j], (uint64_t)k, s_turn[2 * k * a.half + j], s_turn[(2 * k + 1) * a.half + j]);
    }
    __syncthreads();
    pdl_trigger();
    pdl_wait();
    const uint32_t chunks = (uint32_t)a.half / kVec;
    const int64_t groups = (a.positions + kStep - 1) / kStep, n = groups * chunks;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * kThreads) {
        const int64_t g = n <= 0xFFFFFFFFll ? (int64_t)((uint32_t)i / chunks) : i / chunks;
        const uint32_t c = (uint32_t)(i - g * chunks);
        const int64_t p0 = g * kStep;
        float c0[kVec], s0[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            cos_sin_at(a.step[c * kVec + j], (uint64_t)p0, c0[j], s0[j]);
            c0[j] = __fmul_rn(c0[j], a.gain);
            s0[j] = __fmul_rn(s0[j], a.gain);
        }
        uint16_t *row = static_cast<uint16_t *>(a.out) + p0 * 2 * a.half + c * kVec;
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            if (p0 + k >= a.positions)
                break;
            Run<uint16_t, kVec> co, si;
#pragma unroll
            for (int j = 0; j < kVec; j += 2) {
                float x[2] = {0.0f, 0.0f}, y[2] = {0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < (kVec > 1 ? 2 : 1); ++e) {
                    const float *t = s_turn + 2 * k * a.half + c * kVec + j + e;
                    x[e] = __fmaf_rn(c0[j + e], t[0], -__fmul_rn(s0[j + e], t[a.half]));
                    y[e] = __fmaf_rn(s0[j + e], t[0], __fmul_rn(c0[j + e], t[a.half]));
                }
                co.set2(j, x[0], x[1]);
                si.set2(j, y[0], y[1]);
            }
            co.template put<kVec == kWideOf<uint16_t>>(row);
            si.template put<kVec == kWideOf<uint16_t>>(row + a.half);
            row += 2 * a.half;
        }
    }
}

}  // namespace

cudaError_t launch_rope_apply(const RopeLaunch &a, bool x_f32, bool table_f32, bool halves, bool inverse,
                              bool wide, int num_sms, cudaStream_t stream)
{
    if (x_f32)
        return table_f32 ? launch_types<float, float>(a, halves, inverse, wide, num_sms, stream)
                         : launch_types<float, uint16_t>(a, halves, inverse, wide, num_sms, stream);
    return table_f32 ? launch_types<uint16_t, float>(a, halves, inverse, wide, num_sms, stream)
                     : launch_types<uint16_t, uint16_t>(a, halves, inverse, wide, num_sms, stream);
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
    const int vec = half % (f32 ? 4 : 8) == 0 ? (f32 ? 4 : 8) : 1;
    const int64_t n = (f32 ? positions : (positions + kStep - 1) / kStep) * (half / vec);
    const int64_t blocks = std::min<int64_t>((n + kThreads - 1) / kThreads, (int64_t)num_sms * 64);
    auto kernel = f32 ? (vec > 1 ? k6_rope_table_f32<4> : k6_rope_table_f32<1>)
                      : (vec > 1 ? k6_rope_table_bf16<8> : k6_rope_table_bf16<1>);
    const size_t smem = f32 ? 0 : (size_t)half * kStep * 2 * sizeof(float);
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kThreads), smem, stream, 1, a);
}

}  // namespace rc
