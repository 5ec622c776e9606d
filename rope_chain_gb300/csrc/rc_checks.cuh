// Host-side helpers of the C ABI's files for the drafted tokens and the paged
// caches (rc_draft.cu, rc_paged.cu): statuses with messages, alignment and
// overlap of operands.
#pragma once
#include "rope_chain.h"
#include "rc_internal.cuh"

#include <cstdarg>
#include <cstdio>
#include <initializer_list>

namespace rc {

inline rc_status fail(rc_status s, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    set_last_error(msg);
    return s;
}

inline rc_status ok() {
    set_last_error("");
    return RC_OK;
}

inline rc_status cuda_fail(cudaError_t e, const char *what) {
    return fail(RC_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Bytes that a call touches (none without an address).
struct Span {
    const void *p;
    size_t n;
};

inline bool overlap(const Span &written, std::initializer_list<Span> others) {
    for (const Span &o : others)
        if (written.p && o.p && written.n > 0 && o.n > 0 && overlap(written.p, written.n, o.p, o.n))
            return true;
    return false;
}

inline int num_sms_current() {
    static int cache[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 0;
    if (dev < 64 && cache[dev])
        return cache[dev];
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    if (dev < 64)
        cache[dev] = n;
    return n;
}

inline int size_of(int32_t dtype) { return dtype == RC_F32 ? 4 : 2; }

// Strides are kept below 2^40 elements and counts below 2^31, so that byte
// spans stay far from overflowing.
constexpr int64_t kMaxStride = 1LL << 40;

// A view [T, heads, width] with strides in elements (those of an axis of length one
// are taken as 0): the elements from the first to the last, and whether no two of
// them share a place.
struct HeadsView {
    int64_t T, row_stride, head_stride;
    int32_t heads, width;
    int64_t elements() const { return (T - 1) * row_stride + (heads - 1) * head_stride + width; }
    bool distinct() const {
        const int64_t all_heads = (heads - 1) * head_stride + width, all_tokens = (T - 1) * row_stride + width;
        return ((heads == 1 || head_stride >= width) && (T == 1 || row_stride >= all_heads)) ||
               ((T == 1 || row_stride >= width) && (heads == 1 || head_stride >= all_tokens));
    }
};

inline HeadsView heads_view(int64_t T, int64_t row_stride, int64_t head_stride, int32_t heads, int32_t width) {
    return {T, T == 1 ? 0 : row_stride, heads == 1 ? 0 : head_stride, heads, width};
}

}  // namespace rc
