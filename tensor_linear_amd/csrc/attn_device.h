// Device code shared by the kernels that read a paged cache.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attn.h"

namespace tpl {
namespace {

// The sequence that owns row t of a call, by a 64-way search of cu; -1 for none.
__device__ __forceinline__ int64_t sequence_of(const CacheArgs &a, int64_t t, int lane) {
    // the number of sequences s in [0, B) with cu[s] <= t, for non-decreasing cu
    int64_t lo = 0, n = a.B;
    while (n > 0) {
        const int64_t step = (n + 63) / 64;
        const int64_t i = lo + lane * step;
        const bool below = lane * step < n && a.cu[i] <= t;
        const int c = __popcll(__ballot(below));
        if (c == 0) { n = 0; break; }
        const int64_t base = (int64_t)(c - 1) * step;      // the last such probe
        lo += base + 1;
        n = (n - base < step ? n - base : step) - 1;
    }
    const int64_t s = lo - 1;
    return s >= 0 && t < a.cu[s + 1] ? s : -1;
}

// Page and slot of position p >= 0 of a sequence whose table begins at `table`; the
// page is -1 where the position or its page is outside the cache.  Nothing read from
// the caller's arrays is used as an index before it is checked.
struct Row { int64_t page; uint32_t slot; };
__device__ __forceinline__ Row row_of(const CacheArgs &a, const int32_t *table, uint32_t p) {
    const uint32_t i = a.shift >= 0 ? p >> a.shift : p / a.page;
    Row r{-1, p - (a.shift >= 0 ? i << a.shift : i * a.page)};
    if ((int64_t)i < a.max_pages) {
        const int64_t id = table[i];
        if (id >= 0 && id < a.n_pages) r.page = id;
    }
    return r;
}

// One value of a cache: bf16 (2 bytes), fp32 (4) or int8 (1).
template <int CS>
__device__ __forceinline__ float cached(const void *p, int64_t i) {
    if (CS == 1) return (float)((const int8_t *)p)[i];
    return CS == 2 ? (float)((const __bf16 *)p)[i] : ((const float *)p)[i];
}

template <int ES>
__device__ __forceinline__ float value(const void *p, int64_t i) {
    return ES == 2 ? (float)((const __bf16 *)p)[i] : ((const float *)p)[i];
}
template <int ES>
__device__ __forceinline__ void store(void *p, int64_t i, float v) {
    if (ES == 2) ((__bf16 *)p)[i] = (__bf16)v;
    else ((float *)p)[i] = v;
}

}  // namespace
}  // namespace tpl
