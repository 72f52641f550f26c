// Launch interface of the calls that read a paged cache: attention of new tokens and
// the cache's rows as matrices.  Internal, as kernels.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tpl {

// A paged cache: row (page, slot, head) of D contiguous values at page * s_page + slot
// * s_slot + head * s_head (elements), scales likewise by ss_* where ks and vs are set
// (the cache is then int8).  Sequence s has the rows cu[s] .. cu[s + 1] - 1 of a call,
// at the positions from past[s] on; position p lies in slot p % page of cache page
// table[s * ldt + p / page].
struct CacheArgs {
    const int32_t *cu, *past, *table; int64_t ldt, B, max_pages, n_pages;
    uint32_t page;                      // positions are below 2^32 - 1, and so is this
    int32_t shift;                      // page = 1 << shift, or -1
    const void *kc, *vc; int64_t s_page, s_slot, s_head;
    const float *ks, *vs; int64_t ss_page, ss_slot, ss_head;
    int64_t T; int32_t Hkv, D;
    int32_t *bad;
};

// Attention: G query heads read one key head.  `window` keys back at most (2^62: all).
struct AttnArgs {
    CacheArgs c;
    const void *Q; int64_t ldq;
    void *O; int64_t ldo;
    float *lse; int64_t ldl;
    float scale; int64_t window;
    int32_t G;
    void *ws;
};

// Rows of the cache: K and V, either may be NULL.
struct ReadArgs {
    CacheArgs c;
    void *K, *V; int64_t ldk, ldv;
};

hipError_t launch_kv_attention(const AttnArgs &a, int elem_bytes, hipStream_t s);
hipError_t launch_kv_read(const ReadArgs &a, int elem_bytes, hipStream_t s);

// Bytes of workspace an attention of these sizes needs.
size_t attention_workspace(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D);

}  // namespace tpl
