// kv.hpp -- the paged 8-bit key/value cache as the kernels see it, and the
// host checks its entry points share.
#pragma once

#include <hip/hip_runtime.h>

#include "ctx.hpp"
#include "device.hpp"

namespace linrec {

// k: [pages][H][P][D] e4m3 codes, v: [pages][H][D][P], scales [pages][H].
struct KvCache {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    const int* table;
    int64_t table_stride;
    int pages, shift, max_pages, H;   // page = 1 << shift tokens
};

// A sequence's new tokens in a call of T: they follow `past` tokens, n of them
// are there; positions stay below 2^31 - 1.
struct Span {
    int past, n;
    __device__ __forceinline__ Span(const int* past_, const int* n_new, int b, int T)
    {
        const int p = past_[b];
        past = max(p, 0);
        n = n_new ? min(max(n_new[b], 0), T) : T;
        n = p < 0 ? 0 : min(n, 0x7fffffff - past);
    }
};

// The page of a sequence's token block, -1 if there is none.
__device__ __forceinline__ int page_of(const KvCache& c, int b, int block)
{
    if (block < 0 || block >= c.max_pages)
        return -1;
    const int p = c.table[b * c.table_stride + block];
    return p >= 0 && p < c.pages ? p : -1;
}

inline linrec_status check_kv(const linrec_kv_cache* c, int32_t B, int32_t T)
{
    if (!c)
        return LINREC_E_NULL;
    if (B < 1 || B > 32767 || T < 0 || T > LINREC_MAX_T || c->H < 1 || c->H > 65535 ||
        (c->D != 64 && c->D != 128) || c->pages < 1 || c->max_pages < 1 ||
        (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) ||
        (int64_t)c->max_pages * c->page > LINREC_MAX_T)
        return LINREC_E_SHAPE;
    // sizes are known without the pointers (workspace queries stop here)
    return LINREC_OK;
}

inline linrec_status check_kv_ptrs(const linrec_kv_cache* c, int32_t B, const int32_t* past,
                                   const int32_t* n_new)
{
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->table || !past)
        return LINREC_E_NULL;
    if (B > 1 && c->table_stride < 0)
        return LINREC_E_LAYOUT;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
        !aligned(c->table, 4) || !aligned(past, 4) || !aligned(n_new, 4))
        return LINREC_E_ALIGN;
    return LINREC_OK;
}

inline KvCache kv_arg(const linrec_kv_cache* c)
{
    return KvCache{(uint8_t*)c->k, (uint8_t*)c->v, c->k_scale, c->v_scale, c->table, c->table_stride,
                   c->pages, __builtin_ctz(c->page), c->max_pages, c->H};
}

}  // namespace linrec
