// The paged K/V cache's device view and handle, shared by clk_cache.cu and
// the attention kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "clk.h"
#include "clk_host.h"

namespace clk {

// Workspace (see clk_cache_workspace_bytes):
//   status  int32[64]                     latched device error, as in LookupDev
//   len     int32[max_slots]              tokens held
//   firm    int32[max_slots]              rows from the first on that no append writes: those there when a grow
//                                         last failed, and those of pages that a fork shared
//   refs    int32[num_pages]              slots that hold the page
//   bits    u32[ceil(num_pages / 128) * 4] bit p % 32 of word p / 32: page p is free
//   table   int32[max_slots][max_pages]   pages held, -1 past the last
//   req     int2[max_slots]               a call's plan per batch position
//   list    int32[3][num_pages]           a call's page lists
struct CacheDev {
    int32_t* status;
    int32_t* len;
    int32_t* firm;
    int32_t* refs;
    uint32_t* bits;
    int32_t* table;
    int2* req;
    int32_t* list;
    int32_t max_slots, max_pages, num_pages;
    int32_t shift;  // log2(page_tokens)

    __host__ __device__ int32_t page_tokens() const { return 1 << shift; }
    __host__ __device__ int32_t pages(int64_t n) const { return (int32_t)((n + page_tokens() - 1) >> shift); }
    // Pages that a slot of n tokens holds, never past its table row.
    __host__ __device__ int32_t held(int32_t n) const
    {
        const int32_t p = pages(n);
        return p < max_pages ? p : max_pages;
    }
    __host__ __device__ int32_t words() const { return (num_pages + 127) / 128 * 4; }
};

inline int dtype_bytes(int32_t dtype)
{
    return dtype == CLK_DTYPE_F32 ? 4 : dtype == CLK_DTYPE_BF16 || dtype == CLK_DTYPE_F16 ? 2 : 0;
}

// CLK_OK for a pool whose fields are usable.
inline int check_pool(const clk_pool* p)
{
    if (p == nullptr || p->d_base == nullptr) return CLK_EINVAL;
    const int es = dtype_bytes(p->dtype);
    if (es == 0 || !aligned(p->d_base, (size_t)es)) return CLK_EINVAL;
    if (p->planes < 2 || p->planes % 2 != 0 || p->planes > 65534 || p->heads < 1 || p->heads > 65535 || p->dim < 1 ||
        p->dim > 256)
        return CLK_EINVAL;
    if (p->plane_stride < 0 || p->page_stride < 0 || p->head_stride < 0 || p->tok_stride < 0) return CLK_EINVAL;
    return CLK_OK;
}

}  // namespace clk

struct clk_cache {
    clk::CacheDev dev;
    void* ws;
    size_t bytes;
};

namespace clk {

inline int check_cache_batch(const clk_cache* h, int32_t B)
{
    if (h == nullptr || h->ws == nullptr) return CLK_ESTATE;
    if (B < 0 || B > h->dev.max_slots) return CLK_EINVAL;
    return CLK_OK;
}

}  // namespace clk
