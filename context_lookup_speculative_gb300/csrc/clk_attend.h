// Arguments of the attention kernels, shared by clk_attend.cu (the general
// kernel and the entry points) and clk_attend_mma.cu (tensor cores).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "clk.h"
#include "clk_cache.h"
#include "clk_device.cuh"

namespace clk {

struct Attend {
    CacheDev C;            // C.status is null without a cache
    const int32_t* slots;  // null without a cache
    const int32_t* ctx;    // null: the slot's length (tree), 0 (prompt)
    const void *kc, *vc;   // the layer's two planes; null without a cache
    int64_t page_stride, head_stride, tok_stride;
    // a pool in 8 bits: its scales in the two planes (null for one of q's type), a block's rows as a power of two
    const float *ks, *vs;
    int64_t scale_page, scale_head, scale_block;
    int32_t scale_shift;
    const void *q, *k, *v;
    void* out;
    int64_t q_req, q_row, q_head, k_req, k_row, k_head, v_req, v_row, v_head;
    const int32_t* nodes;  // tree: nodes per request
    const int64_t* mask;   // tree: masks [B, N]
    const int64_t* off;    // prompt: row offsets [B + 1]; null for a tree
    int64_t T;             // prompt: rows in all
    int32_t B, N;          // N: tree rows per request
    int32_t q_heads, kv_heads, group, dim, dtype;
    float scale;
};

// One request's share of a call.
struct Request {
    int32_t slot;  // -1 without a cache
    int32_t ctx;   // cached rows
    int32_t rows;  // new rows
    int64_t base;  // prompt: its first row
    bool ok;
};

// Reads and checks request b; a request that is not ok has no rows.
__device__ __forceinline__ Request attend_request(const Attend& A, int b, bool report)
{
    Request r{-1, 0, 0, 0, true};
    int32_t who = b;
    if (A.off != nullptr) {
        const int64_t lo = A.off[b], hi = A.off[b + 1];
        r.ok = lo >= 0 && hi >= lo && hi <= A.T && hi - lo < ((int64_t)1 << 30);
        r.base = lo;
        r.rows = r.ok ? (int32_t)(hi - lo) : 0;
    } else {
        r.rows = A.nodes[b];
        r.ok = r.rows >= 0 && r.rows <= A.N;
    }
    if (A.slots != nullptr) {
        r.slot = A.slots[b];
        const bool fine = r.slot >= 0 && r.slot < A.C.max_slots;
        if (fine) {
            who = r.slot;
            const int32_t len = A.C.len[r.slot];
            r.ctx = A.ctx != nullptr ? A.ctx[b] : A.off != nullptr ? 0 : len;
            r.ok = r.ok && r.ctx >= 0 && r.ctx <= len && A.C.pages(r.ctx) <= A.C.max_pages;
        } else {
            r.ok = false;
        }
    }
    if (!r.ok) {
        r.rows = r.ctx = 0;
        if (report && A.C.status != nullptr) latch(A.C.status, CLK_EINVAL, who);
    }
    return r;
}

// Tensor-core path (clk_attend_mma.cu): whether it takes these shapes, and the launch.
bool attend_mma_takes(const Attend& A);
int attend_mma_launch(const Attend& A, void* scratch, cudaStream_t s);
size_t attend_mma_scratch(int32_t q_heads, int32_t kv_heads, int32_t dim);

}  // namespace clk
