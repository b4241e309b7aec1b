// Trees of drafted tokens: ancestor masks and greedy verification.  One CTA
// of 64 threads per request, thread n for node n; a tree is a few hundred
// bytes, so both are bound by the latency of one launch and of one dependent
// load (the target's answer at the parent): 3 to 4 us each, for 1 request
// and for 64.
#include <cuda_runtime.h>
#include <stdint.h>

#include "clk.h"
#include "clk_device.cuh"
#include "clk_host.h"

namespace clk {
namespace {

constexpr int kNodes = CLK_TREE_MAX;

// The parent of node n, or -1 where it has none (node 0, a bad parent, past the tree).
__device__ __forceinline__ int tree_parent(const int32_t* parent, int64_t at, int n, int nodes)
{
    if (n <= 0 || n >= nodes) return -1;
    const int32_t p = parent[at];
    return p >= 0 && p < n ? p : -1;
}

__global__ void __launch_bounds__(kNodes) k_tree_masks(int32_t N, const int32_t* parent, const int32_t* nodes,
                                                       int64_t* mask)
{
    chained();
    __shared__ int up[kNodes];
    const int b = blockIdx.x, n = threadIdx.x;
    const int count = nodes[b] >= 0 && nodes[b] <= N ? nodes[b] : 0;
    const int64_t at = (int64_t)b * N + n;
    up[n] = tree_parent(parent, at, n, count);
    __syncthreads();
    if (n >= N) return;
    unsigned long long m = 0;
    if (n < count)
        for (int a = n; a >= 0; a = up[a]) m |= 1ull << a;
    mask[at] = (int64_t)m;
}

__global__ void __launch_bounds__(kNodes) k_tree_accept(int32_t N, const int32_t* tok, const int32_t* parent,
                                                        const int32_t* nodes, const int32_t* argmax, int32_t* accept,
                                                        int32_t* path, int32_t* emitted, int32_t* out_tok)
{
    chained();
    __shared__ int up[kNodes], text[kNodes];
    __shared__ bool fits[kNodes];
    __shared__ unsigned hits[2];
    const int b = blockIdx.x, n = threadIdx.x;
    const int count = nodes[b] >= 0 && nodes[b] <= N ? nodes[b] : 0;
    const int64_t at = (int64_t)b * N + n;
    const int p = tree_parent(parent, at, n, count);
    const int t = n < count ? tok[at] : CLK_SENT;
    up[n] = p;
    text[n] = t;
    bool fit = n == 0 ? count > 0 : p >= 0 && t >= 0 && t == argmax[(int64_t)b * N + p];
    __syncthreads();
    // of siblings with the same token the lowest counts
    if (fit && n > 0)
        for (int m = 1; m < n; ++m)
            if (up[m] == p && text[m] == t) fit = false;
    fits[n] = fit;
    __syncthreads();
    bool hit = fit;
    for (int a = up[n]; hit && a >= 0; a = up[a]) hit = fits[a];
    const unsigned here = __ballot_sync(0xffffffffu, hit);
    if ((n & 31) == 0) hits[n >> 5] = here;
    __syncthreads();
    const int taken = __popc(hits[0]) + __popc(hits[1]);
    if (hit) {
        const int rank = __popc(here & ((1u << (n & 31)) - 1u)) + (n >= 32 ? __popc(hits[0]) : 0);
        path[(int64_t)b * N + rank] = n;
        out_tok[(int64_t)b * N + rank] = argmax[at];
    }
    if (n >= taken && n < N) {
        path[at] = -1;
        out_tok[at] = CLK_SENT;
    }
    if (n == 0) {
        accept[b] = taken > 0 ? taken - 1 : 0;
        emitted[b] = taken;
    }
}

int check_tree(int32_t B, int32_t N)
{
    return B < 0 || B > CLK_MAX_BATCH || N < 1 || N > CLK_TREE_MAX ? CLK_EINVAL : CLK_OK;
}

}  // namespace
}  // namespace clk

using namespace clk;

extern "C" int clk_tree_masks(int32_t B, int32_t N, const int32_t* d_parent, const int32_t* d_nodes, int64_t* d_mask,
                              clk_stream_t s)
{
    const int rc = check_tree(B, N);
    if (rc != CLK_OK || B == 0) return rc;
    if (!ok_i32(d_parent) || !ok_i32(d_nodes) || d_mask == nullptr || !aligned(d_mask, 8)) return CLK_EINVAL;
    return launch_chained(k_tree_masks, (unsigned)B, kNodes, (cudaStream_t)s, N, d_parent, d_nodes, d_mask);
}

extern "C" int clk_tree_accept(int32_t B, int32_t N, const int32_t* d_tok, const int32_t* d_parent,
                               const int32_t* d_nodes, const int32_t* d_argmax, int32_t* d_accept, int32_t* d_path,
                               int32_t* d_emitted, int32_t* d_out_tok, clk_stream_t s)
{
    const int rc = check_tree(B, N);
    if (rc != CLK_OK || B == 0) return rc;
    if (!ok_i32(d_tok) || !ok_i32(d_parent) || !ok_i32(d_nodes) || !ok_i32(d_argmax) || !ok_i32(d_accept) ||
        !ok_i32(d_path) || !ok_i32(d_emitted) || !ok_i32(d_out_tok))
        return CLK_EINVAL;
    return launch_chained(k_tree_accept, (unsigned)B, kNodes, (cudaStream_t)s, N, d_tok, d_parent, d_nodes, d_argmax, d_accept,
                          d_path, d_emitted, d_out_tok);
}
