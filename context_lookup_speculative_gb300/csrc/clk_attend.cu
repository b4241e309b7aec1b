// Attention of new tokens over a paged cache: the general kernel, for every
// type, head count and stride, and the entry points.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "clk.h"
#include "clk_attend.h"
#include "clk_cache.h"
#include "clk_host.h"

namespace clk {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxDim = 256;

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half(x); }
template <>
__device__ __forceinline__ float from_f(float x) { return x; }

// One CTA per query row and head: 128 keys at a time, a thread scores one key
// and then accumulates one or two elements of the output over the keys, with
// the running maximum and sum of the softmax.  A key that is not visible is
// not read.  It re-reads K and V for every row, so it is bound by the L2 and
// the loads' latency; the tensor-core path takes the shapes it can.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_attend_rows(Attend A)
{
    __shared__ float sq[kMaxDim], sp[kThreads], red[kThreads / 32];
    const int tid = threadIdx.x, h = blockIdx.y, kh = h / A.group;
    int b, t;
    int64_t row;
    if (A.off != nullptr) {
        row = blockIdx.x;
        // the last request that starts at or before this row
        int lo = 0, hi = A.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (A.off[mid] <= row)
                lo = mid;
            else
                hi = mid - 1;
        }
        b = lo;
        t = 0;
    } else {
        b = blockIdx.x / A.N;
        t = blockIdx.x - b * A.N;
        row = blockIdx.x;
    }
    const bool first = h == 0 && tid == 0 && (A.off != nullptr || t == 0);
    const Request R = attend_request(A, b, first);
    if (A.off != nullptr) {
        if (row < R.base || row - R.base >= R.rows) return;
        t = (int)(row - R.base);
    }
    T* const out = static_cast<T*>(A.out) + (row * A.q_heads + h) * A.dim;
    if (t >= R.rows) {  // past the tree
        for (int d = tid; d < A.dim; d += kThreads) out[d] = from_f<T>(0.0f);
        return;
    }
    const int64_t q0 = A.off != nullptr ? row * A.q_row : b * A.q_req + t * A.q_row;
    const int64_t k0 = (A.off != nullptr ? R.base * A.k_row : b * A.k_req) + kh * A.k_head;
    const int64_t v0 = (A.off != nullptr ? R.base * A.v_row : b * A.v_req) + kh * A.v_head;
    const unsigned long long near = A.off != nullptr ? 0 : (unsigned long long)A.mask[row];
    for (int d = tid; d < A.dim; d += kThreads) sq[d] = to_f(static_cast<const T*>(A.q)[q0 + h * A.q_head + d]);
    float m = -INFINITY, l = 0.0f, acc[2] = {0.0f, 0.0f};
    const int32_t fresh = A.off != nullptr ? t + 1 : R.rows;
    const int64_t keys = (int64_t)R.ctx + fresh;
    for (int64_t j0 = 0; j0 < keys; j0 += kThreads) {
        __syncthreads();
        const int64_t j = j0 + tid;
        float s = -INFINITY;
        bool seen = j < keys;
        if (seen && j >= R.ctx && A.off == nullptr) seen = (near >> (j - R.ctx)) & 1;
        if (seen) {
            const T* key = nullptr;
            if (j < R.ctx) {
                const int32_t page = A.C.table[(int64_t)R.slot * A.C.max_pages + (j >> A.C.shift)];
                if (page >= 0 && page < A.C.num_pages)
                    key = static_cast<const T*>(A.kc) + page * A.page_stride + kh * A.head_stride +
                          (j & (A.C.page_tokens() - 1)) * A.tok_stride;
                else
                    latch(A.C.status, CLK_EINVAL, R.slot);
            } else {
                key = static_cast<const T*>(A.k) + k0 + (j - R.ctx) * A.k_row;
            }
            seen = key != nullptr;
            if (seen) {
                float x = 0.0f;
                for (int d = 0; d < A.dim; ++d) x = fmaf(sq[d], to_f(key[d]), x);
                s = x * A.scale;
            }
        }
        float top = s;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        if ((tid & 31) == 0) red[tid >> 5] = top;
        __syncthreads();
        const float mt = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        const float ref = mt == -INFINITY ? 0.0f : mt;
        const float p = seen ? expf(s - ref) : 0.0f;
        sp[tid] = seen ? p : -1.0f;  // -1: not visible, its value is not read
        const float fix = expf(m - ref);
        float sum = p;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        __syncthreads();
        if ((tid & 31) == 0) red[tid >> 5] = sum;
        __syncthreads();
        l = l * fix + (red[0] + red[1] + red[2] + red[3]);
        m = mt;
        acc[0] *= fix;
        acc[1] *= fix;
        const int n = keys - j0 < kThreads ? (int)(keys - j0) : kThreads;
        for (int i = 0; i < n; ++i) {
            const float w = sp[i];
            if (w < 0.0f) continue;
            const int64_t g = j0 + i;
            const T* val;
            if (g < R.ctx) {
                const int32_t page = A.C.table[(int64_t)R.slot * A.C.max_pages + (g >> A.C.shift)];
                val = static_cast<const T*>(A.vc) + page * A.page_stride + kh * A.head_stride +
                      (g & (A.C.page_tokens() - 1)) * A.tok_stride;
            } else {
                val = static_cast<const T*>(A.v) + v0 + (g - R.ctx) * A.v_row;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = tid + e * kThreads;
                if (d < A.dim) acc[e] = fmaf(w, to_f(val[d]), acc[e]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int d = tid + e * kThreads;
        if (d < A.dim) out[d] = from_f<T>(l == 0.0f ? 0.0f : acc[e] / l);
    }
}

template <typename T>
int launch_rows(const Attend& A, cudaStream_t s)
{
    const int64_t rows = A.off != nullptr ? A.T : (int64_t)A.B * A.N;
    k_attend_rows<T><<<dim3((unsigned)rows, (unsigned)A.q_heads), kThreads, 0, s>>>(A);
    return launch_status();
}

int launch_attend(const Attend& A, void* scratch, size_t bytes, cudaStream_t s)
{
    if (attend_mma_takes(A)) {
        if (scratch == nullptr || !aligned(scratch, 16) || bytes < attend_mma_scratch(A.q_heads, A.kv_heads, A.dim))
            return CLK_EINVAL;
        return attend_mma_launch(A, scratch, s);
    }
    switch (A.dtype) {
    case CLK_DTYPE_BF16: return launch_rows<__nv_bfloat16>(A, s);
    case CLK_DTYPE_F16: return launch_rows<__half>(A, s);
    default: return launch_rows<float>(A, s);
    }
}

// Checks what both calls share and fills the common fields.
int fill_attend(Attend& A, const clk_attn* a, clk_cache* h, const int32_t* d_slots, const clk_pool* pool, int32_t layer,
                const int32_t* d_ctx, int32_t B)
{
    if (a == nullptr || B < 0 || B > CLK_MAX_BATCH) return CLK_EINVAL;
    const int es = dtype_bytes(a->dtype);
    if (es == 0 || a->dim < 1 || a->dim > kMaxDim || a->kv_heads < 1 || a->q_heads < a->kv_heads || a->q_heads > 65535 ||
        a->q_heads % a->kv_heads != 0 || !isfinite(a->scale))
        return CLK_EINVAL;
    for (int64_t st : {a->q_req, a->q_row, a->q_head, a->k_req, a->k_row, a->k_head, a->v_req, a->v_row, a->v_head})
        if (st < 0) return CLK_EINVAL;
    for (const void* p : {a->d_q, a->d_k, a->d_v, (const void*)a->d_out})
        if (!aligned(p, (size_t)es)) return CLK_EINVAL;
    A = Attend{};
    if (h != nullptr) {
        int rc = check_cache_batch(h, B);
        if (rc != CLK_OK) return rc;
        if (check_pool(pool) != CLK_OK || pool->dtype != a->dtype || pool->heads != a->kv_heads || pool->dim != a->dim ||
            layer < 0 || layer >= pool->planes / 2)
            return CLK_EINVAL;
        if (B > 0 && !ok_i32(d_slots)) return CLK_EINVAL;
        A.C = h->dev;
        A.slots = d_slots;
        A.ctx = d_ctx;
        const char* base = static_cast<const char*>(pool->d_base);
        A.kc = base + 2 * (int64_t)layer * pool->plane_stride * es;
        A.vc = base + (2 * (int64_t)layer + 1) * pool->plane_stride * es;
        A.page_stride = pool->page_stride;
        A.head_stride = pool->head_stride;
        A.tok_stride = pool->tok_stride;
    }
    if (!aligned(d_ctx, 4)) return CLK_EINVAL;
    A.q = a->d_q;
    A.k = a->d_k;
    A.v = a->d_v;
    A.out = a->d_out;
    A.q_req = a->q_req;
    A.q_row = a->q_row;
    A.q_head = a->q_head;
    A.k_req = a->k_req;
    A.k_row = a->k_row;
    A.k_head = a->k_head;
    A.v_req = a->v_req;
    A.v_row = a->v_row;
    A.v_head = a->v_head;
    A.B = B;
    A.q_heads = a->q_heads;
    A.kv_heads = a->kv_heads;
    A.group = a->q_heads / a->kv_heads;
    A.dim = a->dim;
    A.dtype = a->dtype;
    A.scale = a->scale;
    return CLK_OK;
}

bool attn_pointers(const clk_attn* a) { return a->d_q != nullptr && a->d_k != nullptr && a->d_v != nullptr && a->d_out != nullptr; }

}  // namespace
}  // namespace clk

using namespace clk;

extern "C" int clk_attend_scratch_bytes(int32_t q_heads, int32_t kv_heads, int32_t dim, size_t* bytes)
{
    if (bytes == nullptr || kv_heads < 1 || q_heads < kv_heads || q_heads % kv_heads != 0 || dim < 1 || dim > kMaxDim)
        return CLK_EINVAL;
    const size_t n = attend_mma_scratch(q_heads, kv_heads, dim);
    *bytes = n > 0 ? n : 16;
    return CLK_OK;
}

extern "C" int clk_tree_attend(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool, int32_t layer,
                               const clk_attn* a, int32_t N, const int32_t* d_nodes, const int64_t* d_mask,
                               const int32_t* d_ctx, void* d_scratch, size_t scratch_bytes, clk_stream_t s)
{
    if (h == nullptr) return CLK_ESTATE;
    Attend A;
    const int rc = fill_attend(A, a, h, d_slots, pool, layer, d_ctx, B);
    if (rc != CLK_OK) return rc;
    if (N < 1 || N > CLK_TREE_MAX) return CLK_EINVAL;
    if (B == 0) return CLK_OK;
    if (!attn_pointers(a) || !ok_i32(d_nodes) || d_mask == nullptr || !aligned(d_mask, 8)) return CLK_EINVAL;
    A.nodes = d_nodes;
    A.mask = d_mask;
    A.N = N;
    return launch_attend(A, d_scratch, scratch_bytes, (cudaStream_t)s);
}

extern "C" int clk_prompt_attend(const clk_attn* a, const int64_t* d_off, int32_t B, int64_t T, clk_cache* h,
                                 const int32_t* d_slots, const clk_pool* pool, int32_t layer, const int32_t* d_ctx,
                                 void* d_scratch, size_t scratch_bytes, clk_stream_t s)
{
    Attend A;
    if (h == nullptr && d_ctx != nullptr) return CLK_EINVAL;
    const int rc = fill_attend(A, a, h, d_slots, pool, layer, d_ctx, B);
    if (rc != CLK_OK) return rc;
    if (T < 0 || T > ((int64_t)1 << 30)) return CLK_EINVAL;
    if (B == 0 || T == 0) return CLK_OK;
    if (!attn_pointers(a) || d_off == nullptr || !aligned(d_off, 8)) return CLK_EINVAL;
    A.off = d_off;
    A.T = T;
    return launch_attend(A, d_scratch, scratch_bytes, (cudaStream_t)s);
}
