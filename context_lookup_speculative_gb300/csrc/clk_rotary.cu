// Position rotation: queries and keys of drafted trees, and keys on their way
// into the pages of a cache, of the rows' type or in 8 bits.
//
// Work is counted in blocks: rows of one request that lie in one aligned
// block of `tokens` positions of its slot (16 where the pool has no scales),
// or 16 nodes of a tree; and in pieces, the heads of a block.  Every CTA counts
// the requests' blocks (a prefix sum over the batch, so offsets may fall and
// requests may be left out) and takes an equal run of all pieces.  What a
// block's rows are and where they go is found once, by a thread per row, and
// lies in shared memory.
//
// Fast rows (16 bits, dim a multiple of 16 up to 128, whole aligned vectors): a
// lane holds two vectors of 8 elements that turn together (j and j + pairs / 8,
// or neighbours), so that no value crosses lanes.  Without scales (k_turn_rows)
// a warp has the same rows of every head and keeps their part of the table in
// registers, four heads' loads in flight.  (With all 16 rows of a head to a warp
// every head read the table again, and blocks went to CTAs whole: 256 trees of
// 32 nodes, 48/8 heads of 128, 53.5 us, now 35.7; 16 prompts of 100 to 2,000
// tokens, 32/8 heads of 128, 92 and 75.)  With scales (k_turn_rows8) a team of
// warps takes a block and head: the rows stay in registers between the search
// for their largest magnitude and their rounding, so every row is read once.
// Where a warp holds half as many rows 24 warps fit an SM instead of 16 (64
// prompts of 100 to 2,000 tokens, 24/4 heads of 64: 132 us, then 125, and 117
// with one multiplication an element where the scale is a power of two).
// Other rows go element by element (k_turn_any), read twice where there are
// scales.
//
// All of it would be bound by memory: rows in, rows out, and 8 bytes a pair and
// position of the table, which the heads of a position share.  Trees reach 5.0,
// prompts 5.7 TB/s (73 and 84% of a copy), into 8 bits 4.8 (71%): there 62
// million warp instructions take half of the issue slots, and chains of loads,
// a barrier of the team and stores the rest.  Slower: the next piece's rows on
// their way to shared memory (136 us against 132), the next block's rows looked
// up meanwhile (145 against 135), q's heads in a launch of their own (128
// against 117).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "clk.h"
#include "clk_cache.h"
#include "clk_device.cuh"
#include "clk_eight.cuh"
#include "clk_host.h"

namespace clk {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostRows = 128;  // of a block

struct Turn {
    CacheDev C;
    const int32_t* slots;
    int32_t B;
    // appended rows
    int64_t N;
    const int64_t* off;
    const int32_t *path, *count;
    // trees (nodes is null for appended rows)
    const int32_t *nodes, *ctx;
    const int64_t* mask;
    // rotation (pairs 0: none)
    const float* table;
    int64_t positions;
    int32_t pairs;
    // sources and results beside the pages; with appended rows *_req are not used
    const void *k, *v, *q;
    void *q_out, *k_out;
    int64_t layer, k_req, k_row, k_head, q_req, q_row, q_head, qo_req, qo_row, qo_head, ko_req, ko_row, ko_head;
    int32_t layers, q_heads, kv_heads, dim;
    // pool (null with trees) and scales
    void* pool;
    int64_t plane, page, head, tok;
    float* scale;
    int64_t s_plane, s_page, s_head, s_block;
    int32_t layer0, shift;  // log2(rows of a block)
};

// What a CTA knows of its block's rows (in shared memory).
struct Rows {
    int64_t k[kMostRows], q[kMostRows];    // source rows, -1 for a row that is not written
    int64_t ko[kMostRows], qo[kMostRows];  // results beside the pages
    int64_t to[kMostRows];                 // in a plane of the pool
    int64_t pos[kMostRows];
    int64_t scale;  // of the block, in a plane of the scales
    int64_t start;  // the block's first row in a plane of the pool
    int32_t first;  // rows of the block before the first written one
};

// Request b's rows: positions p0 .. p0 + n - 1 (append), or its nodes.
struct Span {
    int64_t p0, base, rows;
    int32_t n, slot;
    int err, who;  // why it is left out
};

__device__ __forceinline__ Span span_of(const Turn& A, int b)
{
    Span x{0, 0, 0, 0, -1, CLK_EINVAL, b};
    const int32_t s = A.slots[b];
    if (s < 0 || s >= A.C.max_slots) return x;
    x.slot = x.who = s;
    const int32_t len = A.C.len[s];
    if (A.nodes != nullptr) {
        const int32_t n = A.nodes[b], ctx = A.ctx != nullptr ? A.ctx[b] : len;
        if (n < 0 || n > A.N || ctx < 0 || ctx > len) return x;
        x.p0 = ctx;
        x.n = n;
    } else {
        const int64_t total = A.off != nullptr ? A.N : (int64_t)A.B * A.N;
        const int32_t n = A.count[b];
        x.base = A.off != nullptr ? A.off[b] : b * A.N;
        x.rows = A.off != nullptr ? A.off[b + 1] - x.base : A.N;
        if (n < 0 || n > len - A.C.firm[s] || n > x.rows || x.base < 0 || x.base > total - x.rows) return x;
        if (A.pairs > 0 && n > 0 && len > A.positions) return x;
        x.p0 = len - n;
        x.n = n;
    }
    x.err = CLK_OK;
    return x;
}

__device__ __forceinline__ int32_t blocks_of(const Turn& A, const Span& x)
{
    if (x.err != CLK_OK || x.n == 0) return 0;
    if (A.nodes != nullptr) return (x.n - 1 >> A.shift) + 1;
    return (int32_t)((x.p0 + x.n - 1 >> A.shift) - (x.p0 >> A.shift)) + 1;
}

// before[b]: blocks of the requests before b; before[B]: of all.
__device__ void count_blocks(const Turn& A, int64_t* before)
{
    __shared__ int64_t sums[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool report = blockIdx.x == 0 && blockIdx.y == 0;
    int64_t all = 0;
    for (int at = 0; at < A.B; at += kThreads) {
        const int b = at + tid;
        int64_t n = 0;
        if (b < A.B) {
            const Span x = span_of(A, b);
            if (report && x.err != CLK_OK) latch(A.C.status, x.err, x.who);
            n = blocks_of(A, x);
        }
        int64_t y = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        if (lane == 31) sums[warp] = y;
        __syncthreads();
        int64_t mine = all + y - n;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) mine += sums[w];
            all += sums[w];
        }
        if (b < A.B) before[b] = mine;
        __syncthreads();
    }
    if (tid == 0) before[A.B] = all;
    __syncthreads();
}

// The rows of block `unit`; threads below the block's rows take one each.
__device__ __forceinline__ void find_rows(const Turn& A, const int64_t* before, int64_t unit, Rows& R, bool report)
{
    const int tid = threadIdx.x, T = 1 << A.shift;
    if (tid >= T) return;
    // the last request whose blocks start at or before this one
    int lo = 0, hi = A.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= unit)
            lo = mid;
        else
            hi = mid - 1;
    }
    const Span x = span_of(A, lo);
    const int64_t nth = unit - before[lo];
    int64_t k = -1, q = -1, ko = 0, qo = 0, to = 0, pos = 0;
    if (A.nodes != nullptr) {
        const int64_t n = nth * T + tid;
        if (n < x.n) {
            uint64_t seen = (uint64_t)A.mask[lo * A.N + n];
            if (x.n < 64) seen &= (1ull << x.n) - 1;
            const int deep = __popcll(seen);
            pos = x.p0 + (deep > 0 ? deep - 1 : 0);
            if (pos < A.positions) {
                k = lo * A.k_req + n * A.k_row;
                q = lo * A.q_req + n * A.q_row;
                ko = lo * A.ko_req + n * A.ko_row;
                qo = lo * A.qo_req + n * A.qo_row;
            } else if (report) {
                latch(A.C.status, CLK_EINVAL, x.slot);
            }
        }
    } else {
        const int64_t start = (x.p0 & ~(int64_t)(T - 1)) + nth * T;  // the block's first position
        pos = start + tid;
        const int32_t slot_page = (int32_t)(start >> A.C.shift);
        const int32_t page = slot_page < A.C.max_pages ? A.C.table[(int64_t)x.slot * A.C.max_pages + slot_page] : -1;
        const bool held = page >= 0 && page < A.C.num_pages;
        const int64_t line = start & (A.C.page_tokens() - 1);
        if (pos >= x.p0 && pos < x.p0 + x.n) {
            const int64_t i = pos - x.p0, r = A.path != nullptr ? A.path[x.base + i] : i;
            if (held && r >= 0 && r < x.rows) {
                k = (x.base + r) * A.k_row;
                q = (x.base + r) * A.q_row;
                ko = (x.base + r) * A.ko_row;
                qo = (x.base + r) * A.qo_row;
                to = page * A.page + (line + tid) * A.tok;
            } else if (report) {
                latch(A.C.status, CLK_EINVAL, x.slot);
            }
        }
        if (tid == 0) {
            R.first = x.p0 > start ? (int32_t)(x.p0 - start) : 0;
            R.start = held ? page * A.page + line * A.tok : -1;
            R.scale = held && A.scale != nullptr ? page * A.s_page + (line >> A.shift) * A.s_block : -1;
        }
    }
    R.k[tid] = k;
    R.q[tid] = q;
    R.ko[tid] = ko;
    R.qo[tid] = qo;
    R.to[tid] = to;
    R.pos[tid] = pos;
}

// What a block's warps go through: the layers' K heads, their V heads, the q heads.
struct Piece {
    int kind;  // 0 K, 1 V, 2 q
    int layer, head;
};

__device__ __forceinline__ Piece piece_of(const Turn& A, int e)
{
    const int kv = A.layers * A.kv_heads;
    const int kind = e < kv ? 0 : A.v != nullptr && e < 2 * kv ? 1 : 2;
    if (kind == 2) return Piece{2, 0, e - (A.v != nullptr ? 2 * kv : kv)};
    const int i = kind == 0 ? e : e - kv;
    return Piece{kind, i / A.kv_heads, i % A.kv_heads};
}

__host__ __device__ inline int pieces(const Turn& A)
{
    return A.layers * A.kv_heads * (A.v != nullptr ? 2 : 1) + (A.q != nullptr ? A.q_heads : 0);
}

// The block's scale from its rows' largest finite magnitude, and what its earlier rows had (0: they need no change).
__device__ __forceinline__ float settle(float top, float had, bool before, float* old)
{
    float s = scale_for(top);
    *old = 0.0f;
    if (before && had > 0.0f && had <= FLT_MAX) {
        if (had >= s)
            s = had;
        else
            *old = had;
    }
    return s;
}

// x / s: by the reciprocal where that is exact.
struct Divide {
    float s, inv;
    bool whole;
    __device__ explicit Divide(float scale)
    {
        s = scale;
        inv = 1.0f / scale;
        whole = (__float_as_uint(scale) & 0x7fffffu) == 0;
    }
    __device__ float operator()(float x) const { return whole ? x * inv : __fdiv_rn(x, s); }
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half(x); }
template <>
__device__ __forceinline__ float from_f(float x) { return x; }

// (x, y) turned; the products are rounded before the sums.
__device__ __forceinline__ void turn(float& x, float& y, float c, float s)
{
    const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)), v = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = u;
    y = v;
}

// ---------------------------------------------------------------------------
// Any rows: a warp per block and head, an element pair per lane
// ---------------------------------------------------------------------------
template <typename T, bool NEIGHBOURS, bool EIGHT>
__global__ void __launch_bounds__(kThreads) k_turn_any(const __grid_constant__ Turn A)
{
    chained();
    extern __shared__ int64_t before[];
    __shared__ Rows R;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T_rows = 1 << A.shift;
    count_blocks(A, before);
    const int64_t units = before[A.B];
    const int all = pieces(A);
    const int e0 = (int)((int64_t)all * blockIdx.y / gridDim.y), e1 = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y);
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        __syncthreads();  // the last block's rows are done with
        find_rows(A, before, u, R, blockIdx.y == 0);
        __syncthreads();
        for (int e = e0 + warp; e < e1; e += kWarps) {
            const Piece P = piece_of(A, e);
            const bool turned = P.kind != 1 && A.pairs > 0, paged = A.pool != nullptr && P.kind != 2;
            const T* const src = P.kind == 2 ? static_cast<const T*>(A.q) + P.head * A.q_head
                                             : static_cast<const T*>(P.kind == 1 ? A.v : A.k) + P.layer * A.layer + P.head * A.k_head;
            T* const out = P.kind == 2 ? static_cast<T*>(A.q_out) + P.head * A.qo_head
                           : P.kind == 0 && A.k_out != nullptr ? static_cast<T*>(A.k_out) + P.head * A.ko_head : nullptr;
            const int64_t plane = 2 * ((int64_t)A.layer0 + P.layer) + P.kind;
            const int n = turned ? A.pairs : 0;
            // f(row, element, value) for all elements of the block's rows, an element and its partner at once
            auto each = [&](auto f) {
                for (int r = 0; r < T_rows; ++r) {
                    const int64_t from = P.kind == 2 ? R.q[r] : R.k[r];
                    if (from < 0) continue;
                    const float* const cs = A.table + R.pos[r] * 2 * A.pairs;
                    for (int i = lane; i < n; i += 32) {
                        const int a = NEIGHBOURS ? 2 * i : i, b = NEIGHBOURS ? 2 * i + 1 : i + n;
                        float x = to_f(src[from + a]), y = to_f(src[from + b]);
                        turn(x, y, cs[i], cs[n + i]);
                        f(r, a, x);
                        f(r, b, y);
                    }
                    for (int d = 2 * n + lane; d < A.dim; d += 32) f(r, d, to_f(src[from + d]));
                }
            };
            if (EIGHT && paged) {
                uint8_t* const pool = static_cast<uint8_t*>(A.pool) + plane * A.plane + P.head * A.head;
                float* const scale = R.scale < 0 ? nullptr : A.scale + plane * A.s_plane + P.head * A.s_head + R.scale;
                float top = 0.0f;
                each([&](int, int, float x) { top = fmaxf(top, fabsf(x) <= FLT_MAX ? fabsf(x) : 0.0f); });
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                if (scale == nullptr) continue;
                float old;
                const float s = settle(top, *scale, R.first > 0, &old);
                __syncwarp();
                if (lane == 0) *scale = s;
                const Divide by(s);
                if (old != 0.0f)
                    for (int r = 0; r < R.first; ++r)
                        for (int d = lane; d < A.dim; d += 32) {
                            uint8_t* const p = pool + R.start + r * A.tok + d;
                            *p = (uint8_t)to_e4m3(by(from_e4m3(*p) * old), 0.0f);
                        }
                each([&](int r, int d, float x) {
                    pool[R.to[r] + d] = (uint8_t)to_e4m3(by(x), 0.0f);
                    if (out != nullptr) out[R.ko[r] + d] = from_f<T>(x);
                });
            } else {
                T* const pool = paged ? static_cast<T*>(A.pool) + plane * A.plane + P.head * A.head : nullptr;
                each([&](int r, int d, float x) {
                    const T y = from_f<T>(x);
                    if (paged) pool[R.to[r] + d] = y;
                    if (out != nullptr) out[(P.kind == 2 ? R.qo[r] : R.ko[r]) + d] = y;
                });
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Fast rows
// ---------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ void unpack(uint4 x, float* f)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = y.x;
            f[2 * i + 1] = y.y;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 packed(const float* f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
        else
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint2 packed8(const float* f)
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = to_e4m3(f[4 * i], f[4 * i + 1]) | to_e4m3(f[4 * i + 2], f[4 * i + 3]) << 16;
    return make_uint2(w[0], w[1]);
}

constexpr int kSteps = 4;  // vectors of a row's two halves that a lane holds at a time

// Pieces of all blocks, one after the other; every CTA takes an equal run of them.
struct Share {
    int64_t at, end;
    int all, e0, e1;  // pieces of a block; those taken of this one
    __device__ Share(int64_t units, int pieces)
    {
        all = pieces;
        // (units < 2^40 and gridDim.x < 2^11)
        at = units * all * (int64_t)blockIdx.x / gridDim.x;
        end = units * all * ((int64_t)blockIdx.x + 1) / gridDim.x;
    }
    __device__ bool next(int64_t* unit)
    {
        if (at >= end) return false;
        *unit = at / all;
        e0 = (int)(at - *unit * all);
        e1 = end - at < all - e0 ? e0 + (int)(end - at) : all;
        at += e1 - e0;
        return true;
    }
};

// A warp has the same rows of a block's every head, so its lanes hold their part of the table for all of them.
template <bool BF16, bool NEIGHBOURS>
__global__ void __launch_bounds__(kThreads, 3) k_turn_rows(const __grid_constant__ Turn A)
{
    chained();
    extern __shared__ int64_t before[];
    __shared__ Rows R;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    count_blocks(A, before);
    const int wide = A.dim / 16, tall = 32 / wide, j = lane % wide, r0 = lane / wide;  // lanes of a row, rows of a warp
    const int turning = A.pairs / 8;
    const int steps = (16 + tall - 1) / tall, groups = kWarps / steps;  // warps of a head, heads at a time
    const int group = warp / steps, row = (warp - group * steps) * tall + r0;
    const bool mine = r0 < tall && row < 16 && group < groups;
    // vectors of 8 elements that this lane holds of a row
    const int va = !NEIGHBOURS && j < turning ? j : 2 * j, vb = !NEIGHBOURS && j < turning ? j + turning : 2 * j + 1;
    Share share(before[A.B], pieces(A));
    for (int64_t u; share.next(&u);) {
        __syncthreads();  // the last block's rows are done with
        find_rows(A, before, u, R, share.e0 == 0);
        __syncthreads();
        if (mine && R.k[row] >= 0) {
            float c[8], s[8];
            if (j < turning) {
                const float4* const cs = reinterpret_cast<const float4*>(A.table + R.pos[row] * 2 * A.pairs) + 2 * j;
                const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1), s0 = __ldg(cs + 2 * turning), s1 = __ldg(cs + 2 * turning + 1);
                c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w, c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
                s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w, s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
            }
            const int64_t k = R.k[row], q = R.q[row], ko = R.ko[row], qo = R.qo[row], to = R.to[row];
            for (int e = share.e0 + group; e < share.e1; e += kSteps * groups) {
                uint4 a[kSteps], b[kSteps];
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    if (e + i * groups >= share.e1) break;
                    const Piece P = piece_of(A, e + i * groups);
                    const uint16_t* const src = P.kind == 2 ? static_cast<const uint16_t*>(A.q) + P.head * A.q_head + q
                                                            : static_cast<const uint16_t*>(P.kind == 1 ? A.v : A.k) + P.layer * A.layer + P.head * A.k_head + k;
                    a[i] = __ldcs(reinterpret_cast<const uint4*>(src) + va);
                    b[i] = __ldcs(reinterpret_cast<const uint4*>(src) + vb);
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    if (e + i * groups >= share.e1) break;
                    const Piece P = piece_of(A, e + i * groups);
                    if (P.kind != 1 && j < turning) {
                        float x[8], y[8];
                        unpack<BF16>(a[i], x);
                        unpack<BF16>(b[i], y);
#pragma unroll
                        for (int p = 0; p < 8; ++p) {
                            if (NEIGHBOURS)
                                p < 4 ? turn(x[2 * p & 7], x[2 * p + 1 & 7], c[p], s[p]) : turn(y[2 * p & 7], y[2 * p + 1 & 7], c[p], s[p]);
                            else
                                turn(x[p], y[p], c[p], s[p]);
                        }
                        a[i] = packed<BF16>(x);
                        b[i] = packed<BF16>(y);
                    }
                    if (A.pool != nullptr && P.kind != 2) {
                        const int64_t plane = 2 * ((int64_t)A.layer0 + P.layer) + P.kind;
                        uint4* const out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(A.pool) + plane * A.plane + P.head * A.head + to);
                        out[va] = a[i];
                        out[vb] = b[i];
                    }
                    uint16_t* const out = P.kind == 2 ? static_cast<uint16_t*>(A.q_out) + P.head * A.qo_head + qo
                                          : P.kind == 0 && A.k_out != nullptr ? static_cast<uint16_t*>(A.k_out) + P.head * A.ko_head + ko : nullptr;
                    if (out != nullptr) {
                        reinterpret_cast<uint4*>(out)[va] = a[i];
                        reinterpret_cast<uint4*>(out)[vb] = b[i];
                    }
                }
            }
        }
    }
}

// log2(the rows of a block and head that a warp holds by `steps`)
__host__ __device__ constexpr int team_shift(int dim, int steps)
{
    int n = 0;
    while (2 << n <= steps * (32 / (dim / 16))) ++n;
    return n;
}

// Rows of 128 elements are the longest: with four steps a team's warps hold any block (with two, where the host says so).
static_assert(kWarps << team_shift(128, 4) >= kMostRows, "warps of a team");

// The same into 8 bits: a warp holds rows of a block and head, a team of at most kWarps warps them all.
template <bool BF16, bool NEIGHBOURS, int STEPS>
__global__ void __launch_bounds__(kThreads, STEPS == 2 ? 3 : 2) k_turn_rows8(const __grid_constant__ Turn A)
{
    chained();
    extern __shared__ int64_t before[];
    __shared__ Rows R;
    __shared__ float tops[2][kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    count_blocks(A, before);
    const int wide = A.dim / 16, tall = 32 / wide, j = lane % wide, r0 = lane / wide;  // lanes of a row, rows at a time
    const int turning = A.pairs / 8;
    const bool mine = r0 < tall;
    // vectors of 8 elements that this lane holds of a row
    const int va = !NEIGHBOURS && j < turning ? j : 2 * j, vb = !NEIGHBOURS && j < turning ? j + turning : 2 * j + 1;
    const int shift = min(team_shift(A.dim, STEPS), A.shift);  // log2(rows of a warp)
    const int rows = 1 << shift;
    const int per = 1 << (A.shift - shift);  // warps of a team, at most kWarps
    const int team = warp / per, part = warp - team * per, teams = kWarps / per;
    Share share(before[A.B], pieces(A));
    for (int64_t u; share.next(&u);) {
        __syncthreads();  // the last block's rows are done with
        find_rows(A, before, u, R, share.e0 == 0);
        __syncthreads();
        int flip = 0;
        for (int e = share.e0 + team; e < share.e1; e += teams, flip ^= 1) {
            const Piece P = piece_of(A, e);
            const bool turned = P.kind != 1 && j < turning, paged = A.pool != nullptr && P.kind != 2;
            const uint16_t* const src =
                P.kind == 2 ? static_cast<const uint16_t*>(A.q) + P.head * A.q_head
                            : static_cast<const uint16_t*>(P.kind == 1 ? A.v : A.k) + P.layer * A.layer + P.head * A.k_head;
            uint16_t* const out = P.kind == 2 ? static_cast<uint16_t*>(A.q_out) + P.head * A.qo_head
                                  : P.kind == 0 && A.k_out != nullptr ? static_cast<uint16_t*>(A.k_out) + P.head * A.ko_head : nullptr;
            const int64_t plane = 2 * ((int64_t)A.layer0 + P.layer) + P.kind;
            uint4 a[STEPS], b[STEPS];
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int r = rows * part + i * tall + r0;
                const int64_t from = mine && i * tall + r0 < rows ? (P.kind == 2 ? R.q[r] : R.k[r]) : -1;
                a[i] = b[i] = make_uint4(0, 0, 0, 0);
                if (from >= 0) {
                    a[i] = *reinterpret_cast<const uint4*>(src + from + 8 * va);
                    b[i] = *reinterpret_cast<const uint4*>(src + from + 8 * vb);
                }
            }
            float x[STEPS][8], y[STEPS][8];
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int r = rows * part + i * tall + r0;
                const bool real = mine && i * tall + r0 < rows && R.k[r] >= 0;
                unpack<BF16>(a[i], x[i]);
                unpack<BF16>(b[i], y[i]);
                if (real && turned) {
                    const float4* const cs = reinterpret_cast<const float4*>(A.table + R.pos[r] * 2 * A.pairs) + 2 * j;
                    const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1), s0 = __ldg(cs + 2 * turning), s1 = __ldg(cs + 2 * turning + 1);
                    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        if (NEIGHBOURS)
                            p < 4 ? turn(x[i][2 * p & 7], x[i][2 * p + 1 & 7], c[p], s[p]) : turn(y[i][2 * p & 7], y[i][2 * p + 1 & 7], c[p], s[p]);
                        else
                            turn(x[i][p], y[i][p], c[p], s[p]);
                    }
                }
                if (paged) {
#pragma unroll
                    for (int p = 0; p < 8; ++p) top = fmaxf(top, fmaxf(fabsf(x[i][p]), fabsf(y[i][p])));
                }
            }
            if (out != nullptr) {
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int r = rows * part + i * tall + r0;
                    if (!(mine && i * tall + r0 < rows && R.k[r] >= 0)) continue;
                    const uint4 xa = packed<BF16>(x[i]), xb = packed<BF16>(y[i]);
                    uint16_t* const to = out + (P.kind == 2 ? R.qo[r] : R.ko[r]);
                    *reinterpret_cast<uint4*>(to + 8 * va) = xa;
                    *reinterpret_cast<uint4*>(to + 8 * vb) = xb;
                }
            }
            if (!paged) continue;
            // ---- 8 bits: the team's largest magnitude, the scale, the codes. ----
            auto over_team = [&](float m) {
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                return m;
            };
            top = over_team(top);
            if (!(top <= FLT_MAX)) {  // infinities do not count
                top = 0.0f;
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        if (fabsf(x[i][p]) <= FLT_MAX) top = fmaxf(top, fabsf(x[i][p]));
                        if (fabsf(y[i][p]) <= FLT_MAX) top = fmaxf(top, fabsf(y[i][p]));
                    }
                top = over_team(top);
            }
            float* const scale = R.scale < 0 ? nullptr : A.scale + plane * A.s_plane + P.head * A.s_head + R.scale;
            const float had = scale != nullptr && R.first > 0 ? *scale : 0.0f;
            if (per > 1) {
                // (the two places alternate, so that one barrier a piece is enough)
                if (lane == 0) tops[flip][warp] = top;
                asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * per) : "memory");
                for (int w = 0; w < per; ++w) top = fmaxf(top, tops[flip][team * per + w]);
            }
            if (scale == nullptr) continue;
            float old;
            const float s = settle(top, had, R.first > 0, &old);
            __syncwarp();
            if (part == 0 && lane == 0) *scale = s;
            const Divide by(s);
            uint8_t* const pool = static_cast<uint8_t*>(A.pool) + plane * A.plane + P.head * A.head;
            if (old != 0.0f && mine) {
                for (int i = r0; i < rows; i += tall) {
                    const int r = rows * part + i;
                    if (r >= R.first) break;
                    uint2* const p = reinterpret_cast<uint2*>(pool + R.start + r * A.tok + 16 * j);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint2 w = p[h];
                        float f[8];
                        from_e4m3x4(w.x, f);
                        from_e4m3x4(w.y, f + 4);
#pragma unroll
                        for (int i2 = 0; i2 < 8; ++i2) f[i2] = by(f[i2] * old);
                        p[h] = packed8(f);
                    }
                }
            }
            if (by.whole) {
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
#pragma unroll
                    for (int p = 0; p < 8; ++p) x[i][p] *= by.inv, y[i][p] *= by.inv;
            } else {
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
#pragma unroll
                    for (int p = 0; p < 8; ++p) x[i][p] = by(x[i][p]), y[i][p] = by(y[i][p]);
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int r = rows * part + i * tall + r0;
                if (!(mine && i * tall + r0 < rows && R.k[r] >= 0)) continue;
                *reinterpret_cast<uint2*>(pool + R.to[r] + 8 * va) = packed8(x[i]);
                *reinterpret_cast<uint2*>(pool + R.to[r] + 8 * vb) = packed8(y[i]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
int check_rotary(const clk_rotary* r, int32_t dim)
{
    if (r->d_table == nullptr || !aligned(r->d_table, 4) || r->positions < 1 || r->positions > ((int64_t)1 << 31) || r->pairs < 1 ||
        2 * (int64_t)r->pairs > dim || (r->neighbours != 0 && r->neighbours != 1))
        return CLK_EINVAL;
    return CLK_OK;
}

// Whether rows of these shapes go by vectors.
bool fast_rows(const Turn& A, int es, bool eight)
{
    if (es != 2 || A.dim % 16 != 0 || A.dim > 128 || A.pairs % 8 != 0 || !aligned(A.table, 16)) return false;
    for (const void* p : {A.k, A.v, A.q, (const void*)A.q_out, (const void*)A.k_out})
        if (!aligned(p, 16)) return false;
    for (int64_t st : {A.layer, A.k_req, A.k_row, A.k_head, A.q_req, A.q_row, A.q_head, A.qo_req, A.qo_row, A.qo_head, A.ko_req, A.ko_row,
                       A.ko_head})
        if (st % 8 != 0) return false;
    // a vector of 8 elements of the pool: 16 bytes, or 8 of codes
    if (!aligned(A.pool, eight ? 8 : 16)) return false;
    for (int64_t st : {A.plane, A.page, A.head, A.tok})
        if (st % 8 != 0) return false;
    return true;
}

// resident: CTAs an SM, 0 for k_turn_any's grid of blocks and shares of their heads.
template <void (*kern)(Turn)>
int launch_turn(const Turn& A, int64_t units, int resident, cudaStream_t s)
{
    const size_t bytes = ((size_t)A.B + 1) * sizeof(int64_t);
    if (bytes > 32768) {
        // The limit is the kernel's, not the call's: the largest batch's, so that calls from other threads may rely on it.
        static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return CLK_ECUDA;
        const unsigned long long bit = 1ull << (dev & 63);
        if (!(ready.load(std::memory_order_relaxed) & bit) || dev > 63) {
            constexpr int most = (CLK_MAX_BATCH + 1) * (int)sizeof(int64_t);
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return CLK_ECUDA;
            ready.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    const int all = pieces(A);
    int64_t x, y = 1;
    if (resident > 0) {
        const int64_t most = resident * (int64_t)num_sms(), useful = (all + kWarps - 1) / kWarps;
        x = units >= most || units * useful >= most ? most : units * useful;
    } else {
        // Blocks are dealt out to four CTAs an SM; where there are fewer, their heads go to several CTAs.
        const int64_t most = 4 * (int64_t)num_sms();
        y = most / (units < 1 ? 1 : units);
        const int64_t useful = (all + kWarps - 1) / kWarps;
        if (y > useful) y = useful;
        if (y < 1) y = 1;
        x = units < most ? units : most;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(x < 1 ? 1 : x), (unsigned)y);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kern, A));
}

template <bool EIGHT>
int launch_kind(const Turn& A, int32_t dtype, bool neighbours, int64_t units, cudaStream_t s)
{
    if (fast_rows(A, dtype_bytes(dtype), EIGHT)) {
        const bool bf = dtype == CLK_DTYPE_BF16;
        const bool two = EIGHT && 1 << A.shift <= kWarps << team_shift(A.dim, 2);
#define CLK_GO(BF, NEIGHBOURS)                                                                   \
    do {                                                                                         \
        if (!EIGHT) return launch_turn<k_turn_rows<BF, NEIGHBOURS>>(A, units, 3, s);             \
        if (two) return launch_turn<k_turn_rows8<BF, NEIGHBOURS, 2>>(A, units, 3, s);            \
        return launch_turn<k_turn_rows8<BF, NEIGHBOURS, 4>>(A, units, 2, s);                     \
    } while (0)
        if (bf && neighbours) CLK_GO(true, true);
        if (bf) CLK_GO(true, false);
        if (neighbours) CLK_GO(false, true);
        CLK_GO(false, false);
#undef CLK_GO
    }
#define CLK_GO(T) \
    return neighbours ? launch_turn<k_turn_any<T, true, EIGHT>>(A, units, 0, s) : launch_turn<k_turn_any<T, false, EIGHT>>(A, units, 0, s)
    switch (dtype) {
    case CLK_DTYPE_BF16: CLK_GO(__nv_bfloat16);
    case CLK_DTYPE_F16: CLK_GO(__half);
    default: CLK_GO(float);
    }
#undef CLK_GO
}

}  // namespace
}  // namespace clk

using namespace clk;

extern "C" int clk_tree_rotate(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_turn* t, int32_t N,
                               const int32_t* d_nodes, const int64_t* d_mask, const int32_t* d_ctx, const clk_rotary* rotary,
                               clk_stream_t s)
{
    const int rc = check_cache_batch(h, B);
    if (rc != CLK_OK) return rc;
    if (B > CLK_MAX_BATCH || N < 1 || N > CLK_TREE_MAX || t == nullptr || rotary == nullptr) return CLK_EINVAL;
    const int es = dtype_bytes(t->dtype);
    if (es == 0 || t->dim < 1 || t->dim > 256 || t->kv_heads < 1 || t->q_heads < 1 || t->q_heads > 65535 || t->kv_heads > 65535)
        return CLK_EINVAL;
    if (check_rotary(rotary, t->dim) != CLK_OK) return CLK_EINVAL;
    for (int64_t st : {t->q_req, t->q_row, t->q_head, t->k_req, t->k_row, t->k_head, t->qo_req, t->qo_row, t->qo_head, t->ko_req, t->ko_row,
                       t->ko_head})
        if (st < 0) return CLK_EINVAL;
    if (B == 0) return CLK_OK;
    for (const void* p : {t->d_q, t->d_k, (const void*)t->d_q_out, (const void*)t->d_k_out})
        if (p == nullptr || !aligned(p, (size_t)es)) return CLK_EINVAL;
    if (!ok_i32(d_slots) || !ok_i32(d_nodes) || d_mask == nullptr || !aligned(d_mask, 8) || !aligned(d_ctx, 4)) return CLK_EINVAL;
    Turn A = {};
    A.C = h->dev;
    A.slots = d_slots;
    A.B = B;
    A.N = N;
    A.nodes = d_nodes;
    A.ctx = d_ctx;
    A.mask = d_mask;
    A.table = rotary->d_table;
    A.positions = rotary->positions;
    A.pairs = rotary->pairs;
    A.k = t->d_k;
    A.q = t->d_q;
    A.q_out = t->d_q_out;
    A.k_out = t->d_k_out;
    A.k_req = t->k_req;
    A.k_row = t->k_row;
    A.k_head = t->k_head;
    A.q_req = t->q_req;
    A.q_row = t->q_row;
    A.q_head = t->q_head;
    A.qo_req = t->qo_req;
    A.qo_row = t->qo_row;
    A.qo_head = t->qo_head;
    A.ko_req = t->ko_req;
    A.ko_row = t->ko_row;
    A.ko_head = t->ko_head;
    A.layers = 1;
    A.q_heads = t->q_heads;
    A.kv_heads = t->kv_heads;
    A.dim = t->dim;
    A.shift = 4;
    return launch_kind<false>(A, t->dtype, rotary->neighbours != 0, (int64_t)B * ((N + 15) / 16), (cudaStream_t)s);
}

extern "C" int clk_cache_append_rotary(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool,
                                       const clk_scales* scales, int32_t layer0, int32_t layers, int32_t dtype, const void* d_k,
                                       const void* d_v, int64_t layer_stride, int64_t row_stride, int64_t head_stride, int64_t N,
                                       const int64_t* d_off, const int32_t* d_path, const int32_t* d_count,
                                       const clk_rotary* rotary, const clk_turn* turn, clk_stream_t s)
{
    const int rc = check_cache_batch(h, B);
    if (rc != CLK_OK) return rc;
    const int es = dtype_bytes(dtype);
    if (B > CLK_MAX_BATCH || es == 0) return CLK_EINVAL;
    const bool eight = scales != nullptr;
    if (eight ? check_pool8(pool, scales, h->dev.page_tokens()) != CLK_OK : check_pool(pool) != CLK_OK || pool->dtype != dtype) return CLK_EINVAL;
    if (layers < 0 || layer0 < 0 || layers > pool->planes / 2 - layer0) return CLK_EINVAL;
    if (N < 0 || layer_stride < 0 || row_stride < 0 || head_stride < 0) return CLK_EINVAL;
    if (rotary != nullptr && check_rotary(rotary, pool->dim) != CLK_OK) return CLK_EINVAL;
    const bool side = turn != nullptr && (turn->d_q != nullptr || turn->d_k_out != nullptr);
    if (side) {
        if (rotary == nullptr || layers > 1 || d_path != nullptr || turn->dtype != dtype || turn->dim != pool->dim ||
            turn->kv_heads != pool->heads)
            return CLK_EINVAL;
        if ((turn->d_q != nullptr) != (turn->d_q_out != nullptr) || (turn->d_q != nullptr && (turn->q_heads < 1 || turn->q_heads > 65535)))
            return CLK_EINVAL;
        for (const void* p : {turn->d_q, (const void*)turn->d_q_out, (const void*)turn->d_k_out})
            if (!aligned(p, (size_t)es)) return CLK_EINVAL;
        for (int64_t st : {turn->q_row, turn->q_head, turn->qo_row, turn->qo_head, turn->ko_row, turn->ko_head})
            if (st < 0) return CLK_EINVAL;
    }
    // (a block's pieces, and a little more, are counted in 32 bits)
    if (2 * (int64_t)layers * pool->heads + (side && turn->d_q != nullptr ? turn->q_heads : 0) > (1 << 30)) return CLK_EINVAL;
    if (B == 0 || N == 0 || layers == 0) return CLK_OK;
    if (!ok_i32(d_slots) || !ok_i32(d_count) || d_k == nullptr || d_v == nullptr || !aligned(d_k, (size_t)es) || !aligned(d_v, (size_t)es))
        return CLK_EINVAL;
    if ((d_off != nullptr && (!aligned(d_off, 8) || d_path != nullptr)) || !aligned(d_path, 4)) return CLK_EINVAL;
    if (N > ((int64_t)1 << 40) / B) return CLK_EINVAL;
    Turn A = {};
    A.C = h->dev;
    A.slots = d_slots;
    A.B = B;
    A.N = N;
    A.off = d_off;
    A.path = d_path;
    A.count = d_count;
    if (rotary != nullptr) {
        A.table = rotary->d_table;
        A.positions = rotary->positions;
        A.pairs = rotary->pairs;
    }
    A.k = d_k;
    A.v = d_v;
    A.layer = layers > 1 ? layer_stride : 0;
    A.k_row = row_stride;
    A.k_head = pool->heads > 1 ? head_stride : 0;
    A.layers = layers;
    A.kv_heads = pool->heads;
    A.dim = pool->dim;
    if (side && turn->d_q != nullptr) {
        A.q = turn->d_q;
        A.q_out = turn->d_q_out;
        A.q_heads = turn->q_heads;
        A.q_row = turn->q_row;
        A.q_head = turn->q_head;
        A.qo_row = turn->qo_row;
        A.qo_head = turn->qo_head;
    }
    if (side && turn->d_k_out != nullptr) {
        A.k_out = turn->d_k_out;
        A.ko_row = turn->ko_row;
        A.ko_head = turn->ko_head;
    }
    A.pool = pool->d_base;
    A.plane = pool->plane_stride;
    A.page = pool->page_stride;
    A.head = pool->head_stride;
    A.tok = pool->tok_stride;
    A.layer0 = layer0;
    A.shift = 4;
    if (eight) {
        A.scale = scales->d_base;
        A.s_plane = scales->plane_stride;
        A.s_page = scales->page_stride;
        A.s_head = scales->head_stride;
        A.s_block = scales->block_stride;
        while ((1 << A.shift) < scales->tokens) ++A.shift;
    }
    // n rows lie in at most (n - 2) / T + 2 blocks
    const int64_t T = (int64_t)1 << A.shift, units = d_off != nullptr ? N / T + 2 * (int64_t)B : (int64_t)B * ((N + 2 * T - 2) / T);
    const bool neighbours = rotary != nullptr && rotary->neighbours != 0;
    return eight ? launch_kind<true>(A, dtype, neighbours, units, (cudaStream_t)s) : launch_kind<false>(A, dtype, neighbours, units, (cudaStream_t)s);
}
