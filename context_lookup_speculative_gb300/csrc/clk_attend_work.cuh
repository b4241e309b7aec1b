// How the attention kernels on the tensor cores share out their work: items,
// equal shares of all key tiles, a CTA's way through its share, and the
// joining of items that a cut fell into.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "clk.h"
#include "clk_attend.h"
#include "clk_cache.h"
#include "clk_host.h"
#include "clk_mma.cuh"

namespace clk {

constexpr int kTile = 128;  // keys of a tile, rows of a row tile
constexpr int kNear = 4;    // requests whose data a CTA keeps

struct Maps {
    CUtensorMap q, k, v, kc, vc;
};

// How a call's rows are tiled.
struct Shape {
    int32_t tok;    // tokens of a row tile: 128 / group
    int32_t block;  // tokens of an item: tok, or 2 tok for prompts
    int32_t qbox, kbox, vbox;  // tokens of a box of q, rows of a box of new keys, of new values
    int32_t ctas;
    float log2_scale;  // scale * log2(e)
    bool wide_out;     // rows of out are whole 32-byte sectors
};

// Scratch: the status of calls since it was zeroed, a flag per CTA (a count of
// calls), row statistics and partial sums, two parts a CTA.
struct Scratch {
    int32_t* status;  // latched as a cache's; a prompt without a cache has no other place for it
    uint32_t* flag;   // [ctas]
    float2* ml;       // [ctas][2][rows]
    float* sums;      // [ctas][2][DP / 4][rows][4]
};

__host__ __device__ inline int pad_dim(int dim) { return dim <= 64 ? 64 : 128; }

constexpr size_t kStatusBytes = 128;

__host__ __device__ inline size_t flag_bytes(int ctas) { return ((size_t)ctas * sizeof(uint32_t) + 127) / 128 * 128; }

__host__ __device__ inline Scratch scratch_of(void* base, int ctas, int rows)
{
    Scratch s;
    char* p = static_cast<char*>(base);
    s.status = reinterpret_cast<int32_t*>(p);
    p += kStatusBytes;
    s.flag = reinterpret_cast<uint32_t*>(p);
    p += flag_bytes(ctas);
    s.ml = reinterpret_cast<float2*>(p);
    p += (size_t)ctas * 2 * rows * sizeof(float2);
    s.sums = reinterpret_cast<float*>(p);
    return s;
}

// a / b for a >= 0, b > 0.  Small numbers go by a reciprocal that is off by
// at most one, which is a fifth of the integer division's latency.
__device__ __forceinline__ uint32_t quotient(uint32_t a, uint32_t b)
{
    if (a >= (1u << 22)) return a / b;
    uint32_t q = (uint32_t)__fdividef((float)a, (float)b);
    const int r = (int)(a - q * b);
    q += r >= (int)b ? 1 : r < 0 ? -1 : 0;
    return q;
}

__device__ __forceinline__ long long quotient(long long a, long long b)
{
    return ((a | b) >> 31) == 0 ? (long long)quotient((uint32_t)a, (uint32_t)b) : a / b;
}

// sum over i < n of floor((a i + b) / m), for m > 0 and a n + b < 2^32: the
// lattice points under a line.  The known reduction, as Euclid's algorithm
// goes: whole parts of the slope and of the start are summed at once, what is
// left of the line is read with its axes changed.
__device__ inline long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b)
{
    long long s = 0;
    while (n > 0) {
        if (a >= m) {
            const uint32_t q = quotient(a, m);
            s += ((long long)n * (n - 1) >> 1) * q;
            a -= q * m;
        }
        if (b >= m) {
            const uint32_t q = quotient(b, m);
            s += (long long)n * q;
            b -= q * m;
        }
        const uint32_t y = a * n + b;
        if (y < m) break;
        n = quotient(y, m);
        b = y - n * m;
        const uint32_t u = m;
        m = a;
        a = u;
    }
    return s;
}

// A request's tiles: per K/V head, `items` row tiles; item i has ctx_tiles
// tiles of cached keys and new_tiles(i) of new ones.
struct Reach {
    int32_t ctx, rows, slot;
    int32_t ctx_tiles, items;
    int32_t base;
};

__device__ __forceinline__ Reach reach_of(const Request& r, const Shape& S)
{
    Reach x;
    x.ctx = r.ctx;
    x.rows = r.rows;
    x.slot = r.slot;
    x.base = (int32_t)r.base;  // at most 2^30 rows
    x.ctx_tiles = (r.ctx + kTile - 1) / kTile;
    x.items = (r.rows + S.block - 1) / S.block;
    return x;
}

template <typename K>
__device__ __forceinline__ int new_tiles(const Reach& x, const Shape& S, int item)
{
    if (!K::prompt) return 1;  // at most 64 new tokens
    const int end = (item + 1) * S.block < x.rows ? (item + 1) * S.block : x.rows;
    return (end - 1) / kTile + 1;
}

// What the kinds of calls differ in.
struct Trees {
    static constexpr bool prompt = false;
    static constexpr bool in_log2 = false;  // a part's reference is a score, not yet times log2_scale
    // What an item costs besides its tiles (its result, the next one's start),
    // in tiles: about 6,000 cycles beside 2,100 a tile with prompts and 4,300
    // beside 1,800 with trees, rows of 64.  Counting it balances short items
    // with long ones.  Measured without and with: 16 prompts of 500 to 1,500 tokens
    // (24/4 heads of 64) 141 and 117 us, the same behind prefixes of up to 8,192
    // (100 to 2,000 tokens) 561 and 460, 256 requests of 300 to 4,096 tokens and 13
    // nodes 128 and 117, one token over 2,048 rows (32/8 heads of 128) 13.7 and 13.1.
    static constexpr int extra = 3;
    // Items of at most so many tiles are not cut: joining parts takes 10,000
    // cycles and more.  They go to the CTA that holds their middle unit.
    // Measured on prompts without a limit, of 8 and of 16 tiles: one of 1,000
    // tokens (32/8 heads of 128) 34.9, 22.2, 22.1 us, one of 4,000 118, 118, 120;
    // 16 of 500 to 1,500 221, 209, 208, with 24/4 heads of 64 126, 123, 117.  256
    // requests of 64 to 512 tokens and 13 nodes (24/4 heads of 64): without 67.9,
    // of 2 tiles 68.3, of 4 62.2 us.
    static constexpr int whole = 4;
};
// Over a cache in 8 bits an item's ends (its Q in parts before its first scores)
// cost more beside its tiles.  Measured with 3, 5 and 8 more units: 64 requests
// of 2,000 to 32,000 tokens and 16 nodes (32/8 heads of 128) 525, 519, 517 us,
// 256 of 300 to 4,096 and 13 nodes (24/4 heads of 64) 204, 202, 195; one token
// over 2,048 rows 24.7, 28.7, 26.6.  Items of up to 4, 6 and 12 tiles uncut: 256
// requests of 64 to 512 tokens and 13 nodes 111, 103, 102, 64 of 64 to 1,024 and
// 16 nodes (32/8 heads of 128) 81, 81, 77, the 256 longer ones 195, 195, 196.
struct Trees8 {
    static constexpr bool prompt = false, in_log2 = true;
    static constexpr int extra = 8, whole = 6;
};
struct Prompts {
    static constexpr bool prompt = true, in_log2 = false;
    static constexpr int extra = 4, whole = 16;
};

// Units of the items before `item` of one K/V head.
template <typename K>
__device__ __forceinline__ long long units_before(const Reach& x, const Shape& S, int item)
{
    if (!K::prompt) return (long long)item * (x.ctx_tiles + 1 + K::extra);
    if (item <= 0) return 0;
    const bool all = item >= x.items;
    const int whole = all ? x.items - 1 : item;
    long long n = (long long)item * (x.ctx_tiles + K::extra) + whole + floor_sum(whole, kTile, S.block, S.block - 1);
    if (all) n += (x.rows - 1) / kTile + 1;
    return n;
}

template <typename K>
__device__ __forceinline__ long long units_of(const Reach& x, const Shape& S)
{
    return x.items == 0 ? 0 : units_before<K>(x, S, x.items);
}

// `all` units in shares of q or q + 1: the first r CTAs have one more.
struct Cuts {
    long long q;
    int r;
    __device__ Cuts(long long all, int ctas)
    {
        q = ctas > 0 ? quotient(all, ctas) : 0;
        r = (int)(all - q * ctas);
    }
    __device__ long long begin(int c) const { return q * c + (c < r ? c : r); }
    // the CTA whose share holds unit g
    __device__ int holder(long long g) const
    {
        const long long big = (q + 1) * r;
        return (int)(g < big ? quotient(g, q + 1) : r + quotient(g - big, q));
    }
};

// What a CTA knows after planning (in shared memory).
struct Plan {
    long long all, g0, g1;  // units in all, this CTA's share
    int ctas;               // CTAs that have a share
    int b, h, item, at;     // where the share begins: unit `at` of the item
    uint32_t call;          // this CTA's flag before this call
    long long began;        // when the CTA began, in its clocks
};

// An item whose tiles lie in several CTAs' shares.
struct Cut {
    Reach x;
    int b, h, item, total;  // total: its tiles, 0 for none
    long long begin;        // its first unit
};

// The CTA's way through its share, segment by segment (an item's tiles t0 ..
// t1-1), the same in every warp.  The softmax warps keep theirs in shared
// memory: their registers are full.
template <typename K>
struct Walk {
    Reach x;
    int b, h, item, t0, t1, total;
    int left;  // units of the share from this segment's on; 0 at the end
    int took;  // this segment's units

    __device__ void start(const Attend& A, const Shape& S, const Plan& P, const Reach* near)
    {
        left = (int)(P.g1 - P.g0);
        took = 0;
        b = P.b;
        h = P.h;
        item = P.item;
        if (left == 0) return;
        load(A, S, P, near);
        cut(S, P.at);
        if (t0 == t1) next(A, S, P, near);
    }
    __device__ void load(const Attend& A, const Shape& S, const Plan& P, const Reach* near)
    {
        const int i = b - P.b;
        x = i < kNear ? near[i] : reach_of(attend_request(A, b, false), S);
    }
    // From unit `at` of the item on, as far as the share goes.
    __device__ void cut(const Shape& S, int at)
    {
        constexpr int extra = K::extra;
        total = x.ctx_tiles + new_tiles<K>(x, S, item);
        took = extra + total - at < left ? extra + total - at : left;
        if (total <= K::whole) {
            const int middle = (extra + total) / 2;
            t0 = 0;
            t1 = at <= middle && middle < at + took ? total : 0;
        } else {
            t0 = at > extra ? at - extra : 0;
            t1 = at + took > extra ? at + took - extra : 0;
        }
    }
    // The next segment that has tiles.
    __device__ void next(const Attend& A, const Shape& S, const Plan& P, const Reach* near)
    {
        do {
            left -= took;
            if (left <= 0) {
                left = 0;
                return;
            }
            if (++item == x.items) {
                item = 0;
                if (++h == A.kv_heads) {
                    h = 0;
                    do {
                        ++b;
                        load(A, S, P, near);
                    } while (x.items == 0);
                }
            }
            cut(S, 0);
        } while (t0 == t1);
    }
    // Tiles [t0, last(s)) of this segment are stream s's, with prompts.
    __device__ int last(const Shape& S, int s) const
    {
        const int first = item * S.block + s * S.tok;
        if (first >= x.rows) return t0;
        const int end = first + S.tok < x.rows ? first + S.tok : x.rows;
        const int n = x.ctx_tiles + (end - 1) / kTile + 1;
        return n < t0 ? t0 : n < t1 ? n : t1;
    }
};

// A wait has run out: the call's results are not whole.
__device__ __forceinline__ void gave_up(const Attend& A, const Scratch& W)
{
    latch(W.status, CLK_ECUDA, -1);
    if (A.C.status != nullptr) latch(A.C.status, CLK_ECUDA, -1);
}

template <int N>
struct Count {
    static constexpr int value = N;
};

// All requests' tiles, this CTA's share and where it begins: `plan`, the first
// requests of the share in `near`.  `sums` is scratch for a value a warp; `warp` the
// thread's.  (The caller's own where its registers are full: shuffled again it
// spilled in the trees' kernel over 16 bits, rows of 64: 256 requests 123 us, 121 so.)
template <typename K, int THREADS>
__device__ __forceinline__ void make_plan(const Attend& A, const Shape& S, long long* sums, Plan& plan, Reach* near, Cut* cut,
                                          volatile int* stop, uint32_t call, long long began, int warp)
{
    constexpr int kThreads = THREADS, kWarps = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31;
    const bool once = A.B <= kThreads;  // the batch is seen in one pass
    long long all = 0;
    int ctas = 0;
    Cuts cuts(0, 0);
    Reach x{};
    for (int pass = 0;; ++pass) {
        long long before = 0;
        for (int at = 0; at < A.B; at += kThreads) {
            const int b = at + tid;
            long long each = 0;  // units of one K/V head
            if (b < A.B) {
                x = reach_of(attend_request(A, b, pass == 0 && blockIdx.x == 0), S);
                each = units_of<K>(x, S);
            }
            const long long u = each * A.kv_heads;
            long long y = u;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const long long z = __shfl_up_sync(0xffffffffu, y, d);
                if (lane >= d) y += z;
            }
            if (lane == 31) sums[warp] = y;
            __syncthreads();
            long long mine = before + y - u;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) mine += sums[w];
                before += sums[w];
            }
            if (once) all = before;
            if (once || pass == 1) {
                // The warp that has the share's first request finds the place in it.
                if (at == 0) {
                    ctas = all < S.ctas ? (int)all : S.ctas;
                    cuts = Cuts(all, ctas);
                }
                const long long g0 = (int)blockIdx.x < ctas ? cuts.begin(blockIdx.x) : all;
                const unsigned who = __ballot_sync(0xffffffffu, u > 0 && mine <= g0 && g0 < mine + u);
                if (who != 0) {
                    const int src = __ffs((int)who) - 1;
                    Reach z;
                    z.rows = __shfl_sync(0xffffffffu, x.rows, src);
                    z.ctx_tiles = __shfl_sync(0xffffffffu, x.ctx_tiles, src);
                    z.items = __shfl_sync(0xffffffffu, x.items, src);
                    const long long off = __shfl_sync(0xffffffffu, g0 - mine, src), per = __shfl_sync(0xffffffffu, each, src);
                    const int h = (int)quotient(off, per);
                    const long long o = off - h * per;
                    // the last item with units_before <= o, and those units
                    int lo = 0;
                    long long below = 0;
                    if (!K::prompt) {
                        lo = (int)quotient(o, z.ctx_tiles + 1 + K::extra);
                        below = units_before<K>(z, S, lo);
                    }
                    for (int span = K::prompt ? z.items : 1; span > 1;) {  // 32 ways at a time
                        const int step = (span + 31) / 32, end = lo + span;
                        const long long n = lane * step < span ? units_before<K>(z, S, lo + lane * step) : o + 1;
                        const int last = __popc(__ballot_sync(0xffffffffu, n <= o)) - 1;
                        below = __shfl_sync(0xffffffffu, n, last);
                        lo += last * step;
                        span = lo + step < end ? step : end - lo;
                    }
                    if (lane == 0) {
                        plan.b = at + 32 * warp + src;
                        plan.h = h;
                        plan.item = lo;
                        plan.at = (int)(o - below);
                    }
                }
            }
            __syncthreads();
        }
        if (pass == 0) all = before;
        if (once || pass == 1) break;
    }
    const bool busy = (int)blockIdx.x < ctas;
    if (tid == 0) {
        plan.all = all;
        plan.ctas = ctas;
        plan.g0 = busy ? cuts.begin(blockIdx.x) : all;
        plan.g1 = busy ? cuts.begin(blockIdx.x + 1) : all;
        plan.call = call;
        plan.began = began;
        *stop = 0;
        cut[0].total = cut[1].total = 0;
    }
    if (busy) {
        if (once) {
            const int i = tid - plan.b;
            if (i >= 0 && i < kNear) near[i] = x;
        } else if (tid < kNear && plan.b + tid < A.B) {
            near[tid] = reach_of(attend_request(A, plan.b + tid, false), S);
        }
    }
}

// x 2^d, d <= 0, where 2^d may be less than a float32 holds.
__device__ __forceinline__ float moved(float x, float d)
{
    const float half = exp2_fast(0.5f * d);
    return x * half * half;
}

// This CTA's share of an item whose tiles lie in several CTAs' shares.
template <int DP, bool BF16, typename K, int THREADS>
__device__ __forceinline__ void join_item(const Attend& A, const Shape& S, const Scratch& W, const Plan& plan, const Cuts& cuts,
                                          const Cut& cut, volatile int* stop)
{
    constexpr int rows = K::prompt ? 2 * kTile : kTile, kThreads = THREADS;
    const int tid = threadIdx.x;
    const long long tile0 = cut.begin + K::extra;
    const int c0 = cuts.holder(tile0), c1 = cuts.holder(tile0 + cut.total - 1), parts = c1 - c0 + 1;
    auto part = [&](int c) { return 2 * (c0 + c) + (c == 0 ? 1 : 0); };
    // All CTAs of the grid are resident, and none waits before it has raised its own flag.  Shares are equal but not
    // equally long: a CTA waits, beyond the usual limit, for as long as its own share took.
    for (int c = tid; c < parts; c += kThreads) {
        uint32_t seen;
        const long long t0 = clock64();
        for (;;) {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(seen) : "l"(W.flag + c0 + c) : "memory");
            if (seen != plan.call || *stop != 0) break;
            if (clock64() - t0 > kWaitClocks + (t0 - plan.began)) *stop = 1;
        }
    }
    __syncthreads();
    if (*stop != 0) {
        if (tid == 0) gave_up(A, W);
        return;
    }
    const int quads = A.dim / 4;
    const int left = cut.x.rows - cut.item * S.block, tokens = left < S.block ? left : S.block;
    const int used = tokens * A.group;   // rows of the item, tile after tile
    const int full = S.tok * A.group;    // rows in use of a whole row tile
    const int mine = (int)blockIdx.x - c0;
    const int all = used * quads;
    const int lo = (int)((long long)all * mine / parts), hi = (int)((long long)all * (mine + 1) / parts);
    const float4* const sums = reinterpret_cast<const float4*>(W.sums);
    const float cs = K::in_log2 ? 1.0f : S.log2_scale;
    // U elements of four columns a thread, F parts of each: eight loads in flight.
    auto rows_of = [&](auto fc, auto uc) {
        constexpr int F = decltype(fc)::value, U = decltype(uc)::value;
        for (int i0 = lo + tid; i0 < hi; i0 += U * kThreads) {
            float top[U], l[U];
            float4 o[U];
            int64_t at[U];
            int row[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kThreads < hi ? i0 + u * kThreads : i0;
                const int q = (int)quotient((uint32_t)i, (uint32_t)used), r = i - q * used;
                row[u] = r < full ? r : kTile + r - full;
                at[u] = (int64_t)q * rows + row[u];
                top[u] = -INFINITY;
                l[u] = 0.0f;
                o[u] = make_float4(0, 0, 0, 0);
            }
            // in the order of the parts
            for (int c = 0; c < parts; c += F) {
                float2 ml[U][F];
                float4 v[U][F];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int e = 0; e < F; ++e) {
                        // past the end the last part is read again, with no weight
                        const int64_t p = part(c + e < parts ? c + e : parts - 1);
                        ml[u][e] = __ldcg(W.ml + p * rows + row[u]);
                        v[u][e] = __ldcg(sums + p * (DP / 4) * rows + at[u]);
                    }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float to = top[u];
#pragma unroll
                    for (int e = 0; e < F; ++e) to = fmaxf(to, ml[u][e].x);
                    const float f = top[u] == -INFINITY ? 0.0f : exp2_fast((top[u] - to) * cs);
                    const float top_was = top[u];
                    top[u] = to;
                    l[u] = !K::in_log2 ? l[u] * f : top_was == -INFINITY ? 0.0f : moved(l[u], top_was - to);
                    o[u] = make_float4(o[u].x * f, o[u].y * f, o[u].z * f, o[u].w * f);
#pragma unroll
                    for (int e = 0; e < F; ++e) {
                        // a part that saw nothing has no weight (and its reference is -inf)
                        const bool use = c + e < parts && !(ml[u][e].x == -INFINITY && ml[u][e].y == 0.0f);
                        const float g = exp2_fast((ml[u][e].x - to) * cs);
                        l[u] += !use ? 0.0f : K::in_log2 ? moved(ml[u][e].y, ml[u][e].x - to) : ml[u][e].y * g;
                        o[u].x += use ? v[u][e].x * g : 0.0f;
                        o[u].y += use ? v[u][e].y * g : 0.0f;
                        o[u].z += use ? v[u][e].z * g : 0.0f;
                        o[u].w += use ? v[u][e].w * g : 0.0f;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * kThreads;
                if (i >= hi) break;
                const int q = (int)quotient((uint32_t)i, (uint32_t)used), r = i - q * used;
                const float inv = l[u] == 0.0f ? 0.0f : 1.0f / l[u];
                const int rt = (int)quotient((uint32_t)r, (uint32_t)A.group);
                const int tok = cut.item * S.block + rt, head = cut.h * A.group + r - rt * A.group;
                const int64_t out_row = (K::prompt ? (int64_t)cut.x.base : (int64_t)cut.b * A.N) + tok;
                uint2 y;
                y.x = pack2<BF16>(o[u].x * inv, o[u].y * inv);
                y.y = pack2<BF16>(o[u].z * inv, o[u].w * inv);
                *reinterpret_cast<uint2*>(static_cast<char*>(A.out) + ((out_row * A.q_heads + head) * A.dim + 4 * q) * 2) = y;
            }
        }
    };
    if (parts <= 2)
        rows_of(Count<2>{}, Count<4>{});
    else
        rows_of(Count<8>{}, Count<1>{});
}

// Trees over a cache in 8 bits (clk_attend_tree8.cu).
int attend_tree8_launch(const Attend& A, const Shape& S, const Maps& M, void* scratch, cudaStream_t s);

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encoder()
{
    static std::atomic<void*> found{nullptr};
    void* p = found.load(std::memory_order_acquire);
    if (p == nullptr) {
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &st) != cudaSuccess ||
            st != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(p, std::memory_order_release);
    }
    return reinterpret_cast<EncodeFn>(p);
}

// A map over [n3][n2][n1][dim] elements with the given strides (in
// elements), copied in boxes of b0 x b1 x b2 (x 1).
inline bool encode(EncodeFn f, CUtensorMap* m, int32_t dtype, const void* base, int64_t dim, const int64_t n[3], const int64_t st[3],
            int b0, int b1, int b2, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B)
{
    const cuuint64_t es = dtype == CLK_DTYPE_E4M3 ? 1 : 2;
    const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)n[0], (cuuint64_t)n[1], (cuuint64_t)n[2]};
    cuuint64_t strides[3];
    // the stride of an axis of one is not used; it still has to be a valid one
    for (int i = 0; i < 3; ++i) strides[i] = n[i] > 1 ? (cuuint64_t)st[i] * es : 256;
    const cuuint32_t box[4] = {(cuuint32_t)b0, (cuuint32_t)b1, (cuuint32_t)b2, 1}, one[4] = {1, 1, 1, 1};
    const CUtensorMapDataType type = es == 1                    ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : dtype == CLK_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return f(m, type, 4, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A stride (in elements, so many to 16 bytes) that a tensor map can take, for an axis of n.
inline bool map_stride(int64_t st, int64_t n, int per = 8) { return n <= 1 || (st > 0 && st % per == 0 && st < ((int64_t)1 << 38)); }

}  // namespace clk
