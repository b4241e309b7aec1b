// Attention of new tokens over a paged cache on the tensor cores (sm_103a).
//
// Rows.  The query heads that share a K/V head are packed with the tokens
// into the rows of one product: row r of a tile is token r / group, head
// r % group of the group, so K and V are read once for all of them and a
// step's 16 nodes times a group of 8 fill the 128 rows.
//
// Work.  An item is one (request, K/V head, row tile); its work is a list of
// 128-key tiles, those of the cached rows first, then those of the new
// tokens.  All items' tiles in order, with a few units before each item for
// what it costs besides them, form one line, which the CTAs (one per SM) cut
// into equal shares: ragged contexts, causal rows of every length
// and a single long request all balance, whatever the batch.  An item that
// a cut falls into is left as partial results (float32 sums and the
// softmax's reference and sum per row).  The grid is launched cooperatively;
// a CTA that has written its parts raises its flag, waits for the flags of
// the CTAs that share its cut items (there are at most two), and joins its
// share of their rows, the parts in the order of their keys.
//
// A CTA.  Two warps copy tiles into two rings in shared memory (pages and
// packed rows are boxes of tensor maps, 128-byte swizzle); one warp issues the
// products; two groups of four warps do the softmax, a thread per row; one
// warp looks after V tiles.  The two groups work on two accumulator
// streams so that the tensor cores run on one while the other is
// exponentiated: for trees the streams take alternate key tiles of one row
// tile, for prompts two row tiles share every key tile.  Scores
// S = Q K^T arrive in tensor memory in float32; a thread reads its row,
// keeps the running maximum and sum, and writes the weights P back over S in
// 16 bits, from where the second product O += P V takes them.  O is rescaled
// only when a row's maximum has grown by more than a factor of 2^8 over the
// reference in use: between that, weights are up to 2^8 (which costs no
// precision in floating point).  float16 weights carry another factor of
// 2^7, so that small ones keep their bits (2^15 stays below the type's
// largest).
//
// What is not visible.  Scores of hidden keys are replaced by -inf, so K may
// hold anything there; but 0 * V is not 0 for an infinity or a NaN.  So the V
// warps clear the rows past a tile's end (the rest of a page, the next
// request's tokens), and in tiles of new tokens whose keys not all rows see,
// they clear rows that are not finite and note them: a row that sees such a
// key gets NaN for its sum.
//
// Bounds and figures.  Trees stream K and V: 64 requests of 2,000 to 32,000
// tokens (heads 32/8 of 128, 4.8 GB) 690 us, 8 of 262,144 (16/2 heads) 317 us,
// 6.9 TB/s; one token over 2,048 rows 14 us, launch, planning and joining.
// Prompts of rows of 128 are bound by the products: 25,000 tokens 3.0 to
// 3.1 ms, 1,640 to 1,720 TFLOP/s of the causal half, a step of two row tiles
// 2,350 cycles of which 2,048 are products.  Rows of 64 have half the products
// a weight, and the softmax bounds them: 2,100 cycles a step, of which the
// products are 1,024; so their P has columns of its own beside S (the next
// scores need not wait for the values' product) and the maximum is only looked
// for when a tile's sum has grown too large.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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
namespace {

constexpr int kTile = 128;     // keys of a tile, rows of a row tile
constexpr int kWarps = 12;     // 8 softmax, 2 copies, 1 products, 1 V tiles
constexpr int kThreads = 32 * kWarps;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kCopyWarp2 = 10, kValueWarp = 11;
constexpr int kNear = 4;            // requests whose data a CTA keeps

struct Maps {
    CUtensorMap q, k, v, kc, vc;
};

// How a call's rows are tiled.
struct Shape {
    int32_t tok;    // tokens of a row tile: 128 / group
    int32_t block;  // tokens of an item: tok, or 2 tok for prompts
    int32_t qbox, kbox;  // tokens of a box of q, rows of a box of new keys
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
__device__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b)
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

template <bool PROMPT>
__device__ __forceinline__ int new_tiles(const Reach& x, const Shape& S, int item)
{
    if (!PROMPT) return 1;  // at most 64 new tokens
    const int end = (item + 1) * S.block < x.rows ? (item + 1) * S.block : x.rows;
    return (end - 1) / kTile + 1;
}

// What an item costs besides its tiles (its result, the next one's start),
// in tiles: about 6,000 cycles beside 2,100 a tile with prompts and 4,300
// beside 1,800 with trees, rows of 64.  Counting it balances short items
// with long ones.  Measured without and with: 16 prompts of 500 to 1,500 tokens
// (24/4 heads of 64) 141 and 117 us, the same behind prefixes of up to 8,192
// (100 to 2,000 tokens) 561 and 460, 256 requests of 300 to 4,096 tokens and 13
// nodes 128 and 117, one token over 2,048 rows (32/8 heads of 128) 13.7 and 13.1.
template <bool PROMPT>
constexpr int kExtra = PROMPT ? 4 : 3;

// Items of at most so many tiles are not cut: joining parts takes 10,000
// cycles and more.  They go to the CTA that holds their middle unit.
// Measured on prompts without a limit, of 8 and of 16 tiles: one of 1,000
// tokens (32/8 heads of 128) 34.9, 22.2, 22.1 us, one of 4,000 118, 118, 120;
// 16 of 500 to 1,500 221, 209, 208, with 24/4 heads of 64 126, 123, 117.  256
// requests of 64 to 512 tokens and 13 nodes (24/4 heads of 64): without 67.9,
// of 2 tiles 68.3, of 4 62.2 us.
template <bool PROMPT>
constexpr int kWhole = PROMPT ? 16 : 4;

// Units of the items before `item` of one K/V head.
template <bool PROMPT>
__device__ __forceinline__ long long units_before(const Reach& x, const Shape& S, int item)
{
    if (!PROMPT) return (long long)item * (x.ctx_tiles + 1 + kExtra<PROMPT>);
    if (item <= 0) return 0;
    const bool all = item >= x.items;
    const int whole = all ? x.items - 1 : item;
    long long n = (long long)item * (x.ctx_tiles + kExtra<PROMPT>) + whole + floor_sum(whole, kTile, S.block, S.block - 1);
    if (all) n += (x.rows - 1) / kTile + 1;
    return n;
}

template <bool PROMPT>
__device__ __forceinline__ long long units_of(const Reach& x, const Shape& S)
{
    return x.items == 0 ? 0 : units_before<PROMPT>(x, S, x.items);
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
template <bool PROMPT>
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
        constexpr int extra = kExtra<PROMPT>;
        total = x.ctx_tiles + new_tiles<PROMPT>(x, S, item);
        took = extra + total - at < left ? extra + total - at : left;
        if (total <= kWhole<PROMPT>) {
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

template <int DP, bool PROMPT>
struct Lay {
    static constexpr int kHalves = DP / 64;
    static constexpr int kHalf = kTile * 128;  // bytes of 64 columns of a tile
    static constexpr int kBytes = kHalves * kHalf;
    // Rows of 64 leave room in tensor memory for weights beside the scores (two streams of 128 + 64 + 64
    // columns), so that the next scores are computed while this tile's are exponentiated; with rows of 128
    // the weights lie over the scores.
    static constexpr bool kApart = DP == 64;
    static constexpr int kQ = PROMPT ? 2 : 1;                      // row tiles of an item
    static constexpr int kQB = DP == 128 && PROMPT ? 1 : 2;        // items whose Q is held
    static constexpr int kK = DP == 128 ? (PROMPT ? 3 : 2) : (PROMPT ? 5 : 4);  // K tiles in the ring
    static constexpr int kV = DP == 128 ? 2 : (PROMPT ? 5 : 4);
    static constexpr int kTiles = kQ * kQB + kK + kV;
    // after the tiles
    static constexpr int oKFull = kTiles * kBytes, oKEmpty = oKFull + 8 * kK;
    static constexpr int oVFull = oKEmpty + 8 * kK, oVReady = oVFull + 8 * kV, oVEmpty = oVReady + 8 * kV;
    static constexpr int oQFull = oVEmpty + 8 * kV, oQEmpty = oQFull + 8 * kQB;
    static constexpr int oSFull = oQEmpty + 8 * kQB, oSFree = oSFull + 16, oPReady = oSFree + 16, oPHalf = oPReady + 16, oODone = oPHalf + 16;
    static constexpr int oStatReady = oODone + 16, oDrain = oStatReady + 8;
    static constexpr int oBars = oDrain + 8;  // end of the barriers
    static constexpr int oBad = (oBars + 15) / 16 * 16;               // uint32[kV][4]
    static constexpr int oNear = oBad + 16 * kV;                      // Reach[kNear]
    static constexpr int oPlan = oNear + kNear * (int)sizeof(Reach);  // Plan, stop flag, tmem address
    static constexpr int oCut = oPlan + (int)sizeof(Plan);            // Cut[2]: of items that end here, that begin here
    static constexpr int oWalk = (oCut + 2 * (int)sizeof(Cut) + 7) / 8 * 8;  // Walk[8]
    static constexpr int oStop = oWalk + 8 * (int)sizeof(Walk<PROMPT>), oTmem = oStop + 4;
    static constexpr int oStat = (oTmem + 4 + 15) / 16 * 16;          // float2[2][128] for trees
    static constexpr int kTotal = oStat + (PROMPT ? 0 : 2 * kTile * 8);
    static_assert(kTotal <= 232448, "shared memory");
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

// This CTA's share of an item whose tiles lie in several CTAs' shares.
template <int DP, bool BF16, bool PROMPT>
__device__ __forceinline__ void join_item(const Attend& A, const Shape& S, const Scratch& W, const Plan& plan, const Cuts& cuts,
                                          const Cut& cut, volatile int* stop)
{
    constexpr int rows = PROMPT ? 2 * kTile : kTile;
    const int tid = threadIdx.x;
    const long long tile0 = cut.begin + kExtra<PROMPT>;
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
    const float cs = S.log2_scale;
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
                    top[u] = to;
                    l[u] *= f;
                    o[u] = make_float4(o[u].x * f, o[u].y * f, o[u].z * f, o[u].w * f);
#pragma unroll
                    for (int e = 0; e < F; ++e) {
                        // a part that saw nothing has no weight (and its reference is -inf)
                        const bool use = c + e < parts && !(ml[u][e].x == -INFINITY && ml[u][e].y == 0.0f);
                        const float g = exp2_fast((ml[u][e].x - to) * cs);
                        l[u] += use ? ml[u][e].y * g : 0.0f;
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
                const int64_t out_row = (PROMPT ? (int64_t)cut.x.base : (int64_t)cut.b * A.N) + tok;
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

template <int DP, bool BF16, bool PROMPT>
__global__ void __launch_bounds__(kThreads, 1) k_attend(const __grid_constant__ Maps M, const __grid_constant__ Attend A,
                                                        const __grid_constant__ Shape S, void* scratch)
{
    using L = Lay<DP, PROMPT>;
    extern __shared__ __align__(1024) char sm[];
    // the shuffle tells the compiler that a warp has one role
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = smem_addr(sm);
    Plan& plan = *reinterpret_cast<Plan*>(sm + L::oPlan);
    Reach* const near = reinterpret_cast<Reach*>(sm + L::oNear);
    Cut* const cut = reinterpret_cast<Cut*>(sm + L::oCut);
    volatile int* const stop = reinterpret_cast<volatile int*>(sm + L::oStop);
    volatile uint32_t* const bad = reinterpret_cast<volatile uint32_t*>(sm + L::oBad);
    const Scratch W = scratch_of(scratch, S.ctas, PROMPT ? 2 * kTile : kTile);

    const uint32_t call = tid == 0 ? __ldcg(W.flag + blockIdx.x) : 0;
    const long long began = clock64();
    // ---- Start: tensor memory, barriers and descriptors, while the requests' data is on its way. ----
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + L::oTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (warp == kCopyWarp) {
        if (lane < 5)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<const char*>(&M) + lane * sizeof(CUtensorMap)) : "memory");
    } else if (tid == 32 * kValueWarp) {
        for (int i = 0; i < L::kK; ++i) {
            bar_init(base + L::oKFull + 8 * i, 1);
            bar_init(base + L::oKEmpty + 8 * i, 1);
        }
        for (int i = 0; i < L::kV; ++i) {
            bar_init(base + L::oVFull + 8 * i, 1);
            bar_init(base + L::oVReady + 8 * i, 1);
            bar_init(base + L::oVEmpty + 8 * i, 1);
        }
        for (int i = 0; i < L::kQB; ++i) {
            bar_init(base + L::oQFull + 8 * i, 1);
            bar_init(base + L::oQEmpty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(base + L::oSFull + 8 * i, 1);
            bar_init(base + L::oSFree + 8 * i, 4);
            bar_init(base + L::oPHalf + 8 * i, 4);
            bar_init(base + L::oPReady + 8 * i, 4);
            bar_init(base + L::oODone + 8 * i, 1);
        }
        bar_init(base + L::oStatReady, 8);
        bar_init(base + L::oDrain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    // ---- Plan: all requests' tiles, this CTA's share, where it begins. ----
    {
        long long* const sums = reinterpret_cast<long long*>(sm);  // the rings are not in use yet
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
                    each = units_of<PROMPT>(x, S);
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
                        if (!PROMPT) {
                            lo = (int)quotient(o, z.ctx_tiles + 1 + kExtra<PROMPT>);
                            below = units_before<PROMPT>(z, S, lo);
                        }
                        for (int span = PROMPT ? z.items : 1; span > 1;) {  // 32 ways at a time
                            const int step = (span + 31) / 32, end = lo + span;
                            const long long n = lane * step < span ? units_before<PROMPT>(z, S, lo + lane * step) : o + 1;
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
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the planning scratch lies where tiles go
    tmem_before();
    __syncthreads();
    tmem_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::oTmem);
    const uint32_t qs = base, ks = base + L::kQ * L::kQB * L::kBytes, vs = ks + L::kK * L::kBytes;

    // Registers: 384 threads x 168 at launch; 256 x 208 + 128 x 80 after the split.
    if (warp < kCopyWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // ---- Softmax: a thread per row. ----
        const int s = warp >> 2, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t tS = lanes + 128 * s, tO = lanes + 256 + s * DP, tP = L::kApart ? lanes + 384 + 64 * s : tS;
        const int tk = row / A.group, g = row - tk * A.group;  // token of the row tile, head of the group
        const float cs = S.log2_scale;
        constexpr float lift = BF16 ? 0.0f : 7.0f;
        // A weight is exp2(x cs - ref cs).  One fused operation with ref cs computed beforehand is off by that product's
        // rounding: up to here at most 2^-17 of a weight; in the millions by whole powers of two, each reference by
        // another one, so that weights overflow or vanish.  Beyond, ref is taken off x itself, which is exact where it
        // counts.  Likewise references are compared as scores wherever sums meet (streams, parts), not times cs.
        constexpr float far_off = 256.0f;
        uint32_t sp = 0, od = 0;
        int gi = 0;
        bool ok = true;
        Walk<PROMPT>& w = reinterpret_cast<Walk<PROMPT>*>(sm + L::oWalk)[warp];
        if (lane == 0) w.start(A, S, plan, near);
        __syncwarp();
        while (ok && w.left > 0) {
            const int len = w.t1 - w.t0, t0 = w.t0;
            const int mine = PROMPT ? w.last(S, s) - t0 : (len + 1 - s) / 2;
            const int first = w.item * S.block + (PROMPT ? s * S.tok : 0);  // first token of the row tile
            const int token = first + tk;
            const int ctx = w.x.ctx, ctx_tiles = w.x.ctx_tiles;
            const bool real = tk < S.tok && token < w.x.rows;
            unsigned long long seen = 0;
            if (!PROMPT && real && w.t1 > ctx_tiles) {
                seen = (unsigned long long)A.mask[(int64_t)w.b * A.N + token];
                if (w.x.rows < 64) seen &= (1ull << w.x.rows) - 1;
            }
            float ref = -INFINITY, sum = 0.0f;
            bool settled = false;  // every row has a reference, and none is far off
            bool far = false;      // some row's is far off
            uint32_t x[kTile];     // a tile's scores
            float2 both;           // sums of its weights
            int t = 0, n0 = 0;
            bool cached = false;
            auto away = [&] { return ref != -INFINITY && fabsf(ref * cs) > far_off; };
            // Tile j's scores, those of hidden keys replaced.
            auto fetch = [&](int j) -> bool {
                t = t0 + (PROMPT ? j : 2 * j + s);
                if (!warp_wait(base + L::oSFull + 8 * s, sp, stop)) return false;
                sp ^= 1;
                tmem_after();
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_load(tS + 32 * c, x + 32 * c);
                tmem_load_wait();
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_loaded(x + 32 * c);
                if (L::kApart) {
                    tmem_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(base + L::oSFree + 8 * s);
                }
                // Hidden keys: a limit for most tiles, a mask for a tree's.
                cached = t < ctx_tiles;
                n0 = (t - ctx_tiles) * kTile;
                if (cached || PROMPT) {
                    const int most = cached ? ctx - t * kTile : n0 + kTile - 1 > first ? token - n0 + 1 : kTile;
                    if (!cached ? n0 + kTile - 1 > first : most < kTile) {
#pragma unroll
                        for (int c = 0; c < kTile; ++c)
                            if (c >= most) x[c] = 0xff800000u;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        if (!(seen >> c & 1)) x[c] = 0xff800000u;
#pragma unroll
                    for (int c = 64; c < kTile; ++c) x[c] = 0xff800000u;
                }
                if (L::kApart && j > 0) {
                    // this stream's last product is done with O and the weights
                    if (!warp_wait(base + L::oODone + 8 * s, od, stop)) return false;
                    od ^= 1;
                    tmem_after();
                }
                return true;
            };
            // The references follow tile j's maxima where these have grown by more than a factor of 2^8.
            auto follow = [&](int j) {
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < kTile; c += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        m[e] = max3(m[e], __uint_as_float(x[c + 2 * e]), __uint_as_float(x[c + 2 * e + 1]));
                const float top = max3(m[0], m[1], fmaxf(m[2], m[3]));
                const bool grow = (top - ref) * cs > 8.0f;
                if (!__any_sync(0xffffffffu, grow)) return;
                const float to = grow ? top : ref;
                const float fix = grow ? exp2_fast((ref - to) * cs) : 1.0f;
                ref = to;
                sum *= fix;
                if (j > 0) {
                    // O is complete: weights over the scores mean that these scores' product was issued
                    // after this stream's last P V; else it was waited for.
#pragma unroll
                    for (int c = 0; c < DP / 16; ++c) {
                        uint32_t o[16];
                        tmem_load16(tO + 16 * c, o);
                        tmem_load_wait();
                        tmem_loaded16(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fix);
                        tmem_store16(tO + 16 * c, o);
                    }
                }
                settled = __all_sync(0xffffffffu, !real || fabsf(ref * cs) <= far_off);
                far = __any_sync(0xffffffffu, real && away());
            };
            // References that are far off are taken off the scores (trees).
            auto rebase = [&] {
                const float off = away() ? ref : 0.0f;
#pragma unroll
                for (int c = 0; c < kTile; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) - off);
            };
            // The tile's weights, and their sums.  References that are far off are taken off the scores on the way
            // (take_off), or were before.
            auto weigh = [&](auto take_off, bool taken_off) {
                constexpr bool kTake = decltype(take_off)::value != 0;
                const bool apart = (kTake || taken_off) && away();
                const float shift = ref == -INFINITY ? 0.0f : apart ? lift : lift - ref * cs;
                const uint32_t off = __float_as_uint(apart ? -ref : 0.0f);
                const uint64_t cs2 = pair(__float_as_uint(cs), __float_as_uint(cs)), off2 = pair(off, off);
                const uint64_t shift2 = pair(__float_as_uint(shift), __float_as_uint(shift));
                uint64_t part[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t y[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        uint64_t v = pair(x[32 * c + 2 * e], x[32 * c + 2 * e + 1]);
                        if (kTake) v = add2(v, off2);
                        const float2 z = unpair(fma2(v, cs2, shift2));
                        const float p0 = exp2_fast(z.x), p1 = exp2_fast(z.y);
                        part[e & 1] = add2(part[e & 1], pair(__float_as_uint(p0), __float_as_uint(p1)));
                        y[e] = pack2<BF16>(p0, p1);
                    }
                    tmem_store16(tP + 16 * c, y);
                    if (c == 1 && !L::kApart) {
                        // the first half's product starts while the second half is computed
                        tmem_store_wait();
                        tmem_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(base + L::oPHalf + 8 * s);
                    }
                }
                both = unpair(add2(part[0], part[1]));
            };
            // Hands tile j's weights over.
            auto give = [&](int j) -> bool {
                sum += both.x + both.y;
                if (!cached && (!PROMPT || n0 + kTile - 1 > first - (PROMPT ? s * S.tok : 0))) {
                    // Rows of V that were not finite: NaN for those who see them.
                    const int i = gi + (PROMPT ? j : 2 * j + s), vi = i % L::kV;
                    if (!warp_wait(base + L::oVReady + 8 * vi, (uint32_t)(i / L::kV & 1), stop)) return false;
                    const uint32_t odd[4] = {bad[4 * vi], bad[4 * vi + 1], bad[4 * vi + 2], bad[4 * vi + 3]};
                    if ((odd[0] | odd[1] | odd[2] | odd[3]) != 0) {
                        bool hit = false;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            uint32_t vis;
                            if (PROMPT) {
                                const int upto = token - n0 + 1 - 32 * u;
                                vis = upto >= 32 ? 0xffffffffu : upto > 0 ? (1u << upto) - 1u : 0u;
                            } else {
                                vis = u < 2 ? (uint32_t)(seen >> (32 * u)) : 0u;
                            }
                            hit |= (odd[u] & vis) != 0;
                        }
                        if (hit) sum = NAN;
                    }
                }
                tmem_store_wait();
                tmem_before();
                __syncwarp();
                if (lane == 0) bar_arrive(base + L::oPReady + 8 * s);
                return true;
            };
            int j = 0;
            // The segment's tiles; with prompts, up to one with a reference that is far off (true).
            auto tiles = [&]() -> bool {
                for (; j < mine; ++j) {
                    if (!(ok = fetch(j))) return false;
                    // Where the weights lie apart from the scores, the reference is not compared with every tile's
                    // maximum: the sum of the tile's weights shows when one has grown too large (over 2^15), and the tile
                    // is done again.  That spares the maximum's 64 instructions in nearly all tiles; a row's first tile
                    // always takes it, and so do tiles with references that are far off.
                    bool look = !L::kApart || !settled;
                    for (;;) {
                        if (look) {
                            follow(j);
                            if (far && PROMPT) return true;
                            if (far) rebase();
                        }
                        weigh(Count<0>{}, !PROMPT && far);
                        if (look || !__any_sync(0xffffffffu, real && both.x + both.y > 32768.0f)) break;
                        look = true;
                        tmem_store_wait();  // stores to the same columns follow: only this wait orders two of them
                    }
                    if (!(ok = give(j))) return false;
                }
                return false;
            };
            // With prompts, the rest of a segment with a reference that is far off goes through a loop of its own.  In the
            // loop above, the subtraction costs every call time even where it is not taken: 16 chunks with rows of 64 take
            // 296 us so, 284 with two loops, 283 without it; a prompt of 25,000 3,030, 2,975 and 2,980.
            // Trees are bound by memory and have it there: a second loop would not fit their registers (256 requests
            // 151 us, 110 so).
            if (tiles()) {
                for (;;) {
                    weigh(Count<1>{}, false);
                    if (!(ok = give(j)) || ++j == mine || !(ok = fetch(j))) break;
                    follow(j);
                }
            }
            if (!ok) break;
            if (mine > 0) {
                if (!(ok = warp_wait(base + L::oODone + 8 * s, od, stop))) break;
                od ^= 1;
                tmem_after();
            }
            // ---- The segment's result: to the output, or as a part. ----
            const bool whole = w.t0 == 0 && w.t1 == w.total;
            if (!whole && tid == 0) {
                // an item may fill the share: its cuts at both ends are one join
                const long long end = plan.g1 - w.left + w.took;
                cut[w.t0 > 0 ? 0 : 1] = Cut{w.x, w.b, w.h, w.item, w.total, end - w.t1 - kExtra<PROMPT>};
            }
            // the part that begins an item is the CTA's second, so that it never meets the one that ends an item
            const int slot = 2 * (int)blockIdx.x + (w.t0 > 0 ? 0 : 1);
            constexpr int rows = PROMPT ? 2 * kTile : kTile;
            const int64_t out_row = (PROMPT ? (int64_t)w.x.base : (int64_t)w.b * A.N) + token;
            char* const out = static_cast<char*>(A.out) + ((out_row * A.q_heads + w.h * A.group + g) * A.dim) * 2;
            float w0 = 1.0f, w1 = 0.0f, m = ref, l = sum;
            if (!PROMPT) {
                // both streams' statistics, to weigh their sums
                float2* const stat = reinterpret_cast<float2*>(sm + L::oStat);
                stat[s * kTile + row] = make_float2(ref, sum);
                tmem_before();
                __syncwarp();
                if (lane == 0) bar_arrive(base + L::oStatReady);
                if (!(ok = warp_wait(base + L::oStatReady, 0, stop))) break;
                tmem_after();
                const float2 a = stat[row], c = stat[kTile + row];
                m = fmaxf(a.x, c.x);
                w0 = a.x == -INFINITY ? 0.0f : exp2_fast((a.x - m) * cs);
                w1 = c.x == -INFINITY ? 0.0f : exp2_fast((c.x - m) * cs);
                l = a.y * w0 + c.y * w1;
                // a stream without a visible key has no sum of products (or one of zeros)
            }
            const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
            const int c0 = PROMPT ? 0 : s * (DP / 64), c1 = PROMPT ? DP / 32 : (s + 1) * (DP / 64);
            const uint32_t tA = PROMPT ? tO : lanes + 256, tB = lanes + 256 + DP;
            for (int c = c0; c < c1; ++c) {
                uint32_t o[32] = {}, o1[32] = {};
                if (PROMPT ? mine > 0 : true) tmem_load(tA + 32 * c, o);
                if (!PROMPT && len > 1) tmem_load(tB + 32 * c, o1);
                tmem_load_wait();
                tmem_loaded(o);
                tmem_loaded(o1);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float v = 0.0f;
                    if (PROMPT) {
                        if (mine > 0 && l != 0.0f) v = __uint_as_float(o[e]);
                    } else {
                        if (w0 != 0.0f) v = __uint_as_float(o[e]) * w0;
                        if (len > 1 && w1 != 0.0f) v = fmaf(__uint_as_float(o1[e]), w1, v);
                        if (l != l) v = l;
                    }
                    o[e] = __float_as_uint(v * inv);
                }
                if (real) {
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 16) {
                            if (32 * c + e < A.dim) {
                                uint32_t y[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    y[i] = pack2<BF16>(__uint_as_float(o[e + 2 * i]), __uint_as_float(o[e + 2 * i + 1]));
                                // a thread's row by whole sectors, where rows begin on one
                                if (S.wide_out) {
                                    store32(out + (32 * c + e) * 2, y);
                                } else {
                                    *reinterpret_cast<uint4*>(out + (32 * c + e) * 2) = make_uint4(y[0], y[1], y[2], y[3]);
                                    if (32 * c + e + 8 < A.dim)
                                        *reinterpret_cast<uint4*>(out + (32 * c + e + 8) * 2) = make_uint4(y[4], y[5], y[6], y[7]);
                                }
                            }
                        }
                    } else {
                        float4* const to = reinterpret_cast<float4*>(W.sums) + (int64_t)slot * (DP / 4) * rows +
                                           (PROMPT ? s * kTile : 0) + row;
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            to[(int64_t)(8 * c + e / 4) * rows] =
                                make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]), __uint_as_float(o[e + 2]),
                                            __uint_as_float(o[e + 3]));
                    }
                }
            }
            if (!whole && real && (PROMPT || s == 0))
                W.ml[(int64_t)slot * rows + (PROMPT ? s * kTile : 0) + row] = make_float2(m, l);
            // Neither stream's next sums may overwrite what the other still reads.
            tmem_before();
            if (!PROMPT) {
                __syncwarp();
                if (lane == 0) bar_arrive(base + L::oStatReady);
                if (!(ok = warp_wait(base + L::oStatReady, 1, stop))) break;
            }
            gi += len;
            __syncwarp();
            if (lane == 0) w.next(A, S, plan, near);
            __syncwarp();
        }
    } else {
        Walk<PROMPT> w;
        w.start(A, S, plan, near);
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == kCopyWarp || warp == kCopyWarp2) {
            // ---- Copies: two warps (a copy costs its warp about 65 cycles, and pages of 16 rows need 16 a tile). ----
            // With trees one brings K and the other V, so that small pages' copies go side by side (256 short requests,
            // pages of 16: 119 us, by alternate tiles 155); with prompts they take alternate tiles, which keeps K and
            // V in step (a 25,000-token prompt: 3.16 ms, by K and V 3.26).  The first also brings Q.
            const int odd = warp == kCopyWarp ? 0 : 1;
            const bool brings_k = PROMPT || odd == 0, brings_v = PROMPT || odd == 1;
            auto my = [&](int tile) { return !PROMPT || (tile & 1) == odd; };
            int i = 0, seg = 0, nk = 0, nv = 0, nq = 0;  // n*: one past the last tile or item asked for
            bool ok = (base & 1023) == 0;  // the swizzle's period
            if (!ok) *stop = 1;
            const int pages = kTile >> A.C.shift;  // of a tile
            for (; ok && w.left > 0; w.next(A, S, plan, near), ++seg) {
                const int32_t* const table = w.x.slot >= 0 ? A.C.table + (int64_t)w.x.slot * A.C.max_pages : nullptr;
                // Page numbers come 32 at a time, a batch ahead of the one in use: a tile's pages lie in one batch.
                auto batch = [&](int first) {
                    const int64_t p = (int64_t)first + lane;
                    if ((p << A.C.shift) >= w.x.ctx) return -1;
                    int32_t page = table[p];
                    if (page < 0 || page >= A.C.num_pages) {
                        latch(A.C.status, CLK_EINVAL, w.x.slot);
                        page = A.C.num_pages;  // reads as zeros
                    }
                    return page;
                };
                int at = w.t0 * pages & ~31, now = batch(at), then = batch(at + 32);
                const int z = PROMPT ? 0 : w.b, row0 = PROMPT ? w.x.base : 0;
                // the first K goes out before the first V
                if (!PROMPT && odd == 1 && seg == 0 && !(ok = warp_wait(base + L::oQFull, 0, stop))) break;
                if (odd == 0) {
                    const int qi = seg % L::kQB;
                    const uint32_t qb = base + L::oQFull + 8 * qi;
                    if (!(ok = warp_wait(base + L::oQEmpty + 8 * qi, (uint32_t)(seg / L::kQB & 1) ^ 1, stop))) break;
                    ++nq;
                    if (lane == 0) bar_expect(qb, (uint32_t)(L::kQ * L::kHalves) * (uint32_t)(S.qbox * A.group) * 128u);
                    __syncwarp();
                    if (lane < L::kQ * L::kHalves) {
                        const int s = lane / L::kHalves, hf = lane % L::kHalves;
                        copy_box(qs + (qi * L::kQ + s) * L::kBytes + hf * L::kHalf, &M.q, 64 * hf, w.h * A.group,
                                 row0 + w.item * S.block + s * S.tok, z, qb);
                    }
                }
                for (int t = w.t0; t < w.t1; ++t, ++i) {
                    const bool cached = t < w.x.ctx_tiles;
                    if (cached && t * pages - at >= 32) {
                        at += 32;
                        now = then;
                        then = batch(at + 32);
                    }
                    if (!my(i)) continue;
                    int page = __shfl_sync(0xffffffffu, now, (t * pages - at + lane) & 31);
                    if (!cached || lane >= pages) page = -1;
                    const int boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));
                    const uint32_t bytes = (uint32_t)L::kHalves * 128u * (uint32_t)(cached ? boxes << A.C.shift : S.kbox);
                    const int n0 = row0 + (t - w.x.ctx_tiles) * kTile;
                    auto bring = [&](uint32_t bar, uint32_t dst, const CUtensorMap* pool, const CUtensorMap* fresh) {
                        if (lane == 0) bar_expect(bar, bytes);
                        __syncwarp();
                        if (page >= 0) {
#pragma unroll
                            for (int hf = 0; hf < L::kHalves; ++hf)
                                copy_box(dst + hf * L::kHalf + (lane << A.C.shift) * 128, pool, 64 * hf, 0, w.h, page, bar);
                        } else if (!cached && lane < L::kHalves) {
                            copy_box(dst + lane * L::kHalf, fresh, 64 * lane, w.h, n0, z, bar);
                        }
                    };
                    const int ki = i % L::kK, vi = i % L::kV;
                    if (brings_k) {
                        if (!(ok = warp_wait(base + L::oKEmpty + 8 * ki, (uint32_t)(i / L::kK & 1) ^ 1, stop))) break;
                        nk = i + 1;
                        bring(base + L::oKFull + 8 * ki, ks + ki * L::kBytes, &M.kc, &M.k);
                    }
                    if (brings_v) {
                        if (!(ok = warp_wait(base + L::oVEmpty + 8 * vi, (uint32_t)(i / L::kV & 1) ^ 1, stop))) break;
                        nv = i + 1;
                        bring(base + L::oVFull + 8 * vi, vs + vi * L::kBytes, &M.vc, &M.v);
                    }
                }
            }
            if (!ok) {
                // Leave no copy in flight.
                const long long t0 = clock64();
                auto drain = [&](uint32_t bar, uint32_t parity) {
                    while (!bar_try(bar, parity) && clock64() - t0 < kWaitClocks) {}
                };
                for (int j = nq > L::kQB ? nq - L::kQB : 0; j < nq; ++j) drain(base + L::oQFull + 8 * (j % L::kQB), (uint32_t)(j / L::kQB & 1));
                for (int j = nk > L::kK ? nk - L::kK : 0; j < nk; ++j)
                    if (my(j)) drain(base + L::oKFull + 8 * (j % L::kK), (uint32_t)(j / L::kK & 1));
                for (int j = nv > L::kV ? nv - L::kV : 0; j < nv; ++j)
                    if (my(j)) drain(base + L::oVFull + 8 * (j % L::kV), (uint32_t)(j / L::kV & 1));
            }
        } else if (warp == kMmaWarp) {
            // ---- Products: one lane issues them, the warp goes along. ----
            {
                // Shuffled values are the same in every lane for the compiler too.
                auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
                const uint32_t tm = (uint32_t)same((int)tmem);
                constexpr uint32_t types = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((kTile >> 4) << 24);
                constexpr uint32_t kind_s = types | ((kTile >> 3) << 17);
                constexpr uint32_t kind_o = types | (1u << 16) | ((DP >> 3) << 17);  // V's rows run along the output
                uint32_t ps[2] = {0, 0}, fs[2] = {1, 1};  // phases of PReady and SFree
                int seg = 0, qi = 0;
                uint32_t qp = 0;
                bool ok = true;
                // This warp's instructions bound the rate at which short products follow one another: ring places
                // and phases are counted along, and a tile is waited for once for both streams.
                int ki = 0, vi = 0;
                uint32_t kp = 0, vp = 0;
                auto step = [](int& i, uint32_t& phase, int n) {
                    if (++i == n) {
                        i = 0;
                        phase ^= 1;
                    }
                };
                auto done = [](uint32_t bar) {
                    if (elect()) mma_commit(bar);
                    __syncwarp();
                };
                // descriptors count in 16 bytes
                const uint64_t q0 = operand(qs, 16), k0 = operand(ks, 16), v0 = operand(vs, L::kHalf);
                auto wait_k = [&] { return warp_wait(base + L::oKFull + 8 * ki, kp, stop); };
                auto wait_v = [&] { return warp_wait(base + L::oVReady + 8 * vi, vp, stop); };
                // Stream s's scores with K tile ki.
                auto scores = [&](int s) {
                    if (L::kApart) {
                        if (!warp_wait(base + L::oSFree + 8 * s, fs[s], stop)) return false;
                        fs[s] ^= 1;
                    }
                    tmem_after();
                    const uint64_t q = q0 + (qi * L::kQ + (PROMPT ? s : 0)) * (L::kBytes / 16), k = k0 + ki * (L::kBytes / 16);
                    if (elect()) {
#pragma unroll
                        for (int e = 0; e < DP / 16; ++e) {
                            constexpr int next = L::kHalf / 16;
                            const int at = (e / 4) * next + (e % 4) * 2;
                            mma_ss(tm + 128 * s, q + at, k + at, kind_s, e > 0);
                        }
                        mma_commit(base + L::oSFull + 8 * s);
                    }
                    __syncwarp();
                    return true;
                };
                // Stream s's weights with V tile vi.  Where the weights lie over the scores, the chain of one stream
                // is what counts, and their first half's product does not wait for the second.
                auto values = [&](int s, bool add) {
                    const uint64_t v = v0 + vi * (L::kBytes / 16);
                    constexpr int steps = L::kApart ? 8 : 4;  // 16 keys each
#pragma unroll
                    for (int part = 0; part < 8; part += steps) {
                        if (!warp_wait(base + (part + steps < 8 ? L::oPHalf : L::oPReady) + 8 * s, ps[s], stop)) return false;
                        tmem_after();
                        if (elect()) {
#pragma unroll
                            for (int e = part; e < part + steps; ++e)
                                mma_ts(tm + 256 + s * DP, tm + (L::kApart ? 384 + 64 * s : 128 * s) + 8 * e, v + 128 * e, kind_o,
                                       add || e > 0);
                        }
                        __syncwarp();
                    }
                    ps[s] ^= 1;
                    return true;
                };
                for (; ok; w.next(A, S, plan, near), ++seg) {
                    const int len = same(w.left > 0 ? w.t1 - w.t0 : 0);
                    if (len == 0) break;
                    if (!(ok = warp_wait(base + L::oQFull + 8 * qi, qp, stop))) break;
                    if (PROMPT) {
                        const int n[2] = {same(w.last(S, 0) - w.t0), same(w.last(S, 1) - w.t0)};
                        if (!(ok = wait_k())) break;
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            if (ok && n[s] > 0) ok = scores(s);
                        if (!ok) break;
                        done(base + L::oKEmpty + 8 * ki);
                        step(ki, kp, L::kK);
                        if (len == 1) done(base + L::oQEmpty + 8 * qi);
                        for (int j = 0; j < len; ++j) {
                            const bool more = j + 1 < len;
                            if (L::kApart && more && !(ok = wait_k())) break;
                            if (!(ok = wait_v())) break;
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                if (!ok) continue;
                                if (L::kApart && j + 1 < n[s]) ok = scores(s);
                                if (ok && j < n[s]) {
                                    ok = values(s, j > 0);
                                    if (ok && (L::kApart || j + 1 == n[s])) done(base + L::oODone + 8 * s);
                                }
                                if (!L::kApart && ok && more) {
                                    if (s == 0) ok = wait_k();
                                    if (ok && j + 1 < n[s]) ok = scores(s);
                                }
                            }
                            if (!ok) break;
                            done(base + L::oVEmpty + 8 * vi);
                            step(vi, vp, L::kV);
                            if (more) {
                                done(base + L::oKEmpty + 8 * ki);
                                step(ki, kp, L::kK);
                            }
                            if (j + 2 == len) done(base + L::oQEmpty + 8 * qi);
                        }
                    } else {
                        auto ahead = [&](int j) {
                            if (j >= len) return true;
                            if (!wait_k() || !scores(j & 1)) return false;
                            done(base + L::oKEmpty + 8 * ki);
                            step(ki, kp, L::kK);
                            if (j + 1 == len) done(base + L::oQEmpty + 8 * qi);
                            return true;
                        };
                        ok = ahead(0) && ahead(1);
                        for (int j = 0; ok && j < len; ++j) {
                            const int s = j & 1;
                            if (L::kApart && !(ok = ahead(j + 2))) break;
                            if (!(ok = wait_v() && values(s, j >= 2))) break;
                            if (L::kApart || j + 2 >= len) done(base + L::oODone + 8 * s);
                            done(base + L::oVEmpty + 8 * vi);
                            step(vi, vp, L::kV);
                            if (!L::kApart) ok = ahead(j + 2);
                        }
                    }
                    step(qi, qp, L::kQB);
                }
                if (!ok) {
                    // Products in flight end before tensor memory is given up.
                    done(base + L::oDrain);
                    const long long t0 = clock64();
                    while (!bar_try(base + L::oDrain, 0) && clock64() - t0 < kWaitClocks) {}
                }
            }
            __syncwarp();
        } else {
            // ---- V tiles: rows past the end, and rows that are not finite. ----
            // a value is not finite where its exponent is all ones: one more there carries into the sign
            constexpr uint32_t expo = BF16 ? 0x7f807f80u : 0x7c007c00u, one = BF16 ? 0x00800080u : 0x04000400u;
            if (!PROMPT) {
                // Rows past the node counts are 0; the requests are dealt out to the CTAs.
                for (int b = blockIdx.x; b < A.B; b += gridDim.x) {
                    const int rows = attend_request(A, b, false).rows;
                    const int64_t row = (int64_t)A.q_heads * A.dim / 8;
                    uint4* const out = static_cast<uint4*>(A.out) + ((int64_t)b * A.N + rows) * row;
                    for (int64_t e = lane; e < (A.N - rows) * row; e += 32) out[e] = make_uint4(0, 0, 0, 0);
                }
            }
            int i = 0;
            bool ok = true;
            for (; ok && w.left > 0; w.next(A, S, plan, near)) {
                for (int t = w.t0; t < w.t1; ++t, ++i) {
                    const int vi = i % L::kV;
                    if (!(ok = warp_wait(base + L::oVFull + 8 * vi, (uint32_t)(i / L::kV & 1), stop))) break;
                    const bool cached = t < w.x.ctx_tiles;
                    const int n0 = (t - w.x.ctx_tiles) * kTile;
                    const int have = cached ? w.x.ctx - t * kTile : w.x.rows - n0;
                    const bool look = !cached && (!PROMPT || n0 + kTile - 1 > w.item * S.block);
                    if (have < kTile || look) {
                        char* const tile = sm + (vs - base) + vi * L::kBytes;
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int r = 32 * u + lane;
                            bool clear = r >= have, odd = false;
                            if (look && 32 * u < have) {
                                uint32_t hit = 0;
#pragma unroll
                                for (int c = 0; c < 8 * L::kHalves; ++c) {
                                    // lanes start at different chunks of their rows: no two in one bank
                                    const int at = (c & 8) * (L::kHalf / 8) + r * 128 + (((c & 7) + lane) & 7) * 16;
                                    const uint4 x = *reinterpret_cast<const uint4*>(tile + at);
                                    hit |= ((x.x & expo) + one) | ((x.y & expo) + one) | ((x.z & expo) + one) | ((x.w & expo) + one);
                                }
                                odd = !clear && (hit & 0x80008000u) != 0;
                            }
                            if (clear || odd)
#pragma unroll
                                for (int c = 0; c < 8 * L::kHalves; ++c) {
                                    const int at = (c & 8) * (L::kHalf / 8) + r * 128 + (((c & 7) + lane) & 7) * 16;
                                    *reinterpret_cast<uint4*>(tile + at) = make_uint4(0, 0, 0, 0);
                                }
                            const uint32_t word = __ballot_sync(0xffffffffu, odd);
                            if (lane == 0) bad[4 * vi + u] = word;
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    __syncwarp();
                    if (lane == 0) bar_arrive(base + L::oVReady + 8 * vi);
                }
            }
        }
    }

    // ---- Parts are written: raise the flag, join what was cut. ----
    tmem_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
    if (tid == 0) {
        // after the barrier above, the release covers the whole CTA's parts
        asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(W.flag + blockIdx.x), "r"(plan.call + 1) : "memory");
        if (*stop != 0) gave_up(A, W);
    }
    if (*stop != 0 || plan.g0 >= plan.g1) return;
    const Cuts cuts(plan.all, plan.ctas);
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
        if (cut[i].total > 0) join_item<DP, BF16, PROMPT>(A, S, W, plan, cuts, cut[i], stop);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encoder()
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
// elements), copied in boxes of 64 x b1 x b2 (x 1).
bool encode(EncodeFn f, CUtensorMap* m, int32_t dtype, const void* base, int64_t dim, const int64_t n[3], const int64_t st[3],
            int b1, int b2)
{
    const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)n[0], (cuuint64_t)n[1], (cuuint64_t)n[2]};
    cuuint64_t strides[3];
    // the stride of an axis of one is not used; it still has to be a valid one
    for (int i = 0; i < 3; ++i) strides[i] = n[i] > 1 ? (cuuint64_t)st[i] * 2 : 256;
    const cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1}, one[4] = {1, 1, 1, 1};
    return f(m, dtype == CLK_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A stride (in elements of 2 bytes) that a tensor map can take, for an axis of n.
bool map_stride(int64_t st, int64_t n) { return n <= 1 || (st > 0 && st % 8 == 0 && st < ((int64_t)1 << 38)); }

template <int DP, bool BF16, bool PROMPT>
int launch_mma(const Attend& A, const Shape& S, const Maps& M, void* scratch, cudaStream_t s)
{
    using L = Lay<DP, PROMPT>;
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CLK_ECUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit) || dev > 63) {
        if (cudaFuncSetAttribute(k_attend<DP, BF16, PROMPT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal) != cudaSuccess)
            return CLK_ECUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = L::kTotal;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the joins wait on one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, k_attend<DP, BF16, PROMPT>, M, A, S, scratch));
}

bool mma_dim(int32_t dim) { return dim >= 8 && dim <= 128 && dim % 8 == 0; }

}  // namespace

// Rows of up to 128 elements of 16 bits in whole 16-byte vectors (the copies
// fill them up to 64 or 128 with zeros: 8 requests of 16 nodes over 2,000 rows
// of 40, 32/8 heads, take 20 us, 136 in the general kernel), groups of at most a row tile,
// and strides that tensor maps can take.  A scale that is not positive would
// turn the running maximum around, and one at the end of the range would
// leave it; both are left to the general kernel.
bool attend_mma_takes(const Attend& A)
{
    if (A.dtype == CLK_DTYPE_F32 || !mma_dim(A.dim) || A.group > kTile || !(A.scale >= 1e-20f && A.scale <= 1e20f))
        return false;
    for (const void* p : {A.q, A.k, A.v, (const void*)A.out, A.kc, A.vc})
        if (!aligned(p, 16)) return false;
    const int64_t rows = A.off != nullptr ? A.T : A.N, reqs = A.off != nullptr ? 1 : A.B;
    if (!map_stride(A.q_req, reqs) || !map_stride(A.q_row, rows) || !map_stride(A.q_head, A.q_heads)) return false;
    if (!map_stride(A.k_req, reqs) || !map_stride(A.k_row, rows) || !map_stride(A.k_head, A.kv_heads)) return false;
    if (!map_stride(A.v_req, reqs) || !map_stride(A.v_row, rows) || !map_stride(A.v_head, A.kv_heads)) return false;
    if (A.kc != nullptr && (!map_stride(A.page_stride, A.C.num_pages) || !map_stride(A.head_stride, A.kv_heads) ||
                            !map_stride(A.tok_stride, 2)))
        return false;
    return true;
}

size_t attend_mma_scratch(int32_t q_heads, int32_t kv_heads, int32_t dim)
{
    if (!mma_dim(dim) || q_heads / kv_heads > kTile) return 0;
    const size_t rows = 2 * kTile;
    const int n = num_sms();
    return kStatusBytes + flag_bytes(n) + (size_t)n * 2 * rows * (sizeof(float2) + (size_t)pad_dim(dim) * sizeof(float));
}

int attend_mma_launch(const Attend& A, void* scratch, cudaStream_t s)
{
    const bool prompt = A.off != nullptr;
    const EncodeFn f = encoder();
    if (f == nullptr) return CLK_ECUDA;
    Shape S;
    S.tok = kTile / A.group;
    S.block = prompt ? 2 * S.tok : S.tok;
    const int64_t rows = prompt ? A.T : A.N, reqs = prompt ? 1 : A.B;
    S.qbox = (int32_t)(S.tok < rows ? S.tok : rows);
    S.kbox = (int32_t)(kTile < rows ? kTile : rows);
    S.ctas = num_sms();
    S.wide_out = A.dim % 16 == 0 && aligned(A.out, 32);
    S.log2_scale = (float)((double)A.scale * 1.4426950408889634);
    if (S.ctas < 1) return CLK_ECUDA;
    Maps M;
    const int64_t nq[3] = {A.q_heads, rows, reqs}, nk[3] = {A.kv_heads, rows, reqs};
    const int64_t sq[3] = {A.q_head, A.q_row, A.q_req}, sk[3] = {A.k_head, A.k_row, A.k_req}, sv[3] = {A.v_head, A.v_row, A.v_req};
    bool ok = encode(f, &M.q, A.dtype, A.q, A.dim, nq, sq, A.group, S.qbox) &&
              encode(f, &M.k, A.dtype, A.k, A.dim, nk, sk, 1, S.kbox) && encode(f, &M.v, A.dtype, A.v, A.dim, nk, sv, 1, S.kbox);
    if (A.kc != nullptr) {
        const int64_t np[3] = {A.C.page_tokens(), A.kv_heads, A.C.num_pages};
        const int64_t sp[3] = {A.tok_stride, A.head_stride, A.page_stride};
        ok = ok && encode(f, &M.kc, A.dtype, A.kc, A.dim, np, sp, A.C.page_tokens(), 1) &&
             encode(f, &M.vc, A.dtype, A.vc, A.dim, np, sp, A.C.page_tokens(), 1);
    } else {
        M.kc = M.vc = M.k;  // not read: no request has cached rows
    }
    if (!ok) return CLK_EINVAL;
    const bool wide = A.dim > 64, bf = A.dtype == CLK_DTYPE_BF16;
#define CLK_GO(D, T, P) return launch_mma<D, T, P>(A, S, M, scratch, s)
    if (prompt) {
        if (wide) {
            if (bf) CLK_GO(128, true, true);
            CLK_GO(128, false, true);
        }
        if (bf) CLK_GO(64, true, true);
        CLK_GO(64, false, true);
    }
    if (wide) {
        if (bf) CLK_GO(128, true, false);
        CLK_GO(128, false, false);
    }
    if (bf) CLK_GO(64, true, false);
    CLK_GO(64, false, false);
#undef CLK_GO
}

}  // namespace clk
