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
//
// Prompts over a cache in 8 bits (E8).  Four warps more bring its tiles to 16
// bits, times their scales: a thread takes 16 codes, a warp a half or quarter of
// a tile's rows; new tokens' tiles are brought as they are.  Every pair of row
// tiles converts the tiles again: 3,800 of a step's 9,400 instructions, beside
// 4,800 of the softmax, which together do not stay in the instruction cache (84%
// of the fetches hit).  So a step takes 4,700 cycles: 4,000 tokens behind 25,000
// (32/8 heads of 128) 1,694 us, 1,045 TFLOP/s, where 16 bits reach 1,700; 8
// prompts of 100 to 1,500 behind up to 8,192 (24/4 heads of 64) 330 to 357 us, 600
// to 650 TFLOP/s, where they reach 1,020.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "clk.h"
#include "clk_attend.h"
#include "clk_attend_work.cuh"
#include "clk_cache.h"
#include "clk_eight.cuh"
#include "clk_host.h"
#include "clk_mma.cuh"

namespace clk {
namespace {

// 8 softmax, 2 copies, 1 products, 1 V tiles; with a cache in 8 bits (E8: prompts; trees over one have a kernel of
// their own) 4 that convert its tiles
template <bool E8>
constexpr int kWarps = E8 ? 16 : 12;
template <bool E8>
constexpr int kThreads = 32 * kWarps<E8>;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kCopyWarp2 = 10, kValueWarp = 11, kConvertWarp = 12;

template <int DP, bool PROMPT, bool E8>
struct Lay {
    using K = typename std::conditional<PROMPT, Prompts, Trees>::type;
    static constexpr int kHalves = DP / 64;
    static constexpr int kHalf = kTile * 128;  // bytes of 64 columns of a tile
    static constexpr int kBytes = kHalves * kHalf;
    // Rows of 64 leave room in tensor memory for weights beside the scores (two streams of 128 + 64 + 64
    // columns), so that the next scores are computed while this tile's are exponentiated; with rows of 128
    // the weights lie over the scores.
    static constexpr bool kApart = DP == 64;
    static constexpr int kPart = kTile * DP;                       // bytes of a tile of 8 bits
    static constexpr int kQ = PROMPT ? 2 : 1;                      // row tiles of an item
    static constexpr int kQB = DP == 128 && PROMPT ? 1 : 2;        // items whose Q is held
    // K tiles in the ring
    static constexpr int kK = E8 ? (DP == 128 ? 2 : 3) : DP == 128 ? (PROMPT ? 3 : 2) : (PROMPT ? 5 : 4);
    // V tiles in the ring; with a cache in 8 bits halves of 64 keys, an even number: each half has places of its own
    static constexpr int kV = E8 ? (DP == 128 ? 4 : 6) : DP == 128 ? 2 : (PROMPT ? 5 : 4);
    static constexpr int kVBytes = E8 ? kBytes / 2 : kBytes;
    // tiles as the cache holds them, to be converted
    static constexpr int kG = !E8 ? 0 : DP == 128 ? 2 : 6;
    static_assert(!E8 || kV % 2 == 0, "places of halves");
    static constexpr int kGs = kG > 0 ? kG : 1;
    static constexpr int oK = kQ * kQB * kBytes, oV = oK + kK * kBytes, oG = oV + kV * kVBytes;
    // after the tiles
    static constexpr int oKFull = oG + kG * kPart, oKEmpty = oKFull + 8 * kK;
    static constexpr int oVFull = oKEmpty + 8 * kK, oVReady = oVFull + 8 * kV, oVEmpty = oVReady + 8 * kV;
    static constexpr int oGFull = oVEmpty + 8 * kV, oGEmpty = oGFull + 8 * kG;
    static constexpr int oQFull = oGEmpty + 8 * kG, oQEmpty = oQFull + 8 * kQB;
    static constexpr int oSFull = oQEmpty + 8 * kQB, oSFree = oSFull + 16, oPReady = oSFree + 16, oPHalf = oPReady + 16, oODone = oPHalf + 16;
    static constexpr int oStatReady = oODone + 16, oRaised = oStatReady + 8, oRaisedRead = oRaised + (E8 ? 16 : 0);
    static constexpr int oDrain = oRaisedRead + (E8 ? 16 : 0);
    static constexpr int oBars = oDrain + 8;  // end of the barriers
    static constexpr int oBad = (oBars + 15) / 16 * 16;               // uint32[kV][4]
    static constexpr int oScale = oBad + 16 * kV;                     // float[kG][8]: of blocks of 16 keys
    static constexpr int oRaise = oScale + 32 * kG;                   // uint32[2]: of segments (see kRaised)
    static constexpr int oNear = oRaise + (E8 ? 16 : 0);              // Reach[kNear]
    static constexpr int oPlan = oNear + kNear * (int)sizeof(Reach);  // Plan, stop flag, tmem address
    static constexpr int oCut = oPlan + (int)sizeof(Plan);            // Cut[2]: of items that end here, that begin here
    static constexpr int oWalk = (oCut + 2 * (int)sizeof(Cut) + 7) / 8 * 8;  // Walk[8]
    static constexpr int oStop = oWalk + (E8 ? 12 : 8) * (int)sizeof(Walk<K>), oTmem = oStop + 4;
    static constexpr int oStat = (oTmem + 4 + 15) / 16 * 16;          // float2[2][128] for trees
    static constexpr int kTotal = oStat + (PROMPT ? 0 : 2 * kTile * 8);
    static_assert(kTotal <= 232448, "shared memory");
};

template <int DP, bool BF16, bool PROMPT, bool E8>
__global__ void __launch_bounds__(kThreads<E8>, 1) k_attend(const __grid_constant__ Maps M, const __grid_constant__ Attend A,
                                                            const __grid_constant__ Shape S, void* scratch)
{
    static_assert(PROMPT || !E8, "trees over a cache in 8 bits have a kernel of their own");
    using L = Lay<DP, PROMPT, E8>;
    using K = typename L::K;
    constexpr int kThreads = clk::kThreads<E8>;
    // A cache in 8 bits may hold more than float16's largest.  Where a segment's scales reach beyond 2^7 (448 times that is
    // in range), its cached K and V are converted divided by a power of two each, the least that is enough; scores are
    // multiplied by K's, O counts in V's.  One warp looks through the scales ahead of the others, so that a tile of other
    // segments costs nothing.  (8 prompts of 100 to 1,500 tokens behind up to 8,192, 24/4 heads of 64, 356 us without and
    // with it, 406 with a look at every tile in the loops below; 4,000 behind 25,000, 32/8 heads of 128, 1,317, 1,322, 1,436.)
    constexpr bool kRaised = E8 && !BF16;
    auto power = [](uint32_t e) { return __uint_as_float(127 + e << 23); };
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
            bar_init(base + L::oKFull + 8 * i, E8 ? 4 : 1);
            bar_init(base + L::oKEmpty + 8 * i, 1);
        }
        for (int i = 0; i < L::kV; ++i) {
            bar_init(base + L::oVFull + 8 * i, 1);
            bar_init(base + L::oVReady + 8 * i, E8 ? 2 : 1);
            bar_init(base + L::oVEmpty + 8 * i, 1);
        }
        for (int i = 0; i < L::kG; ++i) {
            bar_init(base + L::oGFull + 8 * i, 1 + 32);  // the copies of a tile, and of its scales by a warp's lanes
            bar_init(base + L::oGEmpty + 8 * i, 4);
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
        for (int i = 0; kRaised && i < 2; ++i) {
            bar_init(base + L::oRaised + 8 * i, 1);
            bar_init(base + L::oRaisedRead + 8 * i, 8 + 4);  // the softmax warps', and those that convert
        }
        bar_init(base + L::oDrain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    // (the rings are not in use yet)
    make_plan<K, kThreads>(A, S, reinterpret_cast<long long*>(sm), plan, near, cut, stop, call, began, E8 ? __shfl_sync(0xffffffffu, tid >> 5, 0) : warp);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the planning scratch lies where tiles go
    tmem_before();
    __syncthreads();
    tmem_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::oTmem);
    const uint32_t qs = base, ks = base + L::oK, vs = base + L::oV;

    // Registers: 384 threads x 168 at launch; 256 x 208 + 128 x 80 after the split.  512 x 128; 256 x 200 + 256 x 56.
    if (warp < kCopyWarp) {
        if (E8)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        else
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
        int gi = 0, seg = 0;
        bool ok = true;
        Walk<K>& w = reinterpret_cast<Walk<K>*>(sm + L::oWalk)[warp];
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
            const uint32_t* const raise = reinterpret_cast<const uint32_t*>(sm + L::oRaise) + (seg & 1);
            if (kRaised && !(ok = warp_wait(base + L::oRaised + 8 * (seg & 1), (uint32_t)(seg >> 1 & 1), stop))) break;
            float ref = -INFINITY, sum = 0.0f;
            bool settled = false;  // every row has a reference, and none is far off
            bool far = false;      // some row's is far off
            uint32_t x[kTile];     // a tile's scores
            float2 both;           // sums of its weights
            int t = 0, n0 = 0;
            bool cached = false;
            auto away = [&] { return ref != -INFINITY && fabsf(ref * cs) > far_off; };
            // Rows of V that were not finite: NaN for those who see them.  (A half of a tile has a place of its own where the
            // cache is in 8 bits, and is gone once the first half's weights are given: there this comes before.)
            auto look_at = [&](int j) -> bool {
                if (!cached && (!PROMPT || n0 + kTile - 1 > first - (PROMPT ? s * S.tok : 0))) {
                    const int i = gi + (PROMPT ? j : 2 * j + s), at = E8 ? 2 * i : i, vi = at % L::kV;
                    if (!warp_wait(base + L::oVReady + 8 * vi, (uint32_t)(at / L::kV & 1), stop)) return false;
                    const int vj = E8 ? (at + 1) % L::kV : vi;
                    if (E8 && !warp_wait(base + L::oVReady + 8 * vj, (uint32_t)((at + 1) / L::kV & 1), stop)) return false;
                    const uint32_t odd[4] = {bad[4 * vi], bad[4 * vi + 1], bad[4 * vj + (E8 ? 0 : 2)], bad[4 * vj + (E8 ? 1 : 3)]};
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
                return true;
            };
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
                if (E8 && !look_at(j)) return false;
                return true;
            };
            // A divided tile's scores times K's power of two; O, which counts in V's up to the cache's end (and is complete, as
            // in follow), times V's before new tokens.
            auto adjust = [&](int j) {
                const uint32_t over = *raise;
                if (cached) {
                    const float up = power(over & 255);
#pragma unroll
                    for (int c = 0; c < kTile; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * up);
                } else if (t == ctx_tiles && j > 0 && over >> 8 != 0) {
                    const float up = power(over >> 8);
#pragma unroll 1
                    for (int c = 0; c < DP; c += 16) {
                        uint32_t o[16];
                        tmem_load16(tO + c, o);
                        tmem_load_wait();
                        tmem_loaded16(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * up);
                        tmem_store16(tO + c, o);
                    }
                    tmem_store_wait();
                }
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
                if (!E8 && !look_at(j)) return false;
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
            // That loop is also taken by segments whose K or V were divided, from their first tile on.
            if (kRaised) {
                const bool raised = *raise != 0 && mine > 0;
                if (raised || tiles()) {
                    for (bool held = !raised;; held = false) {
                        if (!held && !(ok = fetch(j))) break;
                        adjust(j);
                        follow(j);
                        weigh(Count<1>{}, false);
                        if (!(ok = give(j)) || ++j == mine) break;
                    }
                }
            } else if (tiles()) {
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
                cut[w.t0 > 0 ? 0 : 1] = Cut{w.x, w.b, w.h, w.item, w.total, end - w.t1 - K::extra};
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
            // a part that ends in the cache counts in V's power of two
            const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : kRaised && t0 + mine <= ctx_tiles ? power(*raise >> 8) : 1.0f;
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
            if (lane == 0) {
                if (kRaised) bar_arrive(base + L::oRaisedRead + 8 * (seg & 1));
                w.next(A, S, plan, near);
            }
            ++seg;
            __syncwarp();
        }
    } else {
        // (the converting warps keep their way through the share in shared memory too)
        Walk<K> w;
        if (!E8 || warp < kConvertWarp) w.start(A, S, plan, near);
        if (!E8)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (E8 && warp == kCopyWarp2) {
            // ---- Scales beyond 2^7, segment by segment (this warp has nothing to copy). ----
            for (int seg = 0; kRaised && w.left > 0; w.next(A, S, plan, near), ++seg) {
                // A lane has one of eight blocks of 16 keys of every other tile, of K or of V.
                const int key = 16 * (lane & 7), tiles = (w.t1 < w.x.ctx_tiles ? w.t1 : w.x.ctx_tiles) - w.t0;
                const float* const plane = (lane & 8 ? A.vs : A.ks) + w.h * A.scale_head + ((key & (A.C.page_tokens() - 1)) >> A.scale_shift) * A.scale_block;
                const int32_t* const table = A.C.table + (int64_t)w.x.slot * A.C.max_pages;
                uint32_t top = 0;  // as an integer: positive floats are in order
                for (int u = lane >> 4; u < tiles; u += 16) {
                    int32_t page[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int64_t at = (int64_t)(w.t0 + u + 2 * e) * kTile + key;
                        page[e] = u + 2 * e < tiles && at < w.x.ctx ? table[at >> A.C.shift] : -1;
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (page[e] >= 0 && page[e] < A.C.num_pages) {
                            const uint32_t bits = __float_as_uint(plane[page[e] * A.scale_page]) & 0x7fffffffu;
                            if (bits < 0x7f800000u && bits > top) top = bits;
                        }
                }
                const int e = (int)(top + 0x7fffffu >> 23) - (127 + 7);
                const uint32_t over = e > 0 ? (uint32_t)e : 0u;
                const uint32_t both = __reduce_max_sync(0xffffffffu, lane & 8 ? 0u : over) | __reduce_max_sync(0xffffffffu, lane & 8 ? over : 0u) << 8;
                if (!warp_wait(base + L::oRaisedRead + 8 * (seg & 1), (uint32_t)(seg >> 1 & 1) ^ 1, stop)) break;
                if (lane == 0) {
                    reinterpret_cast<uint32_t*>(sm + L::oRaise)[seg & 1] = both;
                    bar_arrive(base + L::oRaised + 8 * (seg & 1));
                }
                __syncwarp();
            }
        } else if (warp == kCopyWarp || warp == kCopyWarp2) {
            // ---- Copies: two warps (a copy costs its warp about 65 cycles, and pages of 16 rows need 16 a tile). ----
            // With trees one brings K and the other V, so that small pages' copies go side by side (256 short requests,
            // pages of 16: 119 us, by alternate tiles 155); with prompts they take alternate tiles, which keeps K and
            // V in step (a 25,000-token prompt: 3.16 ms, by K and V 3.26).  The first also brings Q.
            // With a cache in 8 bits one warp copies all that is not converted.
            const int odd = warp == kCopyWarp ? 0 : 1;
            const bool brings_k = PROMPT || odd == 0, brings_v = PROMPT || odd == 1;
            auto my = [&](int tile) { return !PROMPT || E8 || (tile & 1) == odd; };
            // With a cache in 8 bits: tiles to be converted so far, and places in use, with the phase that ends the last
            // copy to each.
            int g = 0;
            uint32_t g_used = 0, g_phase = 0;
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
                    // what brings the scales of 16 keys each; 0 for keys without a page or past the end (their rows become 0)
                    auto bring_scales = [&](const float* plane, uint32_t dst, uint32_t bar) {
                        const int from = __shfl_sync(0xffffffffu, page, 16 * lane >> A.C.shift & 31);
                        if (lane < 8) {
                            const bool there = from >= 0 && from < A.C.num_pages && t * kTile + 16 * lane < w.x.ctx;
                            const float* const src =
                                plane + (there ? from * A.scale_page + w.h * A.scale_head +
                                                     ((16 * lane & (A.C.page_tokens() - 1)) >> A.scale_shift) * A.scale_block
                                               : 0);
                            copy_word(dst + 4 * lane, src, there);
                        }
                        copies_arrive(bar);
                    };
                    // Tiles to be converted, K before V: one warp sees every phase of their places.
                    if (E8 && cached) {
#pragma unroll 1
                        for (int v = 0; ok && v < 2; ++v, ++g) {
                            const int gi = g % L::kGs;
                            const uint32_t bar = base + L::oGFull + 8 * gi;
                            if (!(ok = warp_wait(base + L::oGEmpty + 8 * gi, (uint32_t)(g / L::kGs & 1) ^ 1, stop))) break;
                            g_used |= 1u << gi;
                            g_phase = (g_phase & ~(1u << gi)) | (uint32_t)(g / L::kGs & 1) << gi;
                            if (lane == 0) bar_expect(bar, (uint32_t)(boxes << A.C.shift) * DP);
                            __syncwarp();
                            if (page >= 0)
                                copy_box(base + L::oG + gi * L::kPart + (lane << A.C.shift) * DP, v == 0 ? &M.kc : &M.vc, 0, 0, w.h, page, bar);
                            bring_scales(v == 0 ? A.ks : A.vs, base + L::oScale + 32 * gi, bar);
                        }
                        if (!ok) break;
                    }
                    if (E8) continue;  // new tokens' tiles are brought by those who convert
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
                for (int j = 0; j < L::kG; ++j)
                    if (g_used >> j & 1) drain(base + L::oGFull + 8 * j, g_phase >> j & 1);
                if (E8) asm volatile("cp.async.wait_all;" ::: "memory");
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
                const uint64_t q0 = operand(qs, 16), k0 = operand(ks, 16), v0 = operand(vs, E8 ? L::kHalf / 2 : L::kHalf);
                auto wait_k = [&] { return warp_wait(base + L::oKFull + 8 * ki, kp, stop); };
                // (with a cache in 8 bits halves of V are waited for as they are used)
                auto wait_v = [&]() -> bool { return E8 || warp_wait(base + L::oVReady + 8 * vi, vp, stop); };
                auto done_v = [&] {
#pragma unroll
                    for (int hf = 0; hf < (E8 ? 2 : 1); ++hf) {
                        done(base + L::oVEmpty + 8 * vi);
                        step(vi, vp, L::kV);
                    }
                };
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
                    constexpr int steps = E8 || !L::kApart ? 4 : 8;  // 16 keys each
                    int vj = vi;
                    uint32_t vq = vp;
#pragma unroll
                    for (int part = 0; part < 8; part += steps) {
                        if (!L::kApart || part == 0)
                            if (!warp_wait(base + (!L::kApart && part == 0 ? L::oPHalf : L::oPReady) + 8 * s, ps[s], stop)) return false;
                        if (E8 && !warp_wait(base + L::oVReady + 8 * vj, vq, stop)) return false;
                        tmem_after();
                        const uint64_t v = v0 + vj * (L::kVBytes / 16);
                        if (elect()) {
#pragma unroll
                            for (int e = part; e < part + steps; ++e)
                                mma_ts(tm + 256 + s * DP, tm + (L::kApart ? 384 + 64 * s : 128 * s) + 8 * e, v + 128 * (E8 ? e - part : e),
                                       kind_o, add || e > 0);
                        }
                        __syncwarp();
                        if (E8) step(vj, vq, L::kV);
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
                            ok = wait_v();
                            if (!ok) break;
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
                            done_v();
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
                            done_v();
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
        } else if (E8 && warp >= kConvertWarp) {
            // ---- Tiles of the cache: to 16 bits, times their scales. ----
            const int me = tid - 32 * kConvertWarp;  // 0 .. 127
            Walk<K>& w = reinterpret_cast<Walk<K>*>(sm + L::oWalk)[8 + warp - kConvertWarp];
            if (lane == 0) w.start(A, S, plan, near);
            __syncwarp();
            // Two warps take a tile's first 64 keys, two the others.  A thread takes 16 elements at the same place of
            // every `step`-th row: the swizzle of its vectors is the same in all of them.  Of eight lanes, whose
            // vectors go out together, four take one half of row r and four that of row r ^ 5 (with rows of 64
            // elements r and r + 1): their loads lie in 32 different banks, and so do both their stores.
            constexpr int chunks = DP / 16, step = 64 / chunks;
            const int team = me >> 6, you = me & 63;
            const int c = (you & 3) + (DP == 128 ? 4 * (you >> 3 & 1) : 0);
            const int row0 = DP == 128 ? (you >> 4) ^ ((you >> 2 & 1) * 5) : you / chunks;
            const int c2 = 2 * c & 7, swizzle = row0 & 7;
            const int at0 = row0 * 128 + (c2 ^ swizzle) * 16, at1 = row0 * 128 + ((c2 + 1) ^ swizzle) * 16;
            const int from = (64 * team + row0) * DP + (DP == 128 ? c ^ swizzle : c) * 16;
            // The team's half of the tile in place gi to rows from dst on, columns 64 .. of which lie `next` bytes
            // further; keys from `have` on become 0.  `over`: the power of two that they are divided by.
            auto convert = [&](int gi, char* dst, int next, int have, uint32_t over) {
                constexpr int turns = 64 / step;
                const char* const src = sm + L::oG + gi * L::kPart + from;
                const float* const all = reinterpret_cast<const float*>(sm + L::oScale) + 8 * gi;
                char* const to = dst + (c >> 2) * next;
                const bool plain = __all_sync(0xffffffffu, fits<BF16>(all[lane & 7]) && (!kRaised || over == 0));
                // Two turns a pass, the next pass's codes on their way.  (More of them unrolled are instructions that with the
                // softmax's do not stay in the instruction cache, and every warp waits: 4,000 tokens behind 25,000, 32/8 heads
                // of 128, took 1,920 us with four turns a pass, 1,844 with two, 1,892 with one, when this was measured.)
                auto passes = [&](auto plain_c) {
                    constexpr bool kPlain = decltype(plain_c)::value != 0;
                    constexpr int pass = kPlain ? 2 : 1;
                    uint4 x[pass];
                    float f[pass];
                    auto load = [&](int u) {
#pragma unroll
                        for (int e = 0; e < pass; ++e) {
                            x[e] = *reinterpret_cast<const uint4*>(src + (u + e) * (step * DP));
                            f[e] = all[4 * team + (u + e) * step / 16];
                            if (kRaised && !kPlain) f[e] *= __uint_as_float(127 - over << 23);
                            if (have < kTile && 64 * team + row0 + (u + e) * step >= have) {
                                x[e] = make_uint4(0, 0, 0, 0);
                                f[e] = 0.0f;
                            }
                        }
                    };
                    load(0);
#pragma unroll 1
                    for (int u = 0; u < turns; u += pass) {
                        uint4 y[pass];
                        float h[pass];
#pragma unroll
                        for (int e = 0; e < pass; ++e) y[e] = x[e], h[e] = f[e];
                        if (u + pass < turns) load(u + pass);
#pragma unroll
                        for (int e = 0; e < pass; ++e) {
                            char* const row = to + (u + e) * (step * 128);
                            const uint32_t mult = pack2<BF16>(h[e], h[e]);
                            *reinterpret_cast<uint4*>(row + at0) = widen<BF16, kPlain>(make_uint2(y[e].x, y[e].y), h[e], mult);
                            *reinterpret_cast<uint4*>(row + at1) = widen<BF16, kPlain>(make_uint2(y[e].z, y[e].w), h[e], mult);
                        }
                    }
                };
                if (plain)
                    passes(Count<1>{});
                else
                    passes(Count<0>{});
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            };
            int i = 0, g = 0;
            bool ok = true;
            // These warps write to the rings, or have it written, in the order of the tiles: they alone wait for every
            // phase of their places.  (A wait tells a phase from the one before it, not from the one before that.)
            const bool brings = (warp & 1) == 0;  // the team's half of new tokens' V tiles; the first team K tiles too
            // places with copies (bits 0 .. of K, 16 .. of V) and the phase that ends the last (8 .., 24 ..)
            uint32_t copies = 0;
            // A tile of the cache: K, then V.  With rows of 64 the conversion's instructions are there once, with rows of 128
            // twice: 8 prompts of 100 to 1,500 tokens behind up to 8,192 (24/4 heads of 64) 343 and 376 us, 4,000 tokens
            // behind 25,000 (32/8 heads of 128) 1,842 and 1,757.
            auto both = [&](int tile, int t, uint32_t over) {
                const int ki = tile % L::kK, at = 2 * tile + team, vi = at % L::kV;
#pragma unroll(DP == 64 ? 1 : 2)
                for (int v = 0; v < 2; ++v) {
                    const int gi = g % L::kGs;
                    const uint32_t empty = v == 0 ? base + L::oKEmpty + 8 * ki : base + L::oVEmpty + 8 * vi;
                    const int turn = v == 0 ? tile / L::kK : at / L::kV;
                    if (!warp_wait(base + L::oGFull + 8 * gi, (uint32_t)(g / L::kGs & 1), stop)) return false;
                    if (!warp_wait(empty, (uint32_t)(turn & 1) ^ 1, stop)) return false;
                    convert(gi, sm + (v == 0 ? L::oK + ki * L::kBytes + team * (64 * 128) : L::oV + vi * L::kVBytes),
                            v == 0 ? L::kHalf : L::kHalf / 2, v == 0 ? kTile : w.x.ctx - t * kTile, over >> 8 * v & 255);
                    if (lane == 0) {
                        bar_arrive(v == 0 ? base + L::oKFull + 8 * ki : base + L::oVReady + 8 * vi);
                        bar_arrive(base + L::oGEmpty + 8 * gi);
                    }
                    ++g;
                }
                return true;
            };
            // A tile of new tokens.
            auto keys = [&](int tile, int t) {
                const int ki = tile % L::kK;
                const uint32_t full = base + L::oKFull + 8 * ki;
                if (!warp_wait(base + L::oKEmpty + 8 * ki, (uint32_t)(tile / L::kK & 1) ^ 1, stop)) return false;
                if (warp != kConvertWarp) {
                    if (lane == 0) bar_arrive(full);
                } else {
                    copies = (copies & ~(0x100u << ki)) | 1u << ki | (uint32_t)(tile / L::kK & 1) << (8 + ki);
                    if (lane == 0) bar_expect(full, (uint32_t)(L::kHalves * S.kbox) * 128u);
                    __syncwarp();
                    if (lane < L::kHalves)
                        copy_box(ks + ki * L::kBytes + lane * L::kHalf, &M.k, 64 * lane, w.h, w.x.base + (t - w.x.ctx_tiles) * kTile, 0, full);
                }
                return true;
            };
            auto values = [&](int tile, int t) {
                const int n0 = (t - w.x.ctx_tiles) * kTile, have = w.x.rows - n0;
                const int at = 2 * tile + team, vi = at % L::kV;
                const uint32_t full = base + L::oVFull + 8 * vi;
                char* const place = sm + L::oV + vi * L::kVBytes;
                if (!warp_wait(base + L::oVEmpty + 8 * vi, (uint32_t)(at / L::kV & 1) ^ 1, stop)) return false;
                if (have > 64 * team) {
                    // (the V warp hands it on)
                    if (brings) {
                        copies ^= (copies >> (16 + vi) & 1) << (24 + vi);
                        copies |= 0x10000u << vi;
                        if (lane == 0) bar_expect(full, (uint32_t)(L::kHalves * S.vbox) * 128u);
                        __syncwarp();
                        if (lane < L::kHalves)
                            copy_box(vs + vi * L::kVBytes + lane * (L::kHalf / 2), &M.v, 64 * lane, w.h, w.x.base + n0 + 64 * team, 0, full);
                    }
                } else {
                    // a half without tokens
                    for (int e = you; e < L::kVBytes / 16; e += 64) *reinterpret_cast<uint4*>(place + 16 * e) = make_uint4(0, 0, 0, 0);
                    if (you < 4) bad[4 * vi + you] = 0;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) bar_arrive(base + L::oVReady + 8 * vi);
                }
                return true;
            };
            for (int seg = 0; ok && w.left > 0; ++seg) {
                uint32_t over = 0;
                if (kRaised) {
                    if (!(ok = warp_wait(base + L::oRaised + 8 * (seg & 1), (uint32_t)(seg >> 1 & 1), stop))) break;
                    over = reinterpret_cast<const uint32_t*>(sm + L::oRaise)[seg & 1];
                    __syncwarp();
                    if (lane == 0) bar_arrive(base + L::oRaisedRead + 8 * (seg & 1));
                }
                for (int t = w.t0; ok && t < w.t1; ++t, ++i) ok = t < w.x.ctx_tiles ? both(i, t, over) : keys(i, t) && values(i, t);
                __syncwarp();
                if (lane == 0) w.next(A, S, plan, near);
                __syncwarp();
            }
            if (!ok && brings) {
                // Leave no copy in flight.
                const long long t0 = clock64();
                auto drain = [&](uint32_t bar, uint32_t parity) {
                    while (!bar_try(bar, parity) && clock64() - t0 < kWaitClocks) {}
                };
                for (int j = 0; j < L::kK; ++j)
                    if (copies >> j & 1) drain(base + L::oKFull + 8 * j, copies >> (8 + j) & 1);
                for (int j = 0; j < L::kV; ++j)
                    if (copies >> (16 + j) & 1) drain(base + L::oVFull + 8 * j, copies >> (24 + j) & 1);
            }
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
            if (E8) {
                // new tokens, by halves of 64 keys; the cache's rows are converted by other warps
                uint32_t phase = 0;  // of each place's copies
                for (; ok && w.left > 0; w.next(A, S, plan, near)) {
                    i += w.t1 - w.t0;
                    for (int t = w.t0 > w.x.ctx_tiles ? w.t0 : w.x.ctx_tiles; ok && t < w.t1; ++t) {
                        const int n0 = (t - w.x.ctx_tiles) * kTile, have = w.x.rows - n0;
                        const bool look = n0 + kTile - 1 > w.item * S.block;
                        for (int hf = 0; hf < 2; ++hf) {
                            const int at = 2 * (i - (w.t1 - t)) + hf, vi = at % L::kV, left = have - 64 * hf;
                            if (left <= 0) break;
                            if (!(ok = warp_wait(base + L::oVFull + 8 * vi, phase >> vi & 1, stop))) break;
                            phase ^= 1u << vi;
                            if (left < 64 || look) {
                                char* const tile = sm + L::oV + vi * L::kVBytes;
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const int r = 32 * u + lane;
                                    const bool clear = r >= left;
                                    bool odd = false;
                                    if (look && 32 * u < left) {
                                        uint32_t hit = 0;
#pragma unroll
                                        for (int c = 0; c < 8 * L::kHalves; ++c) {
                                            const int p = (c & 8) * (L::kHalf / 16) + r * 128 + (((c & 7) + lane) & 7) * 16;
                                            const uint4 x = *reinterpret_cast<const uint4*>(tile + p);
                                            hit |= ((x.x & expo) + one) | ((x.y & expo) + one) | ((x.z & expo) + one) | ((x.w & expo) + one);
                                        }
                                        odd = !clear && (hit & 0x80008000u) != 0;
                                    }
                                    if (clear || odd)
#pragma unroll
                                        for (int c = 0; c < 8 * L::kHalves; ++c) {
                                            const int p = (c & 8) * (L::kHalf / 16) + r * 128 + (((c & 7) + lane) & 7) * 16;
                                            *reinterpret_cast<uint4*>(tile + p) = make_uint4(0, 0, 0, 0);
                                        }
                                    const uint32_t word = __ballot_sync(0xffffffffu, odd);
                                    if (lane == 0) bad[4 * vi + u] = word;
                                }
                                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            }
                            __syncwarp();
                            if (lane < 2) bar_arrive(base + L::oVReady + 8 * vi);
                        }
                    }
                }
            }
            for (; !E8 && ok && w.left > 0; w.next(A, S, plan, near)) {
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
    // The joins run with equal shares of the registers again.  (Behind the barrier: a warp without work would else take back
    // what it gave before the softmax warps have it, and one of them would wait for registers for ever.)
    if (E8) {
        if (warp < kCopyWarp)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 128;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
    }
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
        if (cut[i].total > 0) join_item<DP, BF16, K, kThreads>(A, S, W, plan, cuts, cut[i], stop);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <int DP, bool BF16, bool PROMPT, bool E8>
int launch_mma(const Attend& A, const Shape& S, const Maps& M, void* scratch, cudaStream_t s)
{
    using L = Lay<DP, PROMPT, E8>;
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CLK_ECUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit) || dev > 63) {
        if (cudaFuncSetAttribute(k_attend<DP, BF16, PROMPT, E8>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal) != cudaSuccess)
            return CLK_ECUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)S.ctas);
    cfg.blockDim = dim3(kThreads<E8>);
    cfg.dynamicSmemBytes = L::kTotal;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the joins wait on one another
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, k_attend<DP, BF16, PROMPT, E8>, M, A, S, scratch));
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
    const int per = A.ks != nullptr ? 16 : 8;
    if (A.kc != nullptr && (!map_stride(A.page_stride, A.C.num_pages, per) || !map_stride(A.head_stride, A.kv_heads, per) ||
                            !map_stride(A.tok_stride, 2, per)))
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
    const bool eight = A.ks != nullptr;
    const int vrows = !eight ? kTile : prompt ? kTile / 2 : kTile / 4;  // of V's places
    S.vbox = S.kbox < vrows ? S.kbox : vrows;
    S.ctas = num_sms();
    S.wide_out = A.dim % 16 == 0 && aligned(A.out, 32);
    S.log2_scale = (float)((double)A.scale * 1.4426950408889634);
    if (S.ctas < 1) return CLK_ECUDA;
    Maps M;
    const int64_t nq[3] = {A.q_heads, rows, reqs}, nk[3] = {A.kv_heads, rows, reqs};
    const int64_t sq[3] = {A.q_head, A.q_row, A.q_req}, sk[3] = {A.k_head, A.k_row, A.k_req}, sv[3] = {A.v_head, A.v_row, A.v_req};
    bool ok = encode(f, &M.q, A.dtype, A.q, A.dim, nq, sq, 64, A.group, S.qbox) &&
              encode(f, &M.k, A.dtype, A.k, A.dim, nk, sk, 64, 1, S.kbox) && encode(f, &M.v, A.dtype, A.v, A.dim, nk, sv, 64, 1, S.vbox);
    const bool wide = A.dim > 64, bf = A.dtype == CLK_DTYPE_BF16;
    if (A.kc != nullptr) {
        const int64_t np[3] = {A.C.page_tokens(), A.kv_heads, A.C.num_pages};
        const int64_t sp[3] = {A.tok_stride, A.head_stride, A.page_stride};
        const int32_t type = eight ? CLK_DTYPE_E4M3 : A.dtype;
        const int b0 = eight ? pad_dim(A.dim) : 64;
        // rows of 64 bytes: an operand of the products has their swizzle, what is converted lies as it is
        const CUtensorMapSwizzle vs = b0 * (eight ? 1 : 2) == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE;
        const CUtensorMapSwizzle ks = vs == CU_TENSOR_MAP_SWIZZLE_NONE && !prompt ? CU_TENSOR_MAP_SWIZZLE_64B : vs;
        ok = ok && encode(f, &M.kc, type, A.kc, A.dim, np, sp, b0, A.C.page_tokens(), 1, ks) &&
             encode(f, &M.vc, type, A.vc, A.dim, np, sp, b0, A.C.page_tokens(), 1, vs);
    } else {
        M.kc = M.vc = M.k;  // not read: no request has cached rows
    }
    if (!ok) return CLK_EINVAL;
    if (eight && !prompt) return attend_tree8_launch(A, S, M, scratch, s);
#define CLK_GO(D, T) return eight ? launch_mma<D, T, true, true>(A, S, M, scratch, s) : prompt ? launch_mma<D, T, true, false>(A, S, M, scratch, s) \
                                                                                             : launch_mma<D, T, false, false>(A, S, M, scratch, s)
    if (wide) {
        if (bf) CLK_GO(128, true);
        CLK_GO(128, false);
    }
    if (bf) CLK_GO(64, true);
    CLK_GO(64, false);
#undef CLK_GO
}

}  // namespace clk
