// Attention of drafted trees over a paged cache in 8 bits on the tensor cores
// (sm_103a).
//
// Items, shares and joins are those of clk_attend_work.cuh, rows and streams
// those of the kernel over 16 bits (clk_attend_mma.cu): rows are (token, head
// of the group) pairs, and two groups of softmax warps take alternate tiles of
// 128 keys.
//
// Nothing that the cache holds is multiplied by its scale.  K goes to the
// tensor cores as it is: scores are the sum of products of 8 bits with Q in two
// parts (bfloat16) or three (float16), each the rounding to 8 bits of what the
// parts before it leave of the row over its own power of two.  Such products
// are exact and are summed in float32.  K's scale and the row's power of two
// multiply the scores in the softmax.  V's codes become float16, which holds
// them exactly (one instruction a pair), and its scales go into the weights,
// where a power of two costs nothing: it is part of the exponent.  (Multiplied
// into V instead, V took four times the instructions, and with K in 16 bits too
// eight: 64 requests of 2,000 to 32,000 tokens, 32/8 heads of 128, 1,083 us
// with both in 16 bits, 640 and after some steps 511 with V alone, 506 to 515
// so.)
// New tokens' K and V stay in their own type.
//
// A row's 128 columns belong to two threads in two warps, so that a tile's
// weights take half as long: each has its own sum, but both have the reference
// M, which O shares.  So the pair meets once a tile before it gives its weights
// away; where a row of either asks for it, both take up the new M.  (With one
// thread a row eight requests of 262,144 tokens took 322 us, with two 278; 256
// of 300 to 4,096 tokens with heads of 64, though, 185 and 202, and 191 after
// later steps.)
//
// What bounds it: 128 keys of 128 elements take DRAM 1,400 cycles of an SM.  The
// products take 1,050 (bfloat16; 1,300 float16), those with Q's parts from
// shared memory as long as it needs to pass their operands; shared memory as a
// whole passes 176 KB (208 KB) at 128 bytes a cycle, 1,375 (1,625).  A tile
// measures 2,300: a stream's scores wait for its products with V (they lie where
// the weights were), its softmax (some 2,300 cycles, of which 900 are weights
// and the rest waits, loads of scales, the meeting and the way to tensor memory)
// for the scores, and two streams do not quite fill that.  With heads of 64 the
// tile's fixed costs are the same and its bytes half.
//
// The code of all roles has to stay in the instruction cache; where loops of
// the conversion were unrolled, three quarters of the fetches hit and everything
// waited.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "clk.h"
#include "clk_attend.h"
#include "clk_attend_work.cuh"
#include "clk_cache.h"
#include "clk_eight.cuh"
#include "clk_host.h"
#include "clk_mma.cuh"

namespace clk {
namespace {

// 16 softmax, 2 copies, 1 products, 4 that convert (and one that fills its warpgroup)
constexpr int kWarps = 24, kThreads = 32 * kWarps;
constexpr int kCopyWarp = 16, kMmaWarp = 17, kCopyWarp2 = 18, kConvertWarp = 20;

template <int DP, bool BF16>
struct Lay {
    static constexpr int kHalves = DP / 64;
    static constexpr int kHalf = kTile * 128;  // bytes of 64 columns of a tile of 16 bits
    static constexpr int kBytes = kHalves * kHalf;
    static constexpr int kPart = kTile * DP;   // bytes of a tile of 8 bits
    // Rows of 64 leave room in tensor memory for weights beside the scores; with rows of 128 they lie over them.
    static constexpr bool kApart = DP == 64;
    static constexpr int kParts = BF16 ? 2 : 3;            // of Q
    static constexpr int kQB = DP == 128 ? 1 : 2;          // items whose Q is held
    static constexpr int kK = DP == 128 ? (BF16 ? 3 : 2) : 7;  // K tiles in the ring (8 bits, or 64 new tokens)
    static constexpr int kVBytes = kBytes / 4;             // 32 keys of the V tile of 16 bits
    static constexpr int kG = DP == 128 ? 4 : 7;           // V tiles as the cache holds them
    // (Rows of 64: 256 requests of 300 to 4,096 tokens took 198 us with seven tiles of each, 199 with six, 213 with four of K.
    // A second V tile of 16 bits made no difference.)
    // Scales outlive their tiles: the softmax warps read them.  A place is written again when the tile kScales before is
    // weighed: the copy of a tile waits for the scores of the one kK before, which follow the weights of kK + 2.
    static constexpr int kScales = 16;
    static_assert(kScales >= kK + 2, "scales in use");
    static constexpr int oParts = kQB * kBytes, oK = oParts + kQB * kParts * kPart, oV = oK + kK * kPart, oG = oV + kBytes;
    // after the tiles
    static constexpr int oKFull = oG + kG * kPart, oKEmpty = oKFull + 8 * kK;
    static constexpr int oVFull = oKEmpty + 8 * kK, oVReady = oVFull + 32, oVEmpty = oVReady + 16;  // of quarters; of halves
    static constexpr int oGFull = oVEmpty + 16, oGEmpty = oGFull + 8 * kG;
    static constexpr int oPartsReady = oGEmpty + 8 * kG, oFactorRead = oPartsReady + 8 * kQB;
    static constexpr int oQFull = oFactorRead + 8 * kQB, oQEmpty = oQFull + 8 * kQB;
    static constexpr int oSFull = oQEmpty + 8 * kQB, oSFree = oSFull + 16, oPReady = oSFree + 16, oPHalf = oPReady + 16, oODone = oPHalf + 16;
    static constexpr int oLook = oODone + 16, oPair = oLook + 16;
    static constexpr int oStatReady = oPair + 64, oDrain = oStatReady + 8;
    static constexpr int oBars = oDrain + 8;  // end of the barriers
    static constexpr int oBad = (oBars + 15) / 16 * 16;        // uint32[2]
    static constexpr int oAgree = oBad + 16;               // uint32[8][2][2]: a pair's wishes, by phases
    static constexpr int oScale = oAgree + 128;                // float[kScales][2][8]: K's and V's, of blocks of 16 keys
    static constexpr int oFactor = oScale + 64 * kScales;      // float[kQB][128]: what a row of Q's parts is to be multiplied by
    static constexpr int oNear = oFactor + kQB * kTile * 4;    // Reach[kNear]
    static constexpr int oPlan = oNear + kNear * (int)sizeof(Reach);
    static constexpr int oCut = oPlan + (int)sizeof(Plan);     // Cut[2]: of items that end here, that begin here
    static constexpr int oWalk = (oCut + 2 * (int)sizeof(Cut) + 7) / 8 * 8;  // Walk[20]: softmax and converting warps
    static constexpr int oStop = oWalk + 20 * (int)sizeof(Walk<Trees8>), oTmem = oStop + 4;
    static constexpr int oStat = (oTmem + 4 + 15) / 16 * 16;   // float2[2][2][128]: of streams, of halves of their tiles
    static constexpr int kTotal = oStat + 4 * kTile * 8;
    static_assert(kTotal <= 232448, "shared memory");
};

template <int DP, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) k_attend_tree8(const __grid_constant__ Maps M, const __grid_constant__ Attend A,
                                                              const __grid_constant__ Shape S, void* scratch)
{
    using L = Lay<DP, BF16>;
    using K = Trees8;
    extern __shared__ __align__(1024) char sm[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t base = smem_addr(sm);
    Plan& plan = *reinterpret_cast<Plan*>(sm + L::oPlan);
    Reach* const near = reinterpret_cast<Reach*>(sm + L::oNear);
    Cut* const cut = reinterpret_cast<Cut*>(sm + L::oCut);
    volatile int* const stop = reinterpret_cast<volatile int*>(sm + L::oStop);
    volatile uint32_t* const bad = reinterpret_cast<volatile uint32_t*>(sm + L::oBad);
    const Scratch W = scratch_of(scratch, S.ctas, kTile);

    const uint32_t call = tid == 0 ? __ldcg(W.flag + blockIdx.x) : 0;
    const long long began = clock64();
    // ---- Start: tensor memory, barriers and descriptors, while the requests' data is on its way. ----
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base + L::oTmem) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else if (warp == kCopyWarp) {
        if (lane < 5)
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<const char*>(&M) + lane * sizeof(CUtensorMap)) : "memory");
    } else if (tid == 32 * kConvertWarp) {
        for (int i = 0; i < L::kK; ++i) {
            bar_init(base + L::oKFull + 8 * i, 1 + 32);  // the copies of a tile, and of its scales by a warp's lanes
            bar_init(base + L::oKEmpty + 8 * i, 1);
        }
        for (int i = 0; i < 4; ++i) bar_init(base + L::oVFull + 8 * i, 1);
        for (int i = 0; i < 2; ++i) {
            bar_init(base + L::oVReady + 8 * i, 2);
            bar_init(base + L::oVEmpty + 8 * i, 1);
        }
        for (int i = 0; i < L::kG; ++i) {
            bar_init(base + L::oGFull + 8 * i, 1);
            bar_init(base + L::oGEmpty + 8 * i, 4);
        }
        for (int i = 0; i < L::kQB; ++i) {
            bar_init(base + L::oPartsReady + 8 * i, 4);
            bar_init(base + L::oFactorRead + 8 * i, 16);
            bar_init(base + L::oQFull + 8 * i, 1);
            bar_init(base + L::oQEmpty + 8 * i, 1 + 4);  // the products', and the warps' that split it
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(base + L::oSFull + 8 * i, 1);
            bar_init(base + L::oSFree + 8 * i, 8);
            bar_init(base + L::oPHalf + 8 * i, 4);
            bar_init(base + L::oPReady + 8 * i, 4);
            bar_init(base + L::oODone + 8 * i, 1);
            bar_init(base + L::oLook + 8 * i, 2);
        }
        for (int i = 0; i < 8; ++i) bar_init(base + L::oPair + 8 * i, 2);
        bar_init(base + L::oStatReady, 16);
        bar_init(base + L::oDrain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // (the rings are not in use yet)
    make_plan<K, kThreads>(A, S, reinterpret_cast<long long*>(sm), plan, near, cut, stop, call, began, __shfl_sync(0xffffffffu, tid >> 5, 0));
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the planning scratch lies where tiles go
    tmem_before();
    __syncthreads();
    tmem_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::oTmem);
    const uint32_t qs = base, ks = base + L::oK, vs = base + L::oV;

    // Every wait below tells a phase of its barrier from the one before it, and no others.  So whoever waits on a barrier
    // passes all its phases in order, and no phase ends before those have passed the one before it who wait for both.
    // Registers: 768 threads x 80 at launch; 512 x 88 + 256 x 64 after the split.
    if (warp < kCopyWarp)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
    else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp < kCopyWarp) {
        // ---- Softmax: two threads per row, each with 64 of a tile's columns. ----
        const int s = warp >> 3, h = warp >> 2 & 1, row = tid & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        // this half's scores, the stream's sums, this half's weights
        const uint32_t tS = lanes + 128 * s + 64 * h, tO = lanes + 256 + s * DP, tP = L::kApart ? lanes + 384 + 64 * s + 32 * h : tS;
        const int tk = row / A.group, g = row - tk * A.group;  // token of the row tile, head of the group
        const float cs = S.log2_scale;
        // A weight is p = exp2(z - M), z = x cs, with a whole number M.  V's codes are multiplied by t = p v, v the scale of
        // their 16 keys, in float16.  Where v = 2^k, t = exp2(z + k - M) comes out of the exponential itself, and the sum of
        // p is that of t times 2^-k: no multiplication an element.  M follows a row where its weights have grown too large;
        // up to there size costs no precision in floating point.  (The largest t starts at 2^5 to 2^6, so that small weights
        // keep their bits, and may grow to where 16 of them add up to 2^15.  Rounding loses at most 2^-25 a key: 2^-30 of
        // the largest.  Starting at 2^4, 2^6 and 2^7 measured 507, 511, 520 us with 64 requests of 2,000 to 32,000 tokens.)
        // The largest p starts at up to 2^100: V's scales may be as small as 2^-100.  That t stays a normal number where p
        // matters, however far V's scales lie apart, takes k of -60 to 30 and M not far above the scores; else p and t are
        // computed each.  (Then M may move by more than a float32's exponent, and a sum of p with it in two steps.)
        constexpr float lift = 6.0f, lift_sum = 100.0f, most_sum = 0x1p110f, most_weight = 32768.0f;
        uint32_t sp = 0, od = 0, look = 0, pp = 0;  // phases of SFull, ODone, Look, Pair
        // The two warps with the same rows meet: < 0 if one gave up, else whether one wished.
        auto agree = [&](bool wish) -> int {
            const int pair = 4 * s + (warp & 3);
            volatile uint32_t* const at = reinterpret_cast<volatile uint32_t*>(sm + L::oAgree) + 4 * pair + 2 * pp;
            const bool any = __any_sync(0xffffffffu, wish);
            __syncwarp();
            if (lane == 0) {
                at[h] = any;
                bar_arrive(base + L::oPair + 8 * pair);
            }
            if (!warp_wait(base + L::oPair + 8 * pair, pp, stop)) return -1;
            pp ^= 1;
            return (int)(at[0] | at[1]);
        };
        float2* const stat = reinterpret_cast<float2*>(sm + L::oStat);
        int gi = 0, gk = 0, seg = 0;  // tiles, cached tiles and segments before this segment
        bool ok = true;
        Walk<K>& w = reinterpret_cast<Walk<K>*>(sm + L::oWalk)[warp];
        if (lane == 0) w.start(A, S, plan, near);
        __syncwarp();
        while (ok && w.left > 0) {
            const int len = w.t1 - w.t0, t0 = w.t0, mine = (len + 1 - s) / 2;
            const int token = w.item * S.block + tk;
            const int ctx = w.x.ctx, ctx_tiles = w.x.ctx_tiles;
            const bool real = tk < S.tok && token < w.x.rows;
            unsigned long long seen = 0;
            if (real && w.t1 > ctx_tiles) {
                seen = (unsigned long long)A.mask[(int64_t)w.b * A.N + token];
                if (w.x.rows < 64) seen &= (1ull << w.x.rows) - 1;
            }
            // A warp without rows goes along without its share of the work (its rows of tensor memory are its own).
            const bool idle = !__any_sync(0xffffffffu, real);
            float factor = 0.0f;  // of this row's scores with the cache
            bool has_factor = false;
            float M = -INFINITY, sum = 0.0f;
            bool wide = false;  // M is far above the scores
            for (int j = 0; j < mine; ++j) {
                const int t = t0 + 2 * j + s;
                const bool cached = t < ctx_tiles;
                if (!(ok = warp_wait(base + L::oSFull + 8 * s, sp, stop))) break;
                sp ^= 1;
                tmem_after();
                if (cached && !has_factor) {
                    const int qi = seg % L::kQB;
                    factor = reinterpret_cast<const float*>(sm + L::oFactor)[qi * kTile + row];
                    has_factor = true;
                    __syncwarp();
                    if (lane == 0) bar_arrive(base + L::oFactorRead + 8 * qi);
                }
                if (L::kApart && j > 0) {
                    // this stream's last product is done with O and the weights
                    if (!(ok = warp_wait(base + L::oODone + 8 * s, od, stop))) break;
                    od ^= 1;
                    tmem_after();
                }
                if (!cached) {
                    if (!(ok = warp_wait(base + L::oLook + 8 * s, look, stop))) break;
                    look ^= 1;
                    // rows of V that were not finite: NaN for those who see them (a tree's tokens are the first 64 keys)
                    if ((bad[0] & (uint32_t)seen) != 0 || (bad[1] & (uint32_t)(seen >> 32)) != 0) sum = NAN;
                }
                if (idle) {
                    tmem_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (L::kApart) bar_arrive(base + L::oSFree + 8 * s);
                        bar_arrive(base + (h == 0 ? L::oPHalf : L::oPReady) + 8 * s);
                    }
                    continue;
                }
                const float4* const scales = reinterpret_cast<const float4*>(sm + L::oScale) + 4 * ((gk + t - t0) % L::kScales);
                const int most = ctx - t * kTile;
                // plain: the rows see all of the tile, and exponents of V's scales can go into the weights' without loss
                bool plain = cached && most >= kTile;
                if (plain) {
                    const uint32_t v = reinterpret_cast<const uint32_t*>(scales)[8 + (lane & 7)];
                    plain = __all_sync(0xffffffffu, (v & 0x7fffffu) == 0 && v >= (127u - 60 << 23) && v <= (127u + 30 << 23) && !wide);
                }
                // What the row sees of this half's columns 32 c ..
                auto visible = [&](int c) -> uint32_t {
                    if (!cached) return h == 0 ? (uint32_t)(seen >> (32 * c)) : 0u;
                    const int n = most - 64 * h - 32 * c;
                    return n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
                };
                // The columns' factors, 16 at a time; and V's scales there.
                float f[4], v[4];
                {
                    const float4 f4 = scales[h], v4 = scales[2 + h];
                    const float f0 = factor * cs;
                    f[0] = cached ? f0 * f4.x : cs, f[1] = cached ? f0 * f4.y : cs, f[2] = cached ? f0 * f4.z : cs, f[3] = cached ? f0 * f4.w : cs;
                    v[0] = cached ? v4.x : 1.0f, v[1] = cached ? v4.y : 1.0f, v[2] = cached ? v4.z : 1.0f, v[3] = cached ? v4.w : 1.0f;
                }
                // Some row of the pair got too large weights, or these are its first: M follows, and what was summed up with
                // the old one.
                auto follow = [&]() -> bool {
                    float top = -INFINITY, heavy = -INFINITY;
#pragma unroll 1
                    for (int i = 0; i < 2; ++i) {
                        uint32_t x[32];
                        tmem_load(tS + 32 * i, x);
                        const uint32_t vis = visible(i);
                        tmem_load_wait();
                        tmem_loaded(x);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float fq = i == 0 ? f[q] : f[2 + q], vq = i == 0 ? v[q] : v[2 + q];
                            float m = -INFINITY;
#pragma unroll
                            for (int e = 16 * q; e < 16 * q + 16; ++e)
                                if (vis >> e & 1) m = fmaxf(m, __uint_as_float(x[e]) * fq);
                            top = fmaxf(top, m);
                            heavy = fmaxf(heavy, m + __log2f(fabsf(vq)));
                        }
                    }
                    stat[(2 * s + h) * kTile + row] = make_float2(top, heavy);
                    if (agree(false) < 0) return false;
                    const float2 other = stat[(2 * s + 1 - h) * kTile + row];
                    top = fmaxf(top, other.x);
                    heavy = fmaxf(heavy, other.y);
                    // whole numbers: what is rescaled keeps its digits
                    const bool none = M == -INFINITY;
                    float m = fmaxf(ceilf(heavy) - lift, ceilf(top) - lift_sum);
                    m = top == -INFINITY ? M : none ? m : fmaxf(M, m);
                    const float fix = none ? 1.0f : exp2f(M - m);
                    if (!none) sum = moved(sum, M - m);
                    M = m;
                    wide = M > top + 30.0f;
                    if (!__any_sync(0xffffffffu, fix != 1.0f)) return true;
                    // O is complete: weights over the scores mean that these scores' product was issued after this stream's
                    // last P V; else it was waited for.  Each warp takes half of its columns.
                    if (j > 0)
#pragma unroll 1
                        for (int i = 0; i < DP / 32; ++i) {
                            uint32_t o[16];
                            const uint32_t at = tO + h * (DP / 2) + 16 * i;
                            tmem_load16(at, o);
                            tmem_load_wait();
                            tmem_loaded16(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fix);
                            tmem_store16(at, o);
                        }
                    tmem_store_wait();
                    return true;  // (weights are given away after the pair has met again)
                };
                float chunk;
                uint32_t y[32];
                for (int again = 0;; ++again) {
                    const float off = M == -INFINITY ? 0.0f : -M;
                    float heaviest = 0.0f;
                    chunk = 0.0f;
                    // The weights; kPlain: seen all, V's scales powers of two.
                    auto weigh = [&](auto plain_c) {
                        constexpr bool kPlain = decltype(plain_c)::value != 0;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t x[32];
                            tmem_load(tS + 32 * i, x);
                            const uint32_t vis = kPlain ? 0u : visible(i);
                            tmem_load_wait();
                            tmem_loaded(x);
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const float vq = v[2 * i + q];
                                const uint32_t a = __float_as_uint(f[2 * i + q]);
                                const uint32_t b = __float_as_uint(kPlain ? off + (float)((int)(__float_as_uint(vq) >> 23) - 127) : off);
                                const uint64_t a2 = pair(a, a), b2 = pair(b, b);
                                uint64_t part[2] = {0, 0};
#pragma unroll
                                for (int e = 8 * q; e < 8 * q + 8; ++e) {
                                    float2 z = unpair(fma2(pair(x[2 * e], x[2 * e + 1]), a2, b2));
                                    if (!kPlain) {
                                        if (!(vis >> (2 * e) & 1)) z.x = -INFINITY;
                                        if (!(vis >> (2 * e + 1) & 1)) z.y = -INFINITY;
                                    }
                                    float2 t = make_float2(exp2_fast(z.x), exp2_fast(z.y));
                                    part[e & 1] = add2(part[e & 1], pair(__float_as_uint(t.x), __float_as_uint(t.y)));
                                    if (!kPlain) {
                                        t.x *= vq;
                                        t.y *= vq;
                                    }
                                    y[16 * i + e] = pack2<false>(t.x, t.y);
                                    if (!kPlain && BF16 && !cached) y[16 * i + e] = pack2<true>(t.x, t.y);
                                }
                                const float2 both = unpair(add2(part[0], part[1]));
                                const float t16 = both.x + both.y;
                                // sums of t, and of p = t 2^-k; or the other way round
                                heaviest = fmaxf(heaviest, kPlain ? t16 : t16 * fabsf(vq));
                                chunk = kPlain ? fmaf(t16, __uint_as_float((254u << 23) - __float_as_uint(vq)), chunk) : chunk + t16;
                            }
                        }
                    };
                    if (plain)
                        weigh(Count<1>{});
                    else
                        weigh(Count<0>{});
                    const bool large = chunk > most_sum || heaviest > (BF16 && !cached ? 0x1p60f : most_weight);
                    const int wish = agree(again == 0 && real && (large || M == -INFINITY));
                    ok = wish >= 0;
                    if (wish <= 0) break;
                    ok = follow();
                    if (!ok) break;
                    plain = plain && !__any_sync(0xffffffffu, wide);
                }
                if (!ok) break;
                sum += chunk;
                if (L::kApart) {
                    // the next scores may come
                    tmem_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(base + L::oSFree + 8 * s);
                }
                tmem_store16(tP, y);
                tmem_store16(tP + 16, y + 16);
                tmem_store_wait();
                tmem_before();
                __syncwarp();
                if (lane == 0) bar_arrive(base + (h == 0 ? L::oPHalf : L::oPReady) + 8 * s);
            }
            if (!ok) break;
            if (!has_factor && lane == 0) bar_arrive(base + L::oFactorRead + 8 * (seg % L::kQB));
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
            const int64_t out_row = (int64_t)w.b * A.N + token;
            char* const out = static_cast<char*>(A.out) + ((out_row * A.q_heads + w.h * A.group + g) * A.dim) * 2;
            // both streams' statistics, to weigh their sums
            stat[(2 * s + h) * kTile + row] = make_float2(M, sum);
            tmem_before();
            __syncwarp();
            if (lane == 0) bar_arrive(base + L::oStatReady);
            if (!(ok = warp_wait(base + L::oStatReady, 0, stop))) break;
            tmem_after();
            const float2 a = make_float2(stat[row].x, stat[row].y + stat[kTile + row].y);
            const float2 b = make_float2(stat[2 * kTile + row].x, stat[2 * kTile + row].y + stat[3 * kTile + row].y);
            const float m = fmaxf(a.x, b.x);
            const float w0 = a.x == -INFINITY ? 0.0f : exp2f(a.x - m);
            const float w1 = b.x == -INFINITY ? 0.0f : exp2f(b.x - m);
            const float l = (a.x == -INFINITY ? a.y * w0 : moved(a.y, a.x - m)) + (b.x == -INFINITY ? b.y * w1 : moved(b.y, b.x - m));
            // a stream without a visible key has no sum of products (or one of zeros)
            const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
#pragma unroll 1
            for (int c = (2 * s + h) * (DP / 64); !idle && c < (2 * s + h + 1) * (DP / 64); ++c) {
                uint32_t o[16], o1[16] = {};
                tmem_load16(lanes + 256 + 16 * c, o);
                if (len > 1) tmem_load16(lanes + 256 + DP + 16 * c, o1);
                tmem_load_wait();
                tmem_loaded16(o);
                tmem_loaded16(o1);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float v = 0.0f;
                    if (w0 != 0.0f) v = __uint_as_float(o[e]) * w0;
                    if (len > 1 && w1 != 0.0f) v = fmaf(__uint_as_float(o1[e]), w1, v);
                    if (l != l) v = l;
                    o[e] = __float_as_uint(v * inv);
                }
                if (!real) continue;
                if (whole) {
                    if (16 * c < A.dim) {  // (a multiple of 8)
                        uint32_t y[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) y[i] = pack2<BF16>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                        // a thread's row by whole sectors, where rows begin on one
                        if (S.wide_out) {
                            store32(out + 16 * c * 2, y);
                        } else {
                            *reinterpret_cast<uint4*>(out + 16 * c * 2) = make_uint4(y[0], y[1], y[2], y[3]);
                            if (16 * c + 8 < A.dim) *reinterpret_cast<uint4*>(out + 16 * c * 2 + 16) = make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    }
                } else {
                    float4* const to = reinterpret_cast<float4*>(W.sums) + (int64_t)slot * (DP / 4) * kTile + row;
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        to[(int64_t)(4 * c + e / 4) * kTile] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                                           __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                }
            }
            if (!whole && real && s == 0 && h == 0) W.ml[(int64_t)slot * kTile + row] = make_float2(m, l);
            // Neither stream's next sums may overwrite what the other still reads.
            tmem_before();
            __syncwarp();
            if (lane == 0) bar_arrive(base + L::oStatReady);
            if (!(ok = warp_wait(base + L::oStatReady, 1, stop))) break;
            gi += len;
            ++seg;
            gk += ctx_tiles > t0 ? (ctx_tiles < t0 + len ? ctx_tiles - t0 : len) : 0;
            __syncwarp();
            if (lane == 0) w.next(A, S, plan, near);
            __syncwarp();
        }
    } else if (warp == kCopyWarp || warp == kCopyWarp2) {
        // ---- Copies: one warp brings Q and K, and new tokens' K; one V. ----
        const bool is_k = warp == kCopyWarp;
        Walk<K> w;
        w.start(A, S, plan, near);
        int i = 0, seg = 0, gk = 0;
        int nq = 0, nk = 0;  // one past the last item, or tile of K or V, asked for
        int g = 0;           // V tiles so far
        bool ok = (base & 1023) == 0;  // the swizzle's period
        if (!ok) *stop = 1;
        const int pages = kTile >> A.C.shift;  // of a tile
        for (; ok && w.left > 0; w.next(A, S, plan, near), ++seg) {
            const int32_t* const table = A.C.table + (int64_t)w.x.slot * A.C.max_pages;
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
            if (is_k) {
                const int qi = seg % L::kQB;
                const uint32_t qb = base + L::oQFull + 8 * qi;
                if (!(ok = warp_wait(base + L::oQEmpty + 8 * qi, (uint32_t)(seg / L::kQB & 1) ^ 1, stop))) break;
                ++nq;
                if (lane == 0) bar_expect(qb, (uint32_t)L::kHalves * (uint32_t)(S.qbox * A.group) * 128u);
                __syncwarp();
                if (lane < L::kHalves)
                    copy_box(qs + qi * L::kBytes + lane * L::kHalf, &M.q, 64 * lane, w.h * A.group, w.item * S.block, w.b, qb);
            }
            for (int t = w.t0; t < w.t1; ++t, ++i) {
                const bool cached = t < w.x.ctx_tiles;
                if (cached && t * pages - at >= 32) {
                    at += 32;
                    now = then;
                    then = batch(at + 32);
                }
                int page = __shfl_sync(0xffffffffu, now, (t * pages - at + lane) & 31);
                if (!cached || lane >= pages) page = -1;
                if (!is_k && !cached) continue;  // new tokens' V is brought by those who convert
                const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(0xffffffffu, page >= 0)) << A.C.shift) * DP;
                const int n = is_k ? i : g, rings = is_k ? L::kK : L::kG, at_ring = n % rings;
                const uint32_t bar = base + (is_k ? L::oKFull : L::oGFull) + 8 * at_ring, empty = base + (is_k ? L::oKEmpty : L::oGEmpty) + 8 * at_ring;
                const uint32_t dst = base + (is_k ? L::oK : L::oG) + at_ring * L::kPart;
                if (!(ok = warp_wait(empty, (uint32_t)(n / rings & 1) ^ 1, stop))) break;
                nk = n + 1;
                ++g;
                if (lane == 0) bar_expect(bar, cached ? bytes : (uint32_t)(L::kHalves * S.kbox) * 128u);
                __syncwarp();
                if (cached) {
                    if (page >= 0) copy_box(dst + (lane << A.C.shift) * DP, is_k ? &M.kc : &M.vc, 0, 0, w.h, page, bar);
                    // K brings the scales of 16 keys each of both: 0 for keys without a page
                    // or past the end
                    const int from = __shfl_sync(0xffffffffu, page, 16 * (lane & 7) >> A.C.shift & 31);
                    if (is_k && lane < 16) {
                        const bool there = from >= 0 && from < A.C.num_pages && t * kTile + 16 * (lane & 7) < w.x.ctx;
                        const int64_t block = (16 * (lane & 7) & (A.C.page_tokens() - 1)) >> A.scale_shift;
                        copy_word(base + L::oScale + 64 * ((gk + t - w.t0) % L::kScales) + 4 * lane,
                                  (lane < 8 ? A.ks : A.vs) + (there ? from * A.scale_page + w.h * A.scale_head + block * A.scale_block : 0), there);
                    }
                } else if (lane < L::kHalves) {
                    // at most 64 rows, 64 columns a half
                    copy_box(dst + lane * (L::kHalf / 2), &M.k, 64 * lane, w.h, 0, w.b, bar);
                }
                if (is_k) copies_arrive(bar);
            }
            const int run = (w.t1 < w.x.ctx_tiles ? w.t1 : w.x.ctx_tiles) - w.t0;
            gk += run > 0 ? run : 0;
        }
        if (!ok) {
            // Leave no copy in flight.
            const long long t0 = clock64();
            auto drain = [&](uint32_t bar, uint32_t parity) {
                while (!bar_try(bar, parity) && clock64() - t0 < kWaitClocks) {}
            };
            for (int j = nq > L::kQB ? nq - L::kQB : 0; j < nq; ++j) drain(base + L::oQFull + 8 * (j % L::kQB), (uint32_t)(j / L::kQB & 1));
            const int rings = is_k ? L::kK : L::kG;
            for (int j = nk > rings ? nk - rings : 0; j < nk; ++j)
                drain(base + (is_k ? L::oKFull : L::oGFull) + 8 * (j % rings), (uint32_t)(j / rings & 1));
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        // Rows past the node counts are 0; the requests are dealt out to the CTAs.
        for (int b = blockIdx.x; !is_k && b < A.B; b += gridDim.x) {
            const int rows = attend_request(A, b, false).rows;
            const int64_t row = (int64_t)A.q_heads * A.dim / 8;
            uint4* const out = static_cast<uint4*>(A.out) + ((int64_t)b * A.N + rows) * row;
            for (int64_t e = lane; e < (A.N - rows) * row; e += 32) out[e] = make_uint4(0, 0, 0, 0);
        }
    } else if (warp == kMmaWarp) {
        // ---- Products: one lane issues them, the warp goes along. ----
        Walk<K> w;
        w.start(A, S, plan, near);
        // Shuffled values are the same in every lane for the compiler too.
        auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        const uint32_t tm = (uint32_t)same((int)tmem);
        constexpr uint32_t types = (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((kTile >> 4) << 24);
        constexpr uint32_t kind_n = types | ((64 >> 3) << 17);               // scores of 64 new keys
        constexpr uint32_t kind_v = (1u << 4) | ((kTile >> 4) << 24) | (1u << 16) | ((DP >> 3) << 17);  // V's codes in float16; rows run along the output
        constexpr uint32_t kind_o = types | (1u << 16) | ((DP >> 3) << 17);  // new tokens' V in its own type
        constexpr uint32_t kind_8 = (1u << 4) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24);  // 8 bits, 32 elements a product
        uint32_t ps[2] = {0, 0}, fs[2] = {1, 1};  // phases of PReady and SFree
        int qi = 0, ki = 0;
        uint32_t qp = 0, kp = 0, parts_phase = 0;
        bool ok = true;
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
        const uint64_t q0 = operand(qs, 16), k0 = operand(ks, 16), v0 = operand(vs, L::kHalf / 4);
        const uint64_t p0 = DP == 128 ? operand(base + L::oParts, 16) : operand_64(base + L::oParts);
        const uint64_t c0 = DP == 128 ? k0 : operand_64(ks);
        // Stream s's scores with K tile ki.
        auto scores = [&](int s, bool cached) {
            if (!warp_wait(base + L::oKFull + 8 * ki, kp, stop)) return false;
            if (L::kApart) {
                if (!warp_wait(base + L::oSFree + 8 * s, fs[s], stop)) return false;
                fs[s] ^= 1;
            }
            tmem_after();
            const uint64_t q = q0 + qi * (L::kBytes / 16), k = k0 + ki * (L::kPart / 16);
            const uint64_t p = p0 + qi * L::kParts * (L::kPart / 16), c = c0 + ki * (L::kPart / 16);
            if (elect()) {
                if (cached) {
#pragma unroll
                    for (int e = 0; e < L::kParts * (DP / 32); ++e) {
                        const int part = e / (DP / 32), at = e % (DP / 32) * 2;
                        mma_ss8(tm + 128 * s, p + part * (L::kPart / 16) + at, c + at, kind_8, e > 0);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < DP / 16; ++e)
                        mma_ss(tm + 128 * s, q + (e / 4) * (L::kHalf / 16) + (e % 4) * 2, k + (e / 4) * (L::kHalf / 32) + (e % 4) * 2, kind_n,
                               e > 0);
                }
                mma_commit(base + L::oSFull + 8 * s);
                mma_commit(base + L::oKEmpty + 8 * ki);
            }
            __syncwarp();
            step(ki, kp, L::kK);
            return true;
        };
        // Stream s's weights with the next V tile, by halves of 64 keys.
        uint32_t vp = 0;
        auto values = [&](int s, bool add, bool cached) {
            const uint32_t kind = cached ? kind_v : kind_o;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (!warp_wait(base + (half == 0 ? L::oPHalf : L::oPReady) + 8 * s, ps[s], stop)) return false;
                if (!warp_wait(base + L::oVReady + 8 * half, vp, stop)) return false;
                tmem_after();
                if (elect()) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // 16 keys each
                        mma_ts(tm + 256 + s * DP, tm + (L::kApart ? 384 + 64 * s + 32 * half : 128 * s + 64 * half) + 8 * e,
                               v0 + (2 * half + e / 2) * (L::kVBytes / 16) + 128 * (e & 1), kind, add || half + e > 0);
                    mma_commit(base + L::oVEmpty + 8 * half);
                }
                __syncwarp();
            }
            vp ^= 1;
            ps[s] ^= 1;
            return true;
        };
        for (; ok; w.next(A, S, plan, near)) {
            const int len = same(w.left > 0 ? w.t1 - w.t0 : 0), run = same(w.x.ctx_tiles - w.t0);
            if (len == 0) break;
            if (!(ok = warp_wait(base + L::oQFull + 8 * qi, qp, stop))) break;
            if (run > 0) {
                if (!(ok = warp_wait(base + L::oPartsReady + 8 * qi, parts_phase >> qi & 1, stop))) break;
                parts_phase ^= 1u << qi;
            }
            auto ahead = [&](int j) {
                if (j >= len) return true;
                if (!scores(j & 1, j < run)) return false;
                if (j + 1 == len) done(base + L::oQEmpty + 8 * qi);
                return true;
            };
            ok = ahead(0) && ahead(1);
            for (int j = 0; ok && j < len; ++j) {
                const int s = j & 1;
                if (L::kApart && !(ok = ahead(j + 2))) break;
                if (!(ok = values(s, j >= 2, j < run))) break;
                if (L::kApart || j + 2 >= len) done(base + L::oODone + 8 * s);
                if (!L::kApart) ok = ahead(j + 2);
            }
            step(qi, qp, L::kQB);
        }
        if (!ok) {
            // Products in flight end before tensor memory is given up.
            done(base + L::oDrain);
            const long long t0 = clock64();
            while (!bar_try(base + L::oDrain, 0) && clock64() - t0 < kWaitClocks) {}
        }
        __syncwarp();
    } else if (warp >= kConvertWarp) {
        // ---- V tiles of the cache: codes to float16; and Q in parts. ----
        Walk<K>& w = reinterpret_cast<Walk<K>*>(sm + L::oWalk)[16 + warp - kConvertWarp];
        if (lane == 0) w.start(A, S, plan, near);
        __syncwarp();
        // A warp has a quarter (32 keys) of every tile.  Of eight lanes, whose vectors go out together, four take one half of
        // row r and four that of row r ^ 5 (with rows of 64 elements r and r + 1): their loads of 16 codes lie in 32 different
        // banks, and so do both their stores.
        const int me = tid - 32 * kConvertWarp, team = me >> 5;
        const int c = (lane & 3) + (DP == 128 ? 4 * (lane >> 3 & 1) : 0);
        const int row0 = DP == 128 ? (lane >> 4) ^ ((lane >> 2 & 1) * 5) : lane >> 2;
        const int c2 = 2 * c & 7;
        const int at0 = row0 * 128 + (c2 ^ row0) * 16, from = row0 * DP + (DP == 128 ? c ^ row0 : c) * 16;  // in eight rows
        const uint32_t full = base + L::oVFull + 8 * team;
        int g = 0;                             // V tiles of the cache so far
        uint32_t v_phase = 0, v_used = 0;      // of new tokens' copies; one is in flight
        auto convert = [&](char* place, int gi, int have) {
            const char* const src = sm + L::oG + gi * L::kPart + 32 * team * DP;
            char* const to = place + (c >> 2) * (L::kHalf / 4);
            // Eight rows in one turn (rows of 64) or two: the second takes rows 2 on, the third bit of the swizzle's.
            constexpr int turns = DP / 16;
#pragma unroll
            for (int u = 0; u < turns; ++u) {
                const int eight = DP == 128 ? u >> 1 : u, flip = DP == 128 && (u & 1) ? 2 * 128 + 2 * 16 : 0;
                uint4 x = *reinterpret_cast<const uint4*>(src + eight * 8 * DP + (from ^ flip));
                if (have < kTile && 32 * team + 8 * eight + (row0 ^ (flip != 0 ? 2 : 0)) >= have) x = make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = half_of_e4m3(w[i / 2] >> 16 * (i & 1));
                *reinterpret_cast<uint4*>(to + eight * 1024 + (at0 ^ flip)) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(to + eight * 1024 + (at0 ^ flip ^ 16)) = make_uint4(y[4], y[5], y[6], y[7]);
            }
        };
        auto values = [&](int tile, int t) {
            const bool cached = t < w.x.ctx_tiles;
            const int gi = g % L::kG, rows = w.x.rows;
            if (cached && !warp_wait(base + L::oGFull + 8 * gi, (uint32_t)(g / L::kG & 1), stop)) return false;
            const uint32_t phase = (uint32_t)(tile & 1) ^ 1, half = 8 * (team >> 1);
            char* const place = sm + L::oV + team * L::kVBytes;
            if (!warp_wait(base + L::oVEmpty + half, phase, stop)) return false;
            // What was noted of new tokens before has been looked at when both halves of the tile before are done with.
            if (!cached && !warp_wait(base + L::oVEmpty + 8, phase, stop)) return false;
            if (cached) {
                convert(place, gi, w.x.ctx - t * kTile);
                ++g;
            } else if (rows > 32 * team) {
                // New tokens, at most 64, in their own type: rows past the end and rows that are not finite become 0, and
                // the latter are noted.
                {
                    v_used = 1;
                    if (lane == 0) bar_expect(full, (uint32_t)(L::kHalves * S.vbox) * 128u);
                    __syncwarp();
                    if (lane < L::kHalves) copy_box(smem_addr(place) + lane * (L::kHalf / 4), &M.v, 64 * lane, w.h, 32 * team, w.b, full);
                    if (!warp_wait(full, v_phase, stop)) return false;
                    v_phase ^= 1;
                    v_used = 0;
                    // a value is not finite where its exponent is all ones: one more there carries into the sign
                    constexpr uint32_t expo = BF16 ? 0x7f807f80u : 0x7c007c00u, one = BF16 ? 0x00800080u : 0x04000400u;
                    // lanes start at different chunks of their rows: no two in one bank
                    auto vector = [&](int c) { return reinterpret_cast<uint4*>(place + (c >> 3) * (L::kHalf / 4) + lane * 128 + ((c + lane) & 7) * 16); };
                    uint32_t hit = 0;
#pragma unroll 1
                    for (int c = 0; c < 8 * L::kHalves; ++c) {
                        const uint4 x = *vector(c);
                        hit |= ((x.x & expo) + one) | ((x.y & expo) + one) | ((x.z & expo) + one) | ((x.w & expo) + one);
                    }
                    const bool clear = 32 * team + lane >= rows, odd = !clear && (hit & 0x80008000u) != 0;
                    if (clear || odd)
#pragma unroll 1
                        for (int c = 0; c < 8 * L::kHalves; ++c) *vector(c) = make_uint4(0, 0, 0, 0);
                    const uint32_t word = __ballot_sync(0xffffffffu, odd);
                    if (lane == 0) bad[team] = word;
                }
            } else {
                for (int e = lane; e < L::kVBytes / 16; e += 32) *reinterpret_cast<uint4*>(place + 16 * e) = make_uint4(0, 0, 0, 0);
                if (lane == 0 && team < 2) bad[team] = 0;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                if (cached) bar_arrive(base + L::oGEmpty + 8 * gi);
                if (!cached && team < 2) bar_arrive(base + L::oLook + 8 * ((t - w.t0) & 1));
                bar_arrive(base + L::oVReady + half);
            }
            return true;
        };
        // Row `me` of the item's Q in parts of 8 bits: q = factor (p0 + p1 (+ p2)), each part the rounding of what the
        // parts before it leave, so that together they hold 9 (14) bits of an element, or 2^-18 of the row's largest where
        // that is more: bfloat16 has 8, float16 11.  A row that is not finite gets the factor NaN.
        auto split = [&](int seg) {
            const int qi = seg % L::kQB;
            if (!warp_wait(base + L::oQFull + 8 * qi, (uint32_t)(seg / L::kQB & 1), stop)) return false;
            if (!warp_wait(base + L::oFactorRead + 8 * qi, (uint32_t)(seg / L::kQB & 1) ^ 1, stop)) return false;
            // (No phase of the two is left out, and none passes by: Q's place is free once these warps have been here.)
            if (w.t0 >= w.x.ctx_tiles) {
                if (lane == 0) bar_arrive(base + L::oQEmpty + 8 * qi);
                return true;
            }
            const char* const raw = sm + qi * L::kBytes + me * 128;
            auto load = [&](int i, float* f) {  // elements 8 i .. 8 i + 7
                const uint4 v = *reinterpret_cast<const uint4*>(raw + (i >> 3) * L::kHalf + ((i & 7) ^ (me & 7)) * 16);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 y = BF16 ? make_float2(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xffff0000u)) : halves(u[e]);
                    f[2 * e] = y.x;
                    f[2 * e + 1] = y.y;
                }
            };
            float top = 0.0f;
            bool finite = true;
#pragma unroll 4
            for (int i = 0; i < DP / 8; ++i) {
                float f[8];
                load(i, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    top = fmaxf(top, fabsf(f[e]));
                    finite = finite && fabsf(f[e]) <= 3.4028234e38f;
                }
            }
            const float scale = scale_for(finite ? top : 0.0f), inv = 1.0f / scale;
            char* const parts = sm + L::oParts + qi * L::kParts * L::kPart + me * DP;
#pragma unroll 1
            for (int i = 0; i < DP / 8; ++i) {
                float f[8];
                load(i, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = finite ? f[e] * inv : 0.0f;
                const int at = 16 * (DP == 128 ? i / 2 ^ (me & 7) : i / 2 ^ (me >> 1 & 3)) + 8 * (i & 1);
#pragma unroll
                for (int part = 0; part < L::kParts; ++part) {
                    uint32_t y[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        y[e] = to_e4m3(f[4 * e], f[4 * e + 1]) | to_e4m3(f[4 * e + 2], f[4 * e + 3]) << 16;
                        if (part + 1 < L::kParts) {
                            float h[4];
                            from_e4m3x4(y[e], h);
#pragma unroll
                            for (int k = 0; k < 4; ++k) f[4 * e + k] -= h[k];
                        }
                    }
                    *reinterpret_cast<uint2*>(parts + part * L::kPart + at) = make_uint2(y[0], y[1]);
                }
            }
            reinterpret_cast<float*>(sm + L::oFactor)[qi * kTile + me] = finite ? scale : NAN;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) {
                bar_arrive(base + L::oPartsReady + 8 * qi);
                bar_arrive(base + L::oQEmpty + 8 * qi);
            }
            return true;
        };
        int i = 0;
        bool ok = true;
        for (int seg = 0; ok && w.left > 0; ++seg) {
            ok = split(seg);
            for (int t = w.t0; ok && t < w.t1; ++t, ++i) ok = values(i, t);
            __syncwarp();
            if (lane == 0) w.next(A, S, plan, near);
            __syncwarp();
        }
        if (!ok && v_used != 0) {
            // Leave no copy in flight.
            const long long t0 = clock64();
            while (!bar_try(full, v_phase) && clock64() - t0 < kWaitClocks) {}
        }
    }

    // ---- Parts are written: raise the flag, join what was cut. ----
    tmem_before();
    __syncthreads();
    // The joins run with equal shares of the registers again.  (Behind the barrier: a warp without work would else take back
    // what it gave before the softmax warps have it, and one of them would wait for registers for ever.)
    if (warp < kCopyWarp)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    else
        asm volatile("setmaxnreg.inc.sync.aligned.u32 80;");
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

template <int DP, bool BF16>
int launch(const Attend& A, const Shape& S, const Maps& M, void* scratch, cudaStream_t s)
{
    using L = Lay<DP, BF16>;
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CLK_ECUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit) || dev > 63) {
        if (cudaFuncSetAttribute(k_attend_tree8<DP, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal) != cudaSuccess)
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
    return cuda_status(cudaLaunchKernelEx(&cfg, k_attend_tree8<DP, BF16>, M, A, S, scratch));
}

}  // namespace

int attend_tree8_launch(const Attend& A, const Shape& S, const Maps& M, void* scratch, cudaStream_t s)
{
    const bool bf = A.dtype == CLK_DTYPE_BF16;
    if (A.dim > 64) return bf ? launch<128, true>(A, S, M, scratch, s) : launch<128, false>(A, S, M, scratch, s);
    return bf ? launch<64, true>(A, S, M, scratch, s) : launch<64, false>(A, S, M, scratch, s);
}

}  // namespace clk
