// Attention of new tokens over a paged cache: the general kernel, for every
// type, head count and stride, and the entry points.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "clk.h"
#include "clk_attend.h"
#include "clk_cache.h"
#include "clk_eight.cuh"
#include "clk_host.h"

namespace clk {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;
constexpr int kRows = 32;  // (token, head) rows of a CTA, four a warp
constexpr int kKeys = 64;  // keys of a tile, two a lane
constexpr int kWays = 8;   // CTAs of a cluster at most

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

// Four elements as they are loaded, and as float32.  (Converted where they are
// stored: a conversion beside its load would wait for it before the next.)
// vec: they lie whole in one aligned vector; else `left` of them are there.
__device__ __forceinline__ float4 take4(const float* p, int left, bool vec)
{
    if (vec) return *reinterpret_cast<const float4*>(p);
    return make_float4(p[0], left > 1 ? p[1] : 0.0f, left > 2 ? p[2] : 0.0f, left > 3 ? p[3] : 0.0f);
}
template <typename T>
__device__ __forceinline__ uint2 take4(const T* t, int left, bool vec)
{
    if (vec) return *reinterpret_cast<const uint2*>(t);
    const unsigned short* const p = reinterpret_cast<const unsigned short*>(t);
    const uint32_t a = p[0], b = left > 1 ? p[1] : 0, c = left > 2 ? p[2] : 0, d = left > 3 ? p[3] : 0;
    return make_uint2(a | b << 16, c | d << 16);
}
template <typename T>
struct Four {
    using type = uint2;
};
template <>
struct Four<float> {
    using type = float4;
};
template <typename T>
__device__ __forceinline__ float one(uint32_t bits);
template <>
__device__ __forceinline__ float one<__nv_bfloat16>(uint32_t bits) { return __uint_as_float(bits << 16); }
template <>
__device__ __forceinline__ float one<__half>(uint32_t bits) { return __half2float(__ushort_as_half((unsigned short)bits)); }
template <typename T>
__device__ __forceinline__ float4 to_f4(uint2 x)
{
    return make_float4(one<T>(x.x & 0xffffu), one<T>(x.x >> 16), one<T>(x.y & 0xffffu), one<T>(x.y >> 16));
}
template <typename T>
__device__ __forceinline__ float4 to_f4(float4 x) { return x; }

// Four codes of 8 bits, in the place of four elements, and the elements that they stand for, in float32 (a 16-bit type
// need not hold them: rows at the top of float16's range stand for more than its largest).
template <typename F>
__device__ __forceinline__ F take4_codes(const uint8_t* p, int left, bool vec)
{
    uint32_t w;
    if (vec)
        w = *reinterpret_cast<const uint32_t*>(p);
    else
        w = p[0] | (left > 1 ? p[1] : 0u) << 8 | (left > 2 ? p[2] : 0u) << 16 | (left > 3 ? p[3] : 0u) << 24;
    F x{};
    reinterpret_cast<uint32_t&>(x.x) = w;
    return x;
}
template <typename F>
__device__ __forceinline__ float4 of_codes(F x, float scale)
{
    float f[4];
    from_e4m3x4(reinterpret_cast<const uint32_t&>(x.x), f);
    return make_float4(f[0] * scale, f[1] * scale, f[2] * scale, f[3] * scale);
}

// How a call is cut: a CTA's rows are `tok` tokens x `hp` heads of one K/V
// head's group, a cluster of `ways` CTAs takes every ways-th tile of its keys.
struct Rows {
    int32_t tok, hp, head_blocks, ways;
    bool vec;  // K and V rows start on whole vectors of four elements
};

// NC columns of 32 elements a row.  Shared memory, in floats: K rows are four
// apart from a multiple of 32, so that the lanes' vectors (a key each) miss
// one another's banks.
template <int NC>
struct Sizes {
    static constexpr int kK = NC * 32 + 4, kV = NC * 32, kQ = NC * 32;
    static constexpr int kAtV = kKeys * kK, kAtQ = kAtV + kKeys * kV, kAtP = kAtQ + kRows * kQ;
    static constexpr int kTotal = (kAtP + kRows * kKeys) * 4;  // bytes
};

// The general kernel: out = softmax(scale q K^T) V with the running maximum
// and sum of the softmax, one pass over K and V for 32 rows at a time.
//
// A tile of 64 keys is brought to float32 in shared memory; a warp owns four
// rows through scores, softmax and values: a lane scores two keys against
// them (12 shared-memory passes for 32 multiply-adds) and then holds one of
// every 32 columns of their results.  With 16 rows or fewer the warps without
// rows take shares of the tile's keys (64 single tokens over 2,000 rows of 256:
// 765 us, 1,074 without), and a cluster's CTAs take every ways-th tile; their
// maxima, sums and results are joined in shared memory, in the order of
// warps and ranks, so that a result does not depend on timing.
//
// Everything is float32, products too (tensor cores would round float32
// inputs to 11 bits).  With many rows it is bound by the multiply-adds and
// the shared-memory reads beside them, with few by a tile's latency.
// Measured in float32, heads 32/8 of 128, replayed from a graph: one token over
// 2,048 rows 23 us; 8 requests of 16 nodes over 2,000 rows 237 us; a prompt of
// 1,000 tokens 522 us (16 TFLOP/s of the causal half).
template <typename T, int NC, bool EIGHT>
__device__ __forceinline__ void attend_rows(const Attend& A, const Rows& G, int b, int64_t t0, uint32_t rank)
{
    using Z = Sizes<NC>;
    extern __shared__ __align__(16) float sm[];
    __shared__ int64_t src[2][kKeys];     // offset in the pool, -2 - i for new token i, -1 for none
    __shared__ float stats[kRows][2];
    __shared__ float scales[2][2][EIGHT ? kKeys : 1];  // of K's and V's cached rows
    float *const sk = sm, *const sv = sm + Z::kAtV, *const sq = sm + Z::kAtQ;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kh = blockIdx.y / G.head_blocks, h0 = kh * A.group + (blockIdx.y - kh * G.head_blocks) * G.hp;
    const int hp = min(G.hp, (kh + 1) * A.group - h0);
    const bool prompt = A.off != nullptr;
    const Request R = attend_request(A, b, false);
    // (the whole cluster leaves, or none of it)
    if (t0 < 0 || (prompt && t0 >= R.rows)) return;
    const int64_t row0 = (prompt ? R.base : (int64_t)b * A.N) + t0;
    const int used = (int)min((int64_t)G.tok, (prompt ? R.rows : A.N) - t0) * hp;  // rows to write
    const int have = (int)max((int64_t)0, min((int64_t)G.tok, R.rows - t0)) * hp;  // those of real tokens
    auto put = [&](int r, int d, float x) {
        static_cast<T*>(A.out)[((row0 + r / hp) * A.q_heads + h0 + r % hp) * A.dim + d] = from_f<T>(x);
    };
    if (rank == 0)  // past the tree
        for (int r = have + warp; r < used; r += kThreads / 32)
            for (int d = lane; d < A.dim; d += 32) put(r, d, 0.0f);
    if (have == 0) return;
    const int64_t q0 = prompt ? row0 * A.q_row : b * A.q_req + t0 * A.q_row;
    const int64_t k0 = (prompt ? R.base * A.k_row : b * A.k_req) + kh * A.k_head;
    const int64_t v0 = (prompt ? R.base * A.v_row : b * A.v_req) + kh * A.v_head;
    for (int i = tid; i < kRows * Z::kQ; i += kThreads) {
        const int r = i / Z::kQ, d = i % Z::kQ;
        sq[i] = r < have && d < A.dim ? to_f(static_cast<const T*>(A.q)[q0 + (r / hp) * A.q_row + (h0 + r % hp) * A.q_head + d]) : 0.0f;
    }

    // Warps per four rows: all eight work whatever the rows in use, sharing a
    // tile's keys.  A lane has two keys of 64, one of 32, or a share of the
    // elements of one of 16 or 8.
    const int quads = (have + 3) / 4, share = quads > 4 ? 1 : quads > 2 ? 2 : quads > 1 ? 4 : 8;
    const int quad = warp / share, n_keys = kKeys / share, key0 = (warp - quad * share) * n_keys;
    const int key = lane & (n_keys - 1), slice = share > 1 ? lane / n_keys : 0, slices = share > 1 ? 32 / n_keys : 1;

    // What the warp's rows see of the new tokens: a mask (tree), or tokens up to their own.
    unsigned long long near[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = 4 * quad + q;
        // (rows past the block see everything and are not written)
        near[q] = r >= have ? (prompt ? ~0ull >> 1 : ~0ull)
                  : prompt  ? (unsigned long long)(t0 + r / hp)
                            : (unsigned long long)A.mask[row0 + r / hp];
    }
    const int64_t fresh = prompt ? t0 + have / hp : R.rows;
    const int64_t keys = R.ctx + fresh, all = R.ctx + (prompt ? t0 + 1 : 0);  // keys below `all` are seen by every row
    // (with 8 bits a cached row's scales are put at place `at` beside it)
    auto locate = [&](int64_t j, int at) -> int64_t {
        if (j >= keys) return -1;
        if (j >= R.ctx) return -2 - (j - R.ctx);
        const int32_t page = A.C.table[(int64_t)R.slot * A.C.max_pages + (j >> A.C.shift)];
        if (page >= 0 && page < A.C.num_pages) {
            const int line = (int)(j & (A.C.page_tokens() - 1));
            if (EIGHT) {
                const int64_t i = page * A.scale_page + kh * A.scale_head + (line >> A.scale_shift) * A.scale_block;
                scales[at][0][threadIdx.x] = A.ks[i];
                scales[at][1][threadIdx.x] = A.vs[i];
            }
            return page * A.page_stride + kh * A.head_stride + line * A.tok_stride;
        }
        latch(A.C.status, CLK_EINVAL, R.slot);
        return -1;
    };

    float m[4], l[4], acc[4][NC];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        m[q] = -INFINITY;
        l[q] = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[q][c] = 0.0f;
    }
    const int64_t step = (int64_t)G.ways * kKeys;
    const bool active = 4 * quad < have;
    int cur = 0;
    if (tid < kKeys) src[0][tid] = locate((int64_t)rank * kKeys + tid, 0);
    for (int64_t j0 = (int64_t)rank * kKeys; j0 < keys; j0 += step, cur ^= 1) {
        __syncthreads();  // the last tile is done with, this one's places are known
        if (tid < kKeys) src[cur ^ 1][tid] = locate(j0 + step + tid, cur ^ 1);
        constexpr int kLanes = NC >= 4 ? 32 : NC * 8;        // lanes a row's vectors take
        constexpr int kPass = NC * 8 * kKeys / kThreads;     // vectors a lane takes of K, and of V
        constexpr int kOnce = kPass < 8 ? kPass : 8;
#pragma unroll 1
        for (int i0 = 0; i0 < kPass; i0 += kOnce) {
            typename Four<T>::type kk[kOnce], vv[kOnce];
#pragma unroll
            for (int u = 0; u < kOnce; ++u) {
                const int i = i0 + u;
                const int r = warp * (kKeys / 8) + (NC == 8 ? i >> 1 : i * (32 / kLanes) + lane / kLanes);
                const int x = 4 * (NC == 8 ? lane + 32 * (i & 1) : lane % kLanes);
                const int64_t o = src[cur][r];
                kk[u] = vv[u] = typename Four<T>::type{};
                if (EIGHT && o >= 0) {
                    if (x < A.dim) {
                        kk[u] = take4_codes<typename Four<T>::type>(static_cast<const uint8_t*>(A.kc) + o + x, A.dim - x, G.vec);
                        vv[u] = take4_codes<typename Four<T>::type>(static_cast<const uint8_t*>(A.vc) + o + x, A.dim - x, G.vec);
                    }
                } else if (o != -1 && x < A.dim) {
                    const T* const pk = o >= 0 ? static_cast<const T*>(A.kc) + o : static_cast<const T*>(A.k) + k0 + (-2 - o) * A.k_row;
                    const T* const pv = o >= 0 ? static_cast<const T*>(A.vc) + o : static_cast<const T*>(A.v) + v0 + (-2 - o) * A.v_row;
                    kk[u] = take4(pk + x, A.dim - x, G.vec);
                    vv[u] = take4(pv + x, A.dim - x, G.vec);
                }
            }
#pragma unroll
            for (int u = 0; u < kOnce; ++u) {
                const int i = i0 + u;
                const int r = warp * (kKeys / 8) + (NC == 8 ? i >> 1 : i * (32 / kLanes) + lane / kLanes);
                const int x = 4 * (NC == 8 ? lane + 32 * (i & 1) : lane % kLanes);
                const bool codes = EIGHT && src[cur][r] >= 0;
                *reinterpret_cast<float4*>(sk + r * Z::kK + x) = codes ? of_codes(kk[u], scales[cur][0][EIGHT ? r : 0]) : to_f4<T>(kk[u]);
                *reinterpret_cast<float4*>(sv + r * Z::kV + x) = codes ? of_codes(vv[u], scales[cur][1][EIGHT ? r : 0]) : to_f4<T>(vv[u]);
            }
        }
        __syncthreads();
        if (!active) continue;

        float s[4][2] = {};
        const float4 *const k4 = reinterpret_cast<const float4*>(sk + (key0 + key) * Z::kK);
        const float4 *const q4 = reinterpret_cast<const float4*>(sq + 4 * quad * Z::kQ);
        if (share == 1) {
#pragma unroll 4
            for (int d = 0; d < (A.dim + 3) / 4; ++d) {
                const float4 a = k4[d], c = k4[32 * (Z::kK / 4) + d];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 y = q4[q * (Z::kQ / 4) + d];
                    s[q][0] = fmaf(y.w, a.w, fmaf(y.z, a.z, fmaf(y.y, a.y, fmaf(y.x, a.x, s[q][0]))));
                    s[q][1] = fmaf(y.w, c.w, fmaf(y.z, c.z, fmaf(y.y, c.y, fmaf(y.x, c.x, s[q][1]))));
                }
            }
        } else {
#pragma unroll 4
            for (int d = slice; d < (A.dim + 3) / 4; d += slices) {
                const float4 a = k4[d];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 y = q4[q * (Z::kQ / 4) + d];
                    s[q][0] = fmaf(y.w, a.w, fmaf(y.z, a.z, fmaf(y.y, a.y, fmaf(y.x, a.x, s[q][0]))));
                }
            }
            for (int d = n_keys; d < 32; d <<= 1)
#pragma unroll
                for (int q = 0; q < 4; ++q) s[q][0] += __shfl_xor_sync(0xffffffffu, s[q][0], d);
        }
        uint32_t seen = 0;  // bit 2q + e; a key's first slice sees it
        const uint32_t full = share == 1 ? 0xffu : slice == 0 ? 0x55u : 0u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int k = key0 + key + 32 * e;
            const bool there = (full >> e & 1) != 0 && src[cur][k & (kKeys - 1)] != -1;
            const int64_t i = j0 + k - R.ctx;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                bool see = there;
                if (i >= 0) see = see && (prompt ? i <= (int64_t)near[q] : (bool)((near[q] >> (i & 63)) & 1));
                if (see) seen |= 1u << (2 * q + e);
            }
        }
        const bool whole = j0 + kKeys <= all && __all_sync(0xffffffffu, seen == full);
        float p[4][2];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const bool see0 = seen >> (2 * q) & 1, see1 = seen >> (2 * q + 1) & 1;
            s[q][0] = see0 ? s[q][0] * A.scale : -INFINITY;
            s[q][1] = see1 ? s[q][1] * A.scale : -INFINITY;
            float top = fmaxf(s[q][0], s[q][1]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(top, m[q]);
            const float ref = top == -INFINITY ? 0.0f : top, fix = expf(m[q] - ref);
            p[q][0] = see0 ? expf(s[q][0] - ref) : 0.0f;
            p[q][1] = see1 ? expf(s[q][1] - ref) : 0.0f;
            float sum = p[q][0] + p[q][1];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l[q] = l[q] * fix + sum;
            m[q] = top;
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[q][c] *= fix;
            if (!see0) p[q][0] = -1.0f;  // hidden: its value does not count, whatever it is
            if (!see1) p[q][1] = -1.0f;
        }
        float4* const sp = reinterpret_cast<float4*>(sm + Z::kAtP) + warp * kKeys;
        if (slice == 0) sp[key] = make_float4(p[0][0], p[1][0], p[2][0], p[3][0]);
        if (share == 1) sp[key + 32] = make_float4(p[0][1], p[1][1], p[2][1], p[3][1]);
        __syncwarp();
        const float* const val = sv + key0 * Z::kV + lane;
        if (whole) {
#pragma unroll 4
            for (int j = 0; j < n_keys; ++j) {
                const float4 w = sp[j];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float v = val[j * Z::kV + 32 * c];
                    acc[0][c] = fmaf(w.x, v, acc[0][c]);
                    acc[1][c] = fmaf(w.y, v, acc[1][c]);
                    acc[2][c] = fmaf(w.z, v, acc[2][c]);
                    acc[3][c] = fmaf(w.w, v, acc[3][c]);
                }
            }
        } else {
            const int n = (int)min((int64_t)n_keys, keys - j0 - key0);
            for (int j = 0; j < n; ++j) {
                const float4 w = sp[j];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const float v = val[j * Z::kV + 32 * c];
                    acc[0][c] = w.x < 0.0f ? acc[0][c] : fmaf(w.x, v, acc[0][c]);
                    acc[1][c] = w.y < 0.0f ? acc[1][c] : fmaf(w.y, v, acc[1][c]);
                    acc[2][c] = w.z < 0.0f ? acc[2][c] : fmaf(w.z, v, acc[2][c]);
                    acc[3][c] = w.w < 0.0f ? acc[3][c] : fmaf(w.w, v, acc[3][c]);
                }
            }
        }
    }
    if (G.ways == 1 && share == 1) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int c = 0; c < NC; ++c)
                if (4 * warp + q < have && lane + 32 * c < A.dim)
                    put(4 * warp + q, lane + 32 * c, l[q] == 0.0f ? 0.0f : acc[q][c] / l[q]);
        return;
    }
    __syncthreads();  // K's place takes the results, four rows a warp
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int r = 4 * warp + q;
        if (lane == 0) {
            stats[r][0] = m[q];
            stats[r][1] = l[q];
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) sk[r * Z::kV + lane + 32 * c] = acc[q][c];
    }
    // Row r's part of warp quad * share + i lies at 4 * (that warp) + r % 4; they
    // are joined in the first one's place.
    auto place = [&](int r) { return 4 * share * (r >> 2) + (r & 3); };
    if (share > 1) {
        __syncthreads();
        for (int r = warp; r < have; r += kThreads / 32) {
            const int at = place(r);
            float top = -INFINITY, sum = 0.0f, x[NC] = {};
            for (int i = 0; i < share; ++i) top = fmaxf(top, stats[at + 4 * i][0]);
            const float ref = top == -INFINITY ? 0.0f : top;
            for (int i = 0; i < share; ++i) {
                const float f = expf(stats[at + 4 * i][0] - ref);
                sum += stats[at + 4 * i][1] * f;
#pragma unroll
                for (int c = 0; c < NC; ++c) x[c] += sk[(at + 4 * i) * Z::kV + lane + 32 * c] * f;
            }
            __syncwarp();
            if (lane == 0) {
                stats[at][0] = top;
                stats[at][1] = sum;
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                if (G.ways > 1)
                    sk[at * Z::kV + lane + 32 * c] = x[c];
                else if (lane + 32 * c < A.dim)
                    put(r, lane + 32 * c, sum == 0.0f ? 0.0f : x[c] / sum);
            }
        }
        if (G.ways == 1) return;
    }
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    cluster.sync();
    for (int r = (int)rank + G.ways * warp; r < have; r += G.ways * (kThreads / 32)) {
        const int at = place(r);
        float pm[kWays], pl[kWays], top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
            const float* const st = cluster.map_shared_rank(&stats[at][0], w < G.ways ? w : 0);
            pm[w] = w < G.ways ? st[0] : -INFINITY;
            pl[w] = w < G.ways ? st[1] : 0.0f;
            top = fmaxf(top, pm[w]);
        }
        if (top == -INFINITY) top = 0.0f;
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
            pm[w] = expf(pm[w] - top);
            sum += pl[w] * pm[w];
        }
        for (int d = lane; d < A.dim; d += 32) {
            float x = 0.0f;
#pragma unroll
            for (int w = 0; w < kWays; ++w)
                if (w < G.ways) x += cluster.map_shared_rank(sk, w)[at * Z::kV + d] * pm[w];
            put(r, d, sum == 0.0f ? 0.0f : x / sum);
        }
    }
    cluster.sync();  // no CTA ends while its results are read
}

// A cluster's rows: those of tokens t0 .. t0 + tok - 1 of request b, by its
// place in the grid.
template <typename T, int NC, bool EIGHT>
__global__ void __launch_bounds__(kThreads, 1) k_attend_rows(Attend A, Rows G)
{
    const int tid = threadIdx.x;
    const uint32_t item = blockIdx.x / G.ways, rank = blockIdx.x - item * G.ways;
    if (blockIdx.x == 0 && blockIdx.y == 0)  // what is wrong with a request is reported once
        for (int i = tid; i < A.B; i += kThreads) attend_request(A, i, true);
    // Request b's blocks begin at off[b] / tok + b: never fewer than it needs, and all within the grid.  With offsets
    // that rise an item is one request's at most; where one falls, several good requests may have it.
    __shared__ int first;
    bool falls;
    int b = -1;
    do {
        int64_t t0;
        falls = false;
        if (A.off == nullptr) {
            const int per = (A.N + G.tok - 1) / G.tok;
            b = (int)(item / per);
            t0 = (int64_t)(item - b * per) * G.tok;
        } else {
            if (tid == 0) first = A.B;
            __syncthreads();
            int mine = A.B;
            for (int i = b + 1 + tid; i < A.B; i += kThreads) {
                const int64_t lo = A.off[i], hi = A.off[i + 1];
                falls |= hi < lo;
                if (lo < 0 || hi <= lo || hi > A.T || mine < A.B) continue;
                const uint32_t at = (uint32_t)lo / G.tok + i, blocks = ((uint32_t)(hi - lo) + G.tok - 1) / G.tok;
                if (item >= at && item - at < blocks) mine = i;
            }
            if (mine < A.B) atomicMin(&first, mine);
            falls = __syncthreads_or(falls);
            b = first;
            if (b == A.B) return;
            t0 = (int64_t)(item - (uint32_t)A.off[b] / G.tok - b) * G.tok;
        }
        attend_rows<T, NC, EIGHT>(A, G, b, t0, rank);
        if (falls) __syncthreads();  // shared memory is used again
    } while (falls);
}

template <typename T, int NC, bool EIGHT>
int launch_rows(const Attend& A, const Rows& G, int64_t items, cudaStream_t s)
{
    constexpr int kBytes = Sizes<NC>::kTotal;
    static std::atomic<unsigned long long> ready{0};  // devices whose limit is raised
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return CLK_ECUDA;
    const unsigned long long bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit) || dev > 63) {
        if (cudaFuncSetAttribute(k_attend_rows<T, NC, EIGHT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes) != cudaSuccess)
            return CLK_ECUDA;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * G.ways), (unsigned)(A.kv_heads * G.head_blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)G.ways;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, k_attend_rows<T, NC, EIGHT>, A, G));
}

template <typename T>
int launch_general(const Attend& A, cudaStream_t s)
{
    Rows G;
    G.hp = A.group < kRows ? A.group : kRows;
    G.tok = A.group < kRows ? kRows / A.group : 1;
    G.head_blocks = (A.group + G.hp - 1) / G.hp;
    const int64_t items = A.off != nullptr ? A.T / G.tok + A.B : (int64_t)A.B * ((A.N + G.tok - 1) / G.tok);
    // Keys are shared while that leaves no more than 1.5 CTAs per SM.  Float32
    // rows of 256, 2,000 of them, shared by one, two, four and eight: 8 requests
    // of 8 nodes, 64 CTAs, 407, 218, 239 and 301 us; of 16 nodes, 128 CTAs, 406,
    // 429, 358 and 499.
    G.ways = kWays;
    const int64_t most = num_sms() * 3 / 2;
    while (G.ways > 1 && items * A.kv_heads * G.head_blocks * G.ways > most) G.ways /= 2;
    int64_t odd = A.dim;
    for (int64_t x : {A.k_req, A.k_row, A.k_head, A.v_req, A.v_row, A.v_head}) odd |= x;
    if (A.C.status != nullptr)
        for (int64_t x : {A.page_stride, A.head_stride, A.tok_stride}) odd |= x;
    G.vec = odd % 4 == 0;
    for (const void* x : {A.k, A.v}) G.vec = G.vec && aligned(x, 4 * sizeof(T));
    for (const void* x : {A.kc, A.vc}) G.vec = G.vec && aligned(x, A.ks != nullptr ? 4 : 4 * sizeof(T));
    if (A.ks != nullptr) {
        if (A.dim <= 64) return launch_rows<T, 2, true>(A, G, items, s);
        if (A.dim <= 128) return launch_rows<T, 4, true>(A, G, items, s);
        return launch_rows<T, 8, true>(A, G, items, s);
    }
    if (A.dim <= 64) return launch_rows<T, 2, false>(A, G, items, s);
    if (A.dim <= 128) return launch_rows<T, 4, false>(A, G, items, s);
    return launch_rows<T, 8, false>(A, G, items, s);
}

int launch_attend(const Attend& A, void* scratch, size_t bytes, cudaStream_t s)
{
    if (attend_mma_takes(A)) {
        if (scratch == nullptr || !aligned(scratch, 16) || bytes < attend_mma_scratch(A.q_heads, A.kv_heads, A.dim))
            return CLK_EINVAL;
        return attend_mma_launch(A, scratch, s);
    }
    switch (A.dtype) {
    case CLK_DTYPE_BF16: return launch_general<__nv_bfloat16>(A, s);
    case CLK_DTYPE_F16: return launch_general<__half>(A, s);
    default: return launch_general<float>(A, s);
    }
}

// Checks what both calls share and fills the common fields.
int fill_attend(Attend& A, const clk_attn* a, clk_cache* h, const int32_t* d_slots, const clk_pool* pool, const clk_scales* scales,
                int32_t layer, const int32_t* d_ctx, int32_t B)
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
        if (scales != nullptr ? check_pool8(pool, scales, h->dev.page_tokens()) != CLK_OK
                              : check_pool(pool) != CLK_OK || pool->dtype != a->dtype)
            return CLK_EINVAL;
        if (pool->heads != a->kv_heads || pool->dim != a->dim || layer < 0 || layer >= pool->planes / 2) return CLK_EINVAL;
        if (B > 0 && !ok_i32(d_slots)) return CLK_EINVAL;
        A.C = h->dev;
        A.slots = d_slots;
        A.ctx = d_ctx;
        const char* base = static_cast<const char*>(pool->d_base);
        const int64_t ps = pool_bytes(pool->dtype), kp = 2 * (int64_t)layer;
        A.kc = base + kp * pool->plane_stride * ps;
        A.vc = base + (kp + 1) * pool->plane_stride * ps;
        if (scales != nullptr) {
            A.ks = scales->d_base + kp * scales->plane_stride;
            A.vs = scales->d_base + (kp + 1) * scales->plane_stride;
            A.scale_page = scales->page_stride;
            A.scale_head = scales->head_stride;
            A.scale_block = scales->block_stride;
            while ((1 << A.scale_shift) < scales->tokens) ++A.scale_shift;
        }
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

extern "C" int clk_attend_status(const void* d_scratch, int32_t* dev_status, clk_stream_t s)
{
    if (d_scratch == nullptr || !aligned(d_scratch, 16) || dev_status == nullptr) return CLK_EINVAL;
    const cudaStream_t cs = (cudaStream_t)s;
    int32_t st = 0;
    if (cudaMemcpyAsync(&st, d_scratch, sizeof st, cudaMemcpyDeviceToHost, cs) != cudaSuccess) return CLK_ECUDA;
    if (cudaStreamSynchronize(cs) != cudaSuccess) return CLK_ECUDA;
    *dev_status = st;
    return CLK_OK;
}

namespace clk {
namespace {

int tree_call(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool, const clk_scales* scales, int32_t layer,
              const clk_attn* a, int32_t N, const int32_t* d_nodes, const int64_t* d_mask, const int32_t* d_ctx, void* d_scratch,
              size_t scratch_bytes, cudaStream_t s)
{
    if (h == nullptr) return CLK_ESTATE;
    Attend A;
    const int rc = fill_attend(A, a, h, d_slots, pool, scales, layer, d_ctx, B);
    if (rc != CLK_OK) return rc;
    if (N < 1 || N > CLK_TREE_MAX) return CLK_EINVAL;
    if (B == 0) return CLK_OK;
    if (!attn_pointers(a) || !ok_i32(d_nodes) || d_mask == nullptr || !aligned(d_mask, 8)) return CLK_EINVAL;
    A.nodes = d_nodes;
    A.mask = d_mask;
    A.N = N;
    return launch_attend(A, d_scratch, scratch_bytes, s);
}

int prompt_call(const clk_attn* a, const int64_t* d_off, int32_t B, int64_t T, clk_cache* h, const int32_t* d_slots,
                const clk_pool* pool, const clk_scales* scales, int32_t layer, const int32_t* d_ctx, void* d_scratch,
                size_t scratch_bytes, cudaStream_t s)
{
    Attend A;
    if (h == nullptr && d_ctx != nullptr) return CLK_EINVAL;
    const int rc = fill_attend(A, a, h, d_slots, pool, scales, layer, d_ctx, B);
    if (rc != CLK_OK) return rc;
    if (T < 0 || T > ((int64_t)1 << 30)) return CLK_EINVAL;
    if (B == 0 || T == 0) return CLK_OK;
    if (!attn_pointers(a) || d_off == nullptr || !aligned(d_off, 8)) return CLK_EINVAL;
    A.off = d_off;
    A.T = T;
    return launch_attend(A, d_scratch, scratch_bytes, s);
}

}  // namespace
}  // namespace clk

extern "C" int clk_tree_attend(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool, int32_t layer,
                               const clk_attn* a, int32_t N, const int32_t* d_nodes, const int64_t* d_mask,
                               const int32_t* d_ctx, void* d_scratch, size_t scratch_bytes, clk_stream_t s)
{
    return tree_call(h, d_slots, B, pool, nullptr, layer, a, N, d_nodes, d_mask, d_ctx, d_scratch, scratch_bytes, (cudaStream_t)s);
}

extern "C" int clk_tree_attend_scaled(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool,
                                      const clk_scales* scales, int32_t layer, const clk_attn* a, int32_t N,
                                      const int32_t* d_nodes, const int64_t* d_mask, const int32_t* d_ctx, void* d_scratch,
                                      size_t scratch_bytes, clk_stream_t s)
{
    if (h != nullptr && scales == nullptr) return CLK_EINVAL;
    return tree_call(h, d_slots, B, pool, scales, layer, a, N, d_nodes, d_mask, d_ctx, d_scratch, scratch_bytes, (cudaStream_t)s);
}

extern "C" int clk_prompt_attend(const clk_attn* a, const int64_t* d_off, int32_t B, int64_t T, clk_cache* h,
                                 const int32_t* d_slots, const clk_pool* pool, int32_t layer, const int32_t* d_ctx,
                                 void* d_scratch, size_t scratch_bytes, clk_stream_t s)
{
    return prompt_call(a, d_off, B, T, h, d_slots, pool, nullptr, layer, d_ctx, d_scratch, scratch_bytes, (cudaStream_t)s);
}

extern "C" int clk_prompt_attend_scaled(const clk_attn* a, const int64_t* d_off, int32_t B, int64_t T, clk_cache* h,
                                        const int32_t* d_slots, const clk_pool* pool, const clk_scales* scales, int32_t layer,
                                        const int32_t* d_ctx, void* d_scratch, size_t scratch_bytes, clk_stream_t s)
{
    if (h == nullptr) return CLK_ESTATE;
    if (scales == nullptr) return CLK_EINVAL;
    return prompt_call(a, d_off, B, T, h, d_slots, pool, scales, layer, d_ctx, d_scratch, scratch_bytes, (cudaStream_t)s);
}
