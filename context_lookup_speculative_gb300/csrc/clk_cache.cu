// Pages of the target's K/V cache: taking, filling, forking, freeing and
// compacting them.
//
// Which pages are free is a bit per page, so that the lowest free ones are
// found by a scan of num_pages / 8 bytes and what a call hands out depends
// on nothing but the pages in use: the counts of holders change by atomic
// additions, whose order leaves no trace.  The planning kernels run as one
// CTA (a prefix sum over the batch, one over the free bits); what moves rows
// runs as a grid over all of them.  All the row movement is bound by memory:
// every row is read once and written once, in vectors of up to 16 bytes.
//
// Measured, launches back to back (each waits for the one before it on the
// device, so that their starts overlap).  64 prompts of 200 to 2,000 tokens,
// 8 layers of 8 heads of 128 in 16 bits, taken in, half of them freed and the
// rest compacted: 853 us for 5.7 GB, 98% of the copy rate.  The end of a step
// for 64 such requests of 16 drafted tokens (free, fork, masks, accept, grow,
// append): 56 us, of which the fork's copy of the tails is 23 (20 at the copy
// rate) and the rest six launches' dependent loads; for one request 18 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <new>

#include "clk.h"
#include "clk_cache.h"
#include "clk_device.cuh"
#include "clk_host.h"

namespace clk {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kFailed = -2;  // req[b].y of a request that a plan leaves as it was

struct CacheLayout {
    size_t len, firm, refs, bits, table, req, list, total;
};

int cache_layout(int32_t max_slots, int32_t max_pages, int32_t num_pages, CacheLayout* out)
{
    if (max_slots < 1 || max_pages < 1 || num_pages < 1) return CLK_EINVAL;
    const int64_t most = (int64_t)1 << 30;
    if (max_slots > most || num_pages > most || (int64_t)max_slots * max_pages > most) return CLK_EINVAL;
    CacheLayout L;
    size_t off = align_up(64 * sizeof(int32_t), kAlign);
    L.len = off;
    off = align_up(off + (size_t)max_slots * sizeof(int32_t), kAlign);
    L.firm = off;
    off = align_up(off + (size_t)max_slots * sizeof(int32_t), kAlign);
    L.refs = off;
    off = align_up(off + (size_t)num_pages * sizeof(int32_t), kAlign);
    L.bits = off;
    off = align_up(off + ((size_t)num_pages + 127) / 128 * 16, kAlign);
    L.table = off;
    off = align_up(off + (size_t)max_slots * (size_t)max_pages * sizeof(int32_t), kAlign);
    L.req = off;
    off = align_up(off + (size_t)max_slots * sizeof(int2), kAlign);
    L.list = off;
    off = align_up(off + 3 * (size_t)num_pages * sizeof(int32_t) + 16, kAlign);
    L.total = off;
    *out = L;
    return CLK_OK;
}

__global__ void k_cache_reset(CacheDev C)
{
    const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = at; i < 64; i += step) C.status[i] = 0;
    for (int64_t i = at; i < C.max_slots; i += step) C.len[i] = C.firm[i] = 0;
    for (int64_t i = at; i < C.num_pages; i += step) C.refs[i] = 0;
    for (int64_t i = at; i < C.words(); i += step) {
        const int64_t left = C.num_pages - 32 * i;
        C.bits[i] = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
    }
    for (int64_t i = at; i < (int64_t)C.max_slots * C.max_pages; i += step) C.table[i] = -1;
}

// Exclusive sum over the CTA's 1024 threads, and the total.  `sm` holds 33
// ints; every thread of the CTA takes part.
__device__ __forceinline__ int block_scan(int v, int* sm, int* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int w = sm[lane];
        int z = w;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, z, d);
            if (lane >= d) z += y;
        }
        sm[lane] = z - w;
        if (lane == 31) sm[32] = z;
    }
    __syncthreads();
    const int before = sm[warp];
    *total = sm[32];
    __syncthreads();
    return before + x - v;
}

__device__ __forceinline__ bool slot_ok(const CacheDev& C, int32_t s) { return s >= 0 && s < C.max_slots; }

// Writes the lowest `want` free pages to `list`; returns how many there are
// (at most want).  Every thread of the CTA takes part.
__device__ int lowest_free(const CacheDev& C, int want, int32_t* list, int* sm)
{
    int found = 0;
    const uint4* bits = reinterpret_cast<const uint4*>(C.bits);
    const int vecs = C.words() / 4;
    for (int base = 0; base < vecs && found < want; base += kPlanThreads) {
        const int at = base + (int)threadIdx.x;
        const uint4 v = at < vecs ? bits[at] : make_uint4(0, 0, 0, 0);
        int total;
        int rank = found + block_scan(__popc(v.x) + __popc(v.y) + __popc(v.z) + __popc(v.w), sm, &total);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            for (uint32_t left = w[j]; left != 0 && rank < want; left &= left - 1, ++rank)
                list[rank] = 128 * at + 32 * j + __ffs((int)left) - 1;
        found += total;
    }
    __syncthreads();
    return found < want ? found : want;
}

__device__ __forceinline__ void take_page(const CacheDev& C, int32_t page)
{
    C.refs[page] = 1;
    atomicAnd(C.bits + (page >> 5), ~(1u << (page & 31)));
}

// Plans a call's pages, as one CTA.  FORK = false: clk_cache_grow's whole
// work.  FORK = true: clk_cache_fork's tail pages; req[b].y becomes the tail
// page, -1 without one, kFailed for a request that is left out, and req[b].x
// the tails' rows before it.
template <bool FORK>
__global__ void __launch_bounds__(kPlanThreads) k_cache_plan(CacheDev C, const int32_t* slots, const int32_t* dst,
                                                             const int32_t* count, int32_t B)
{
    chained();
    __shared__ int sm[33];
    __shared__ int2 near[kPlanThreads];
    __shared__ int32_t few[kPlanThreads];
    const int tid = threadIdx.x;
    const int32_t part = C.page_tokens() - 1;
    // Pages of each request: req = (those of the requests before it, its own or kFailed).
    int2* const req = B <= kPlanThreads ? near : C.req;
    int want = 0;
    int32_t firm = 0;  // FORK: the source's, fetched beside its length (of the thread's last request: a small batch's only one)
    for (int base = 0; base < B; base += kPlanThreads) {
        const int b = base + tid;
        int need = 0, state = kFailed;
        if (b < B) {
            const int32_t s = slots[b];
            int err = CLK_OK, who = s;
            if (!slot_ok(C, s)) {
                err = CLK_EINVAL;
                who = b;
            } else if (FORK) {
                const int32_t d = dst[b];
                firm = C.firm[s];
                if (!slot_ok(C, d)) {
                    err = CLK_EINVAL;
                    who = b;
                } else if (d == s || C.len[d] != 0) {
                    err = CLK_EINVAL;
                    who = d;
                } else {
                    need = (C.len[s] & part) != 0;
                }
            } else {
                const int64_t old = C.len[s], now = old + (int64_t)count[b];
                if (count[b] < 0)
                    err = CLK_EINVAL;
                else if (now > ((int64_t)C.max_pages << C.shift))
                    err = CLK_ECAPACITY;
                else
                    need = C.pages(now) - C.pages(old);
                // an append that follows in spite of this writes nothing
                if (err != CLK_OK) C.firm[s] = (int32_t)old;
            }
            if (err != CLK_OK)
                latch(C.status, err, who);
            else
                state = need;
        }
        int total;
        const int before = block_scan(need, sm, &total);
        if (b < B) req[b] = make_int2(want + before, state);
        // Sums stay far below 2^31: a request's pages are at most max_pages, and max_slots * max_pages <= 2^30.
        want += total;
    }
    __syncthreads();
    int32_t* const list = want <= kPlanThreads ? few : C.list;
    const int have = want > 0 ? lowest_free(C, want < C.num_pages ? want : C.num_pages, list, sm) : 0;
    if (!FORK) {
        // Rank r's page goes to the last request whose pages start at or before r.
        for (int r = tid; r < have; r += kPlanThreads) {
            int lo = 0, hi = B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (req[mid].x <= r)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int2 q = req[lo];
            if (q.x + q.y > have) continue;
            const int32_t s = slots[lo], page = list[r];
            C.table[(int64_t)s * C.max_pages + C.pages(C.len[s]) + (r - q.x)] = page;
            take_page(C, page);
        }
        __syncthreads();
    }
    int rows = 0;  // FORK: rows that the copying kernel moves, request after request
    for (int base = 0; base < B; base += kPlanThreads) {
        const int b = base + tid;
        int tail = kFailed, own = 0;
        if (b < B) {
            const int2 q = req[b];
            if (q.y >= 0) {
                if (q.y > 0 && q.x + q.y > have) {
                    latch(C.status, CLK_ECAPACITY, FORK ? dst[b] : slots[b]);
                    if (!FORK) C.firm[slots[b]] = C.len[slots[b]];
                } else if (!FORK) {
                    C.len[slots[b]] += count[b];
                } else {
                    const int32_t n = C.len[slots[b]];
                    // The whole pages are shared from here on (forks of one source raise it to one value).
                    const int32_t shared = max(B <= kPlanThreads ? firm : C.firm[slots[b]], n & ~part);
                    C.firm[slots[b]] = C.firm[dst[b]] = shared;
                    tail = -1;
                    if (q.y > 0) {
                        tail = list[q.x];
                        take_page(C, tail);
                        own = n & part;
                    }
                    C.len[dst[b]] = n;
                }
            }
        }
        if (FORK) {
            int total;
            const int before = block_scan(own, sm, &total);
            if (b < B) C.req[b] = make_int2(rows + before, tail);
            rows += total;
        }
    }
    if (FORK) {
        if (tid == 0) C.list[3 * (int64_t)C.num_pages + 2] = rows;
    }
}

__global__ void __launch_bounds__(kCopyThreads) k_cache_free(CacheDev C, const int32_t* slots, int32_t B)
{
    chained();
    const int b = blockIdx.x;
    const int32_t s = slots[b];
    if (!slot_ok(C, s)) {
        if (threadIdx.x == 0) latch(C.status, CLK_EINVAL, b);
        return;
    }
    const int held = C.held(C.len[s]);
    __syncthreads();  // every thread has the length before it is cleared
    for (int i = threadIdx.x; i < held; i += kCopyThreads) {
        // The exchange gives each entry up once, also where a slot is listed twice.
        const int32_t page = atomicExch(C.table + (int64_t)s * C.max_pages + i, -1);
        if (page >= 0 && page < C.num_pages && atomicSub(C.refs + page, 1) == 1)
            atomicOr(C.bits + (page >> 5), 1u << (page & 31));
    }
    if (threadIdx.x == 0) C.len[s] = C.firm[s] = 0;
}

// A pool in vectors of V: strides in vectors, and vectors per row.
template <typename V>
struct VecPool {
    V* base;
    int64_t plane, page, head, tok;
    int32_t planes, heads, row;
};

// Copies the first `rows` rows of page src to page dst in one plane; the
// CTA's threads take `row` vectors of as many rows at a time as they can,
// eight of them in flight.
template <typename V>
__device__ __forceinline__ void copy_page(const VecPool<V>& A, int64_t src, int64_t dst, int32_t rows, int32_t plane)
{
    constexpr int kFlight = 8;
    const int wide = A.row < kCopyThreads ? A.row : kCopyThreads;
    const int tall = kCopyThreads / wide;
    const int c0 = threadIdx.x % wide, t0 = threadIdx.x / wide;
    if (t0 >= tall) return;
    const int lines = A.heads * rows;
    V* const base = A.base + plane * A.plane;
    const int64_t from = src * A.page, to = dst * A.page;
    for (int i = t0; i < lines; i += kFlight * tall) {
        int64_t off[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const int line = i + u * tall;
            const int head = line / rows;
            off[u] = line < lines ? head * A.head + (int64_t)(line - head * rows) * A.tok : -1;
        }
        for (int c = c0; c < A.row; c += wide) {
            V x[kFlight];
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (off[u] >= 0) x[u] = base[from + off[u] + c];
#pragma unroll
            for (int u = 0; u < kFlight; ++u)
                if (off[u] >= 0) base[to + off[u] + c] = x[u];
        }
    }
}

// A CTA moves `group` rows in every head of planes p0 .. p1-1: their
// sources and places (in vectors, -1 for none) are found once, by as many
// threads, and lie in shared memory.
constexpr int kFewRows = 8, kMostRows = 32;

template <typename V, typename Plane>
__device__ __forceinline__ void move_rows(const int64_t* from, const int64_t* to, int group, const VecPool<V>& A,
                                          int64_t src_head, int p0, int p1, Plane plane_of)
{
    const int wide = A.row < kCopyThreads ? A.row : kCopyThreads;
    const int tall = kCopyThreads / wide;
    const int c0 = threadIdx.x % wide, t0 = threadIdx.x / wide;
    if (t0 >= tall) return;
    int live = group;  // rows past the last one that moves need no turn
    while (live > 0 && to[live - 1] < 0) --live;
    const int lines = live * A.heads;
    for (int plane = p0; plane < p1; ++plane) {
        const V* src;
        V* dst;
        plane_of(plane, src, dst);
        for (int i = t0; i < lines; i += 4 * tall) {
            // rows follow one another in a page, so the rows of one head go together
            int64_t a[4], z[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int line = i + u * tall;
                const int head = line / live, r = line - head * live;
                const bool take = line < lines && to[r] >= 0;
                a[u] = take ? from[r] + head * src_head : -1;
                z[u] = take ? to[r] + head * A.head : -1;
            }
            for (int c = c0; c < A.row; c += wide) {
                V x[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (z[u] >= 0) x[u] = src[a[u] + c];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (z[u] >= 0) dst[z[u] + c] = x[u];
            }
        }
    }
}

// Destination b shares the source's whole pages (the CTAs with blockIdx.y = 0
// write the tables) and its tail's rows are copied: the tails of all
// requests lie one after the other, `group` rows a CTA, so that tails of every
// length balance; blockIdx.y takes a share of the planes.  (Measured with shares
// for 4, 8 and 16 CTAs an SM: 23, 26 and 34 us. More CTAs find the same places.)
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) k_cache_fork(CacheDev C, const int32_t* src, const int32_t* dst, int32_t B,
                                                             VecPool<V> A, int32_t group)
{
    chained();
    __shared__ int64_t from[kMostRows], to[kMostRows];
    __shared__ int32_t before[kCopyThreads];
    const int rows = C.list[3 * (int64_t)C.num_pages + 2];
    const bool few = B <= kCopyThreads;
    if (few && threadIdx.x < B) before[threadIdx.x] = C.req[threadIdx.x].x;
    __syncthreads();
    const int64_t at = (int64_t)blockIdx.x * group + threadIdx.x;
    if (threadIdx.x < group) {
        int64_t a = -1, z = -1;
        if (at < rows) {
            // the last request whose rows start at or before this one
            int lo = 0, hi = B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((few ? before[mid] : C.req[mid].x) <= at)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int2 q = C.req[lo];
            const int32_t s = src[lo], whole = C.held(C.len[s]) - 1;
            const int64_t row = (at - q.x) * A.tok;
            a = C.table[(int64_t)s * C.max_pages + whole] * A.page + row;
            z = q.y * A.page + row;
        }
        from[threadIdx.x] = a;
        to[threadIdx.x] = z;
    }
    if (blockIdx.y == 0 && blockIdx.x < B) {
        const int b = blockIdx.x;
        const int32_t tail = C.req[b].y;
        if (tail != kFailed) {
            const int32_t whole = C.held(C.len[src[b]]) - (tail >= 0 ? 1 : 0);
            const int32_t* const have = C.table + (int64_t)src[b] * C.max_pages;
            int32_t* const row = C.table + (int64_t)dst[b] * C.max_pages;
            for (int i = threadIdx.x; i < whole; i += kCopyThreads) {
                const int32_t page = have[i];
                row[i] = page;
                atomicAdd(C.refs + page, 1);
            }
            if (threadIdx.x == 0 && tail >= 0) row[whole] = tail;
        }
    }
    __syncthreads();
    if ((int64_t)blockIdx.x * group >= rows) return;
    const int p0 = (int)((int64_t)A.planes * blockIdx.y / gridDim.y), p1 = (int)((int64_t)A.planes * (blockIdx.y + 1) / gridDim.y);
    move_rows(from, to, group, A, A.head, p0, p1, [&](int plane, const V*& s, V*& d) { s = d = A.base + plane * A.plane; });
}

// Rows of the new tokens into the pages; blockIdx.y takes a share of the planes.

// Whether n rows of a request with source rows base .. base + rows - 1 can go to the end of a slot's tokens, of which
// `room` follow the firm ones.
__device__ __forceinline__ bool append_ok(int32_t n, int32_t room, int64_t base, int64_t rows, int64_t total)
{
    return n >= 0 && n <= room && n <= rows && base >= 0 && base <= total - rows;
}

template <typename V>
struct VecSrc {
    const V *k, *v;
    int64_t layer, row, head;
};

template <typename V>
__global__ void __launch_bounds__(kCopyThreads) k_cache_append(CacheDev C, const int32_t* slots, int32_t B, VecPool<V> A,
                                                               int32_t layer0, int32_t planes, VecSrc<V> S, int64_t N, const int64_t* off,
                                                               const int32_t* path, const int32_t* count, int32_t group)
{
    chained();
    __shared__ int64_t from[kMostRows], to[kMostRows];
    const int64_t total = off != nullptr ? N : (int64_t)B * N;
    const int64_t first = (int64_t)blockIdx.x * group;
    __shared__ int64_t begin[kCopyThreads];
    const bool few = off != nullptr && B < kCopyThreads;
    if (few && threadIdx.x <= B) begin[threadIdx.x] = off[threadIdx.x];
    __syncthreads();
    const int64_t* const starts = few ? begin : off;
    if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) {
        // one CTA reports the requests that are left out
        for (int b = threadIdx.x; b < B; b += kCopyThreads) {
            const int32_t s = slots[b];
            const int64_t base = off != nullptr ? off[b] : b * N, rows = off != nullptr ? off[b + 1] - base : N;
            if (!slot_ok(C, s))
                latch(C.status, CLK_EINVAL, b);
            else if (!append_ok(count[b], C.len[s] - C.firm[s], base, rows, total))
                latch(C.status, CLK_EINVAL, s);
        }
    }
    // Where row i of request b comes from and goes to; both stay as they are for one that is not written.
    auto find = [&](int b, int64_t i, int64_t base, int64_t rows, int64_t& row, int64_t& place) {
        const int32_t s = slots[b], n = count[b];
        const int32_t len = slot_ok(C, s) ? C.len[s] : -1, room = slot_ok(C, s) ? len - C.firm[s] : -1;
        if (!append_ok(n, room, base, rows, total) || i >= n) return;
        const int64_t r = path != nullptr ? path[base + i] : i;
        const int32_t pos = len - n + (int32_t)i;
        const int32_t page = (pos >> C.shift) < C.max_pages ? C.table[(int64_t)s * C.max_pages + (pos >> C.shift)] : -1;
        if (r < 0 || r >= rows || page < 0 || page >= C.num_pages) {
            latch(C.status, CLK_EINVAL, s);
        } else {
            row = (base + r) * S.row;
            place = page * A.page + (int64_t)(pos & (C.page_tokens() - 1)) * A.tok;
        }
    };
    if (threadIdx.x < group) {
        const int64_t at = first + threadIdx.x;
        int64_t row = -1, place = -1;
        int b = -1;
        int64_t i = 0, rows = N, base = 0;
        if (at < total) {
            if (off == nullptr) {
                b = (int)(at / N);
                i = at - b * N;
                base = b * N;
            } else if (starts[0] <= at) {
                // the last request that starts at or before this row
                int lo = 0, hi = B - 1;
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (starts[mid] <= at)
                        lo = mid;
                    else
                        hi = mid - 1;
                }
                b = lo;
                base = starts[lo];
                i = at - base;
                rows = starts[lo + 1] - base;
            }
        }
        if (b >= 0) find(b, i, base, rows, row, place);
        from[threadIdx.x] = row;
        to[threadIdx.x] = place;
    }
    __syncthreads();
    const int p0 = (int)((int64_t)planes * blockIdx.y / gridDim.y), p1 = (int)((int64_t)planes * (blockIdx.y + 1) / gridDim.y);
    auto planes_of = [&](int plane, const V*& s, V*& d) {
        s = (plane & 1 ? S.v : S.k) + (plane >> 1) * S.layer;
        d = A.base + (2 * (int64_t)layer0 + plane) * A.plane;
    };
    move_rows(from, to, group, A, S.head, p0, p1, planes_of);
    if (off == nullptr || blockIdx.x != gridDim.x - 1) return;
    // The search above relies on offsets that do not fall.  Where one does, it misses rows of the requests around it:
    // the last CTAs write all good requests' rows, those that were found among them once more.
    bool falls = false;
    for (int b = threadIdx.x; b < B; b += kCopyThreads) falls |= starts[b + 1] < starts[b];
    if (!__syncthreads_or(falls)) return;
    for (int b = 0; b < B; ++b) {
        const int64_t base = starts[b], rows = starts[b + 1] - base;
        const int32_t s = slots[b], n = count[b];
        if (!slot_ok(C, s) || !append_ok(n, C.len[s] - C.firm[s], base, rows, total)) continue;
        for (int32_t i = 0; i < n; i += group) {
            __syncthreads();  // the rows before are written
            if (threadIdx.x < group) {
                int64_t row = -1, place = -1;
                find(b, (int64_t)i + threadIdx.x, base, rows, row, place);
                from[threadIdx.x] = row;
                to[threadIdx.x] = place;
            }
            __syncthreads();
            move_rows(from, to, group, A, S.head, p0, p1, planes_of);
        }
    }
}

// Entries of all tables up to which one CTA rewrites them.  Measured with and
// without, a cache's life as above in one layer: 5 prompts of up to 700 tokens (220
// entries) 24.3 and 25.3 us and a launch less for the host; 64 prompts of 2,000
// in 125 pages each 235 and 232.
constexpr int64_t kFewEntries = 2048;

// Compaction, step 2, for entry i of slot s: the table follows, and rank[hole]
// receives the rows that the moving page holds (holes are free, so their
// ranks are not in use).
__device__ __forceinline__ void follow(const CacheDev& C, int s, int i, int32_t n, int32_t live)
{
    if (i >= C.held(n)) return;
    int32_t* const rank = C.list + 2 * (int64_t)C.num_pages;
    int32_t* const entry = C.table + (int64_t)s * C.max_pages + i;
    const int32_t page = *entry;
    if (page < live || page >= C.num_pages) return;
    const int32_t to = C.list[rank[page]];
    *entry = to;
    const int32_t left = n - (i << C.shift);
    rank[to] = left < C.page_tokens() ? left : C.page_tokens();
}

// Compaction, step 1 (one CTA): with L pages in use, list[0] holds the free
// pages below L and list[1] those in use from L on, both ascending and
// equally many; list[2][page] is a moving page's place in list[1].  The free
// bits become what they are after the move.  With small tables (kFewEntries)
// step 2 is done here too, which spares a launch.
__global__ void __launch_bounds__(kPlanThreads) k_compact_plan(CacheDev C, int32_t* moved, bool tables)
{
    chained();
    __shared__ int sm[33];
    const int tid = threadIdx.x;
    const int words = C.words();
    int sum = 0;
    for (int w = tid; w < words; w += kPlanThreads) sum += __popc(C.bits[w]);
    int free_pages;
    block_scan(sum, sm, &free_pages);
    const int live = C.num_pages - free_pages;
    int32_t *const holes = C.list, *const movers = C.list + C.num_pages, *const rank = C.list + 2 * (int64_t)C.num_pages;
    int nh = 0, nm = 0;
    for (int base = 0; base < words; base += kPlanThreads) {
        const int w = base + tid;
        const int64_t p0 = 32 * (int64_t)w;
        uint32_t free_bits = 0, low = 0, all = 0;
        if (w < words) {
            free_bits = C.bits[w];
            const int64_t below = live - p0, valid = C.num_pages - p0;
            low = below >= 32 ? 0xffffffffu : below > 0 ? (1u << below) - 1u : 0u;
            all = valid >= 32 ? 0xffffffffu : valid > 0 ? (1u << valid) - 1u : 0u;
        }
        uint32_t h = free_bits & low, m = ~free_bits & all & ~low;
        int th, tm;
        int rh = nh + block_scan(__popc(h), sm, &th), rm = nm + block_scan(__popc(m), sm, &tm);
        for (; h != 0; h &= h - 1, ++rh) {
            const int32_t page = (int32_t)p0 + __ffs((int)h) - 1;
            holes[rh] = page;
            rank[page] = 0;
        }
        for (; m != 0; m &= m - 1, ++rm) {
            const int32_t page = (int32_t)p0 + __ffs((int)m) - 1;
            movers[rm] = page;
            rank[page] = rm;
        }
        if (w < words) C.bits[w] = all & ~low;
        nh += th;
        nm += tm;
    }
    if (tid == 0) {
        // past the lists: how many move, and how many pages are in use
        C.list[3 * (int64_t)C.num_pages] = nm;
        C.list[3 * (int64_t)C.num_pages + 1] = live;
        if (moved != nullptr) *moved = nm;
    }
    if (!tables || nm == 0) return;
    __syncthreads();
    for (int e = tid; e < C.max_slots * C.max_pages; e += kPlanThreads) {
        const int s = e / C.max_pages;
        follow(C, s, e - s * C.max_pages, C.len[s], live);
    }
}

// Step 2 of the larger ones.
__global__ void __launch_bounds__(kCopyThreads) k_compact_table(CacheDev C)
{
    chained();
    const int s = blockIdx.x;
    const int32_t n = C.len[s], live = C.list[3 * (int64_t)C.num_pages + 1];
    for (int i = threadIdx.x; i < C.held(n); i += kCopyThreads) follow(C, s, i, n, live);
}

// Step 3: rows and counts move.  A CTA takes one plane of one moving page at
// a time.
template <typename V>
__global__ void __launch_bounds__(kCopyThreads) k_compact_copy(CacheDev C, VecPool<V> A)
{
    chained();
    const int32_t *const holes = C.list, *const movers = C.list + C.num_pages, *const rank = C.list + 2 * (int64_t)C.num_pages;
    const int64_t units = (int64_t)C.list[3 * (int64_t)C.num_pages] * A.planes;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int r = (int)(u / A.planes), p = (int)(u - (int64_t)r * A.planes);
        const int32_t src = movers[r], dst = holes[r];
        copy_page(A, src, dst, rank[dst], p);
        if (p == 0 && threadIdx.x == 0) {
            C.refs[dst] = C.refs[src];
            C.refs[src] = 0;
        }
    }
}

// The widest vector that a pool (and a source's pointers and strides, in
// bytes) can be moved in.
int vector_bytes(const clk_pool& p, int64_t more)
{
    const int64_t es = dtype_bytes(p.dtype);
    const int64_t all = (int64_t)(uintptr_t)p.d_base | p.plane_stride * es | p.page_stride * es | p.head_stride * es |
                        p.tok_stride * es | p.dim * es | more;
    const int64_t low = all & -all;
    return low >= 16 ? 16 : (int)low;
}

template <typename V>
VecPool<V> vec_pool(const clk_pool& p)
{
    const int64_t es = dtype_bytes(p.dtype), v = sizeof(V);
    return VecPool<V>{static_cast<V*>(p.d_base),
                      p.plane_stride * es / v,
                      p.page_stride * es / v,
                      p.head_stride * es / v,
                      p.tok_stride * es / v,
                      p.planes,
                      p.heads,
                      (int32_t)(p.dim * es / v)};
}

// Calls f with a value of the vector type of `bytes` bytes.
template <typename F>
int with_vector(int bytes, F f)
{
    switch (bytes) {
    case 16: return f(uint4{});
    case 8: return f(uint2{});
    case 4: return f(uint32_t{});
    case 2: return f(uint16_t{});
    default: return CLK_EINVAL;
    }
}

// How `rows` rows, `bytes` each in all planes, are dealt out: groups of so
// many, and shares of the planes until there are about four CTAs an SM.
// Finding a group's places is a chain of loads, the same for every size, so a
// CTA takes more rows where they are short, as long as the SMs have one each.
// A cache's life by groups of 8, of up to 16 and of up to 32: 64 prompts of 2,000
// in one layer of 4 heads of 64 150, 102 and 80 us, of 8 heads of 128 235, 223
// and 223; with 8 layers they take 8 anyway.  Eight CTAs an SM for four: the end
// of a step for 64 requests 60 us for 56.
struct Deal {
    int32_t group;
    int64_t groups;
    unsigned shares;
};

Deal deal(int64_t rows, int64_t bytes, int32_t planes)
{
    const int64_t sms = num_sms();
    Deal d{kFewRows, 0, 1};
    while (d.group < kMostRows && d.group * bytes < 65536 && rows * planes >= 2 * d.group * sms) d.group *= 2;
    d.groups = (rows + d.group - 1) / d.group;
    const int64_t want = (4 * sms + d.groups - 1) / (d.groups > 0 ? d.groups : 1);
    d.shares = (unsigned)(want < 1 ? 1 : want < planes ? want : planes);
    return d;
}

int64_t token_bytes(const clk_pool& p, int32_t planes) { return (int64_t)planes * p.heads * p.dim * dtype_bytes(p.dtype); }

}  // namespace
}  // namespace clk

using namespace clk;

extern "C" int clk_cache_workspace_bytes(int32_t max_slots, int32_t max_pages, int32_t num_pages, size_t* bytes)
{
    if (bytes == nullptr) return CLK_EINVAL;
    CacheLayout L;
    const int rc = cache_layout(max_slots, max_pages, num_pages, &L);
    if (rc != CLK_OK) return rc;
    *bytes = L.total;
    return CLK_OK;
}

extern "C" int clk_cache_create(clk_cache** h, int32_t max_slots, int32_t max_pages, int32_t num_pages,
                                int32_t page_tokens, void* d_workspace, size_t bytes)
{
    if (h == nullptr) return CLK_EINVAL;
    *h = nullptr;
    CacheLayout L;
    const int rc = cache_layout(max_slots, max_pages, num_pages, &L);
    if (rc != CLK_OK) return rc;
    int shift = 4;
    while (shift < 7 && (1 << shift) != page_tokens) ++shift;
    if ((1 << shift) != page_tokens || ((int64_t)max_pages << shift) > ((int64_t)1 << 30)) return CLK_EINVAL;
    if (d_workspace == nullptr || !aligned(d_workspace, kAlign) || bytes < L.total) return CLK_EINVAL;
    clk_cache* c = new (std::nothrow) clk_cache;
    if (c == nullptr) return CLK_EINVAL;
    char* base = static_cast<char*>(d_workspace);
    c->dev = CacheDev{reinterpret_cast<int32_t*>(base),
                      reinterpret_cast<int32_t*>(base + L.len),
                      reinterpret_cast<int32_t*>(base + L.firm),
                      reinterpret_cast<int32_t*>(base + L.refs),
                      reinterpret_cast<uint32_t*>(base + L.bits),
                      reinterpret_cast<int32_t*>(base + L.table),
                      reinterpret_cast<int2*>(base + L.req),
                      reinterpret_cast<int32_t*>(base + L.list),
                      max_slots,
                      max_pages,
                      num_pages,
                      shift};
    c->ws = d_workspace;
    c->bytes = L.total;
    *h = c;
    return CLK_OK;
}

extern "C" void clk_cache_destroy(clk_cache* h) { delete h; }

extern "C" int clk_cache_reset(clk_cache* h, clk_stream_t s)
{
    const int rc = check_cache_batch(h, 0);
    if (rc != CLK_OK) return rc;
    k_cache_reset<<<304, 256, 0, (cudaStream_t)s>>>(h->dev);
    return launch_status();
}

extern "C" int clk_cache_buffers(clk_cache* h, int32_t** d_len, int32_t** d_table, int32_t** d_refs)
{
    const int rc = check_cache_batch(h, 0);
    if (rc != CLK_OK) return rc;
    if (d_len != nullptr) *d_len = h->dev.len;
    if (d_table != nullptr) *d_table = h->dev.table;
    if (d_refs != nullptr) *d_refs = h->dev.refs;
    return CLK_OK;
}

extern "C" int clk_cache_status(clk_cache* h, int32_t* dev_status, int32_t* detail, clk_stream_t s)
{
    const int rc = check_cache_batch(h, 0);
    if (rc != CLK_OK) return rc;
    if (dev_status == nullptr) return CLK_EINVAL;
    int32_t st[2] = {0, 0};
    cudaStream_t cs = (cudaStream_t)s;
    if (cudaMemcpyAsync(st, h->dev.status, sizeof st, cudaMemcpyDeviceToHost, cs) != cudaSuccess) return CLK_ECUDA;
    if (cudaStreamSynchronize(cs) != cudaSuccess) return CLK_ECUDA;
    *dev_status = st[0];
    if (detail != nullptr) *detail = st[1];
    return CLK_OK;
}

extern "C" int clk_cache_status_clear(clk_cache* h, clk_stream_t s)
{
    const int rc = check_cache_batch(h, 0);
    if (rc != CLK_OK) return rc;
    return cuda_status(cudaMemsetAsync(h->dev.status, 0, 2 * sizeof(int32_t), (cudaStream_t)s));
}

extern "C" int clk_cache_grow(clk_cache* h, const int32_t* d_slots, int32_t B, const int32_t* d_count, clk_stream_t s)
{
    const int rc = check_cache_batch(h, B);
    if (rc != CLK_OK || B == 0) return rc;
    if (!ok_i32(d_slots) || !ok_i32(d_count)) return CLK_EINVAL;
    return launch_chained(k_cache_plan<false>, 1, kPlanThreads, (cudaStream_t)s, h->dev, d_slots, (const int32_t*)nullptr, d_count, B);
}

extern "C" int clk_cache_free(clk_cache* h, const int32_t* d_slots, int32_t B, clk_stream_t s)
{
    const int rc = check_cache_batch(h, B);
    if (rc != CLK_OK || B == 0) return rc;
    if (!ok_i32(d_slots)) return CLK_EINVAL;
    return launch_chained(k_cache_free, (unsigned)B, kCopyThreads, (cudaStream_t)s, h->dev, d_slots, B);
}

extern "C" int clk_cache_fork(clk_cache* h, const int32_t* d_src, const int32_t* d_dst, int32_t B, const clk_pool* pool,
                              clk_stream_t s)
{
    int rc = check_cache_batch(h, B);
    if (rc != CLK_OK) return rc;
    if (check_pool(pool) != CLK_OK) return CLK_EINVAL;
    if (B == 0) return CLK_OK;
    if (!ok_i32(d_src) || !ok_i32(d_dst)) return CLK_EINVAL;
    rc = launch_chained(k_cache_plan<true>, 1, kPlanThreads, (cudaStream_t)s, h->dev, d_src, d_dst, (const int32_t*)nullptr, B);
    if (rc != CLK_OK) return rc;
    const Deal deals = deal((int64_t)B * (h->dev.page_tokens() - 1), token_bytes(*pool, pool->planes), pool->planes);
    const unsigned x = (unsigned)(deals.groups > B ? deals.groups : B);
    return with_vector(vector_bytes(*pool, 0), [&](auto v) {
        using V = decltype(v);
        return launch_chained(k_cache_fork<V>, dim3(x, deals.shares), kCopyThreads, (cudaStream_t)s, h->dev, d_src, d_dst, B,
                            vec_pool<V>(*pool), deals.group);
    });
}

extern "C" int clk_cache_append(clk_cache* h, const int32_t* d_slots, int32_t B, const clk_pool* pool, int32_t layer0,
                                int32_t layers, const void* d_k, const void* d_v, int64_t layer_stride,
                                int64_t row_stride, int64_t head_stride, int64_t N, const int64_t* d_off,
                                const int32_t* d_path, const int32_t* d_count, clk_stream_t s)
{
    const int rc = check_cache_batch(h, B);
    if (rc != CLK_OK) return rc;
    if (check_pool(pool) != CLK_OK || layers < 0 || layer0 < 0 || layers > pool->planes / 2 - layer0) return CLK_EINVAL;
    if (N < 0 || layer_stride < 0 || row_stride < 0 || head_stride < 0) return CLK_EINVAL;
    if (B == 0 || N == 0 || layers == 0) return CLK_OK;
    const size_t es = (size_t)dtype_bytes(pool->dtype);
    if (!ok_i32(d_slots) || !ok_i32(d_count) || d_k == nullptr || d_v == nullptr || !aligned(d_k, es) || !aligned(d_v, es))
        return CLK_EINVAL;
    if ((d_off != nullptr && (!aligned(d_off, 8) || d_path != nullptr)) || !aligned(d_path, 4)) return CLK_EINVAL;
    const int64_t rows = d_off != nullptr ? N : (N > ((int64_t)1 << 40) / B ? -1 : N * B);
    if (rows < 0) return CLK_EINVAL;
    const Deal deals = deal(rows, token_bytes(*pool, 2 * layers), 2 * layers);
    if (deals.groups > 0x7fffffff) return CLK_EINVAL;
    const int64_t b = (int64_t)es;
    const int64_t more = (int64_t)(uintptr_t)d_k | (int64_t)(uintptr_t)d_v | layer_stride * b | row_stride * b | head_stride * b;
    return with_vector(vector_bytes(*pool, more), [&](auto v) {
        using V = decltype(v);
        const int64_t w = (int64_t)sizeof(V);
        const VecSrc<V> src{static_cast<const V*>(d_k), static_cast<const V*>(d_v), layer_stride * b / w, row_stride * b / w,
                            head_stride * b / w};
        return launch_chained(k_cache_append<V>, dim3((unsigned)deals.groups, deals.shares), kCopyThreads, (cudaStream_t)s, h->dev,
                              d_slots, B, vec_pool<V>(*pool), layer0, 2 * layers, src, N, d_off, d_path, d_count, deals.group);
    });
}

extern "C" int clk_cache_compact(clk_cache* h, const clk_pool* pool, int32_t* d_moved, clk_stream_t s)
{
    int rc = check_cache_batch(h, 0);
    if (rc != CLK_OK) return rc;
    if (check_pool(pool) != CLK_OK || !aligned(d_moved, 4)) return CLK_EINVAL;
    cudaStream_t cs = (cudaStream_t)s;
    const bool few = (int64_t)h->dev.max_slots * h->dev.max_pages <= kFewEntries;
    if ((rc = launch_chained(k_compact_plan, 1, kPlanThreads, cs, h->dev, d_moved, few)) != CLK_OK) return rc;
    if (!few && (rc = launch_chained(k_compact_table, dim3((unsigned)h->dev.max_slots), kCopyThreads, cs, h->dev)) != CLK_OK) return rc;
    return with_vector(vector_bytes(*pool, 0), [&](auto v) {
        using V = decltype(v);
        return launch_chained(k_compact_copy<V>, dim3((unsigned)(8 * num_sms())), kCopyThreads, cs, h->dev, vec_pool<V>(*pool));
    });
}
