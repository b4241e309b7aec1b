// Thin wrappers over the sm_103a instructions the attention kernel uses:
// mbarriers with bounded waits, tensor copies, tensor-core products and
// tensor memory.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace clk {

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

// Waits of one CTA give up after about two seconds (in SM clocks), or once
// another wait of the CTA has given up: `*stop` is set and false returned.
constexpr long long kWaitClocks = 4000000000ll;

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* stop)
{
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (!bar_try(bar, parity)) {
        if (*stop != 0) return false;
        if (clock64() - t0 > kWaitClocks) {
            *stop = 1;
            return false;
        }
    }
    return true;
}

// The same for a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop)
{
    return __all_sync(0xffffffffu, bar_wait(bar, parity, stop));
}

// One box of a 4-axis tensor to shared memory; x counts elements.
__device__ __forceinline__ void copy_box(uint32_t dst, const void* map, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Four bytes to shared memory, or zeros where there are none to read.
__device__ __forceinline__ void copy_word(uint32_t dst, const void* src, bool there)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// Arrives on bar once the copy_words that this thread issued so far are done.
__device__ __forceinline__ void copies_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory operand descriptors for rows of 128 bytes in the 128-byte
// swizzle.  by_row: the contraction runs along the 128-byte row (groups of
// eight rows 1024 bytes apart).  Otherwise the row runs along the other
// axis: its next 64 elements are `next` bytes on, and the next eight steps of
// the contraction 1024 bytes on.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t next)
{
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)((next >> 4) & 0x3fff) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// The same for rows of 64 bytes in the 64-byte swizzle (groups of eight rows
// 512 bytes apart), the contraction along them.
__device__ __forceinline__ uint64_t operand_64(uint32_t addr)
{
    return (uint64_t)((addr >> 4) & 0x3fff) | (1ull << 16) | ((uint64_t)(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
}

// One lane of a converged warp, always the same one.  Products are issued
// inside `if (elect())`: the compiler knows that one thread runs there and
// keeps their operands in uniform registers.  (With a lane's own predicate on
// each product an issue took 59 cycles; here 30 to 40, less than the 64 that
// a 128 x 128 x 16 product runs.)
__device__ __forceinline__ bool elect()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"(add)
        : "memory");
}

// The same for operands of 8 bits, 32 elements of the contraction.
__device__ __forceinline__ void mma_ss8(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(kind), "r"(add)
        : "memory");
}

// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, uint32_t add)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(kind), "r"(add)
        : "memory");
}

// Arrives on bar once the products that this lane issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_load_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define CLK_R16(x) \
    x(0), x(1), x(2), x(3), x(4), x(5), x(6), x(7), x(8), x(9), x(10), x(11), x(12), x(13), x(14), x(15)
#define CLK_R32(x)                                                                                                      \
    x(0), x(1), x(2), x(3), x(4), x(5), x(6), x(7), x(8), x(9), x(10), x(11), x(12), x(13), x(14), x(15), x(16), x(17), \
        x(18), x(19), x(20), x(21), x(22), x(23), x(24), x(25), x(26), x(27), x(28), x(29), x(30), x(31)

// 32 columns of the warp's 32 lanes: r[i] is this lane's column i.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t* r)
{
#define CLK_OUT(i) "=r"(r[i])
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : CLK_R32(CLK_OUT)
        : "r"(addr));
#undef CLK_OUT
}

// The same for 16 columns.
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t* r)
{
#define CLK_OUT(i) "=r"(r[i])
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : CLK_R16(CLK_OUT)
        : "r"(addr));
#undef CLK_OUT
}

__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t* r)
{
#define CLK_IN(i) "r"(r[i])
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15};" ::CLK_R16(CLK_IN),
        "r"(addr)
        : "memory");
#undef CLK_IN
}

// Keeps every use of r behind the wait before this call.
__device__ __forceinline__ void tmem_loaded(uint32_t* r)
{
#define CLK_HOLD(i) "+r"(r[i])
    asm volatile("" : CLK_R32(CLK_HOLD));
#undef CLK_HOLD
}

__device__ __forceinline__ void tmem_loaded16(uint32_t* r)
{
#define CLK_HOLD(i) "+r"(r[i])
    asm volatile("" : CLK_R16(CLK_HOLD));
#undef CLK_HOLD
}
#undef CLK_R32
#undef CLK_R16

// 32 bytes to an address that is a multiple of 32.
__device__ __forceinline__ void store32(void* p, const uint32_t* y)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]),
                 "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                 : "memory");
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two float32 operations an instruction.
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float2 unpair(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The largest of three (a NaN does not count).
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two floats rounded to two 16-bit values, `a` in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    uint32_t r;
    if (BF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Two 16-bit values times a float32 power of two.
template <bool BF16>
__device__ __forceinline__ uint32_t times(uint32_t x, float f)
{
    if (BF16) return pack2<true>(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
    float a, b;
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n" : "=f"(a), "=f"(b) : "r"(x));
    return pack2<false>(a * f, b * f);
}

}  // namespace clk
