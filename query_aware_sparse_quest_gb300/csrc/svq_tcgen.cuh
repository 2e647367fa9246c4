// What the kernels on the tcgen05 tensor cores share: descriptors, TMEM accesses,
// paired fp32 arithmetic, and waits that give up.
#pragma once

#include "svq_common.cuh"

namespace svq {
namespace {

// Descriptors differ in their low words only; the high words (stride, version,
// swizzle) are constants.  Eight k steps are issued from one statement, so that
// the issuing thread keeps ahead of the tensor pipe (64 cycles a step): with a
// descriptor built for each step it fell behind it.
constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4 << 16); }

#define SVQ_MMA_SS(ao, bo, acc)                                                  \
    "add.u32 al, %1, " #ao ";\n\tadd.u32 bl, %2, " #bo ";\n\t"                   \
    "mov.b64 ad, {al, %3};\n\tmov.b64 bd, {bl, %4};\n\t"                         \
    "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, " #acc ";\n\t"
#define SVQ_MMA_TS(ao, bo, acc)                                                  \
    "add.u32 al, %1, " #ao ";\n\tadd.u32 bl, %2, " #bo ";\n\t"                   \
    "mov.b64 bd, {bl, %3};\n\t"                                                  \
    "tcgen05.mma.cta_group::1.kind::f16 [%0], [al], bd, %4, " #acc ";\n\t"
// The same by a whole warp that runs in step, one elected lane of which issues (predicate `go`): operands that all lanes
// share stay in uniform registers, where the MMA wants them.  From a branch of one thread each is moved there first,
// 48 cycles an MMA (measured), more than one of 64 x 64 or of 128 x 16 takes.
#define SVQ_MMA_SS_IF(ao, bo, acc)                                               \
    "add.u32 al, %1, " #ao ";\n\tadd.u32 bl, %2, " #bo ";\n\t"                   \
    "mov.b64 ad, {al, %3};\n\tmov.b64 bd, {bl, %4};\n\t"                         \
    "@go tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, " #acc ";\n\t"
#define SVQ_MMA_TS_IF(ao, bo, acc)                                               \
    "add.u32 al, %1, " #ao ";\n\tadd.u32 bl, %2, " #bo ";\n\t"                   \
    "mov.b64 bd, {bl, %3};\n\t"                                                  \
    "@go tcgen05.mma.cta_group::1.kind::f16 [%0], [al], bd, %4, " #acc ";\n\t"
__device__ __forceinline__ uint32_t elected() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e;
}
// A value that all lanes of the warp hold, as the compiler cannot see: a reduction leaves it in a uniform register.
__device__ __forceinline__ int uniform(int v) { return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(v))); }
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tc_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// Two fp32 values in one 64-bit register, for the paired fp32 instructions.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 32 bytes of one thread, a whole sector: rows are written a thread each.
__device__ __forceinline__ void st_v8(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                      uint32_t g, uint32_t h) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e),
                 "r"(f), "r"(g), "r"(h)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
// Waits for a phase of an mbarrier, at most kPolls polls; false when it gave up.
// A poll that finds the phase open takes 4 us on a GB300 (3.95 measured, whatever
// time limit the instruction is given; with none named a chunk of 4096 tokens at
// 32768 takes 1348 us instead of 1255), so that is after half a second; the waits
// that this bounds are for copies and for other warps' work on a few tiles,
// microseconds.  Few instructions, as every role's loop has several: the roles of
// a CTA share the instruction caches.
constexpr uint32_t kPolls = 1u << 17;
constexpr uint32_t kPollNs = 1000;
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, more;\n\t.reg .u32 i;\n\tmov.u32 i, 0;\n"
        "again:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n\t"
        "@p bra done;\n\t"
        "add.u32 i, i, 1;\n\tsetp.lt.u32 more, i, %3;\n\t@more bra again;\n"
        "done:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "n"(kPolls), "r"(kPollNs)
        : "memory");
    return ok != 0;
}
// Whether the phase is over, without waiting.
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for a phase that mostly is over already: a test takes 16 cycles, a wait 125 even then.
__device__ __forceinline__ bool bar_ready(uint32_t bar, uint32_t parity) { return bar_test(bar, parity) || bar_wait(bar, parity); }
// The same by a whole warp; all of it leaves for `out` when it gave up.
#define SVQ_WAIT(bar, parity, out)                                                        \
    do {                                                                                  \
        if (__any_sync(0xffffffffu, !bar_wait(smem_addr(&(bar)), (parity)))) {   \
            if (lane == 0) gave_up(ct);                                                   \
            goto out;                                                                     \
        }                                                                                 \
    } while (0)

// SVQ_WAIT for phases that mostly are over.
#define TEST_WAIT(bar, parity, out)                                                       \
    do {                                                                                  \
        if (__any_sync(0xffffffffu, !bar_ready(smem_addr(&(bar)), (parity)))) {           \
            if (lane == 0) gave_up(ct);                                                   \
            goto out;                                                                     \
        }                                                                                 \
    } while (0)

// Four e4m3 codes -> two bf16 pairs, exactly: the code's exponent and mantissa
// fields are moved under bf16's, which scales the value by 2^-120; the product
// with 2^120 is exact, subnormal codes included.  The two NaN codes would read
// as +-480: see has_nan.
__device__ __forceinline__ void widen4(uint32_t c, uint32_t& lo, uint32_t& hi) {
    const uint32_t a = __byte_perm(c, 0u, 0x1404);   // bytes 1, 0 of c in the high bytes of the halves
    const uint32_t b = __byte_perm(c, 0u, 0x3424);
    const uint32_t x = ((a & 0x7f007f00u) >> 4) | (a & 0x80008000u);
    const uint32_t y = ((b & 0x7f007f00u) >> 4) | (b & 0x80008000u);
    const __nv_bfloat162 two120 = __halves2bfloat162(__ushort_as_bfloat16(0x7b80), __ushort_as_bfloat16(0x7b80));
    const __nv_bfloat162 xr = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), two120);
    const __nv_bfloat162 yr = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y), two120);
    lo = *reinterpret_cast<const uint32_t*>(&xr);
    hi = *reinterpret_cast<const uint32_t*>(&yr);
}
// The same to fp16 by the conversion unit (77 codes a cycle and SM; widen4 28), NaN codes to NaN.
__device__ __forceinline__ void widen4_f16(uint32_t c, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Bit 7 of every byte of c that is a NaN code (0x7f or 0xff).
__device__ __forceinline__ uint32_t has_nan(uint32_t c) { return ((c & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ void keep_nan(uint32_t c, uint32_t& lo, uint32_t& hi) {
    const uint32_t n = has_nan(c);
    if (n & 0x00000080u) lo |= 0x00007fffu;
    if (n & 0x00008000u) lo |= 0x7fff0000u;
    if (n & 0x00800000u) hi |= 0x00007fffu;
    if (n & 0x80000000u) hi |= 0x7fff0000u;
}
}  // namespace
}  // namespace svq
