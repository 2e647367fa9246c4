// Sums of long rows: O and its sum leave TMEM for fp32 sums of their own.
#pragma once

#include "svq_paged.cuh"
#include "svq_tcgen.cuh"

namespace svq {
namespace {

// A row's O so far goes to `to` and its sum to `held`, beside their base; `more`: onto what is there.  By whole
// warps, a row a thread; threads without one (not `valid`) write nothing.
__device__ __noinline__ void fold_out(uint32_t o_col, float* to, bool valid, bool more, float2& held, float m, float l) {
    tc_fence_after();
    const float f = !more || held.x == -INFINITY ? 0.f : ex2(held.x - m);   // bases only grow
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t y[16];
        tc_ld16(o_col + c * 16, y);
        tc_wait_ld();
        float4* const at = reinterpret_cast<float4*>(to + c * 16);
#pragma unroll
        for (int u = 0; u < 4 && valid; ++u) {
            float4 v = make_float4(__uint_as_float(y[4 * u]), __uint_as_float(y[4 * u + 1]), __uint_as_float(y[4 * u + 2]),
                                   __uint_as_float(y[4 * u + 3]));
            if (more) {
                const float4 x = at[u];
                v = make_float4(fmaf(x.x, f, v.x), fmaf(x.y, f, v.y), fmaf(x.z, f, v.z), fmaf(x.w, f, v.w));
            }
            at[u] = v;
        }
    }
    held = make_float2(m, more ? fmaf(held.y, f, l) : l);
    tc_fence_before();
}
// The other way, at the segment's end: O gets what was folded; returns the whole sum.
__device__ __noinline__ float fold_in(uint32_t o_col, const float* from, bool valid, const float2& held, float m, float l) {
    tc_fence_after();
    const float f = held.x == -INFINITY ? 0.f : ex2(held.x - m);
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        uint32_t y[16];
        tc_ld16(o_col + c * 16, y);
        tc_wait_ld();
        const float4* const at = reinterpret_cast<const float4*>(from + c * 16);
#pragma unroll
        for (int u = 0; u < 4 && valid; ++u) {
            const float4 x = at[u];
            y[4 * u] = __float_as_uint(fmaf(x.x, f, __uint_as_float(y[4 * u])));
            y[4 * u + 1] = __float_as_uint(fmaf(x.y, f, __uint_as_float(y[4 * u + 1])));
            y[4 * u + 2] = __float_as_uint(fmaf(x.z, f, __uint_as_float(y[4 * u + 2])));
            y[4 * u + 3] = __float_as_uint(fmaf(x.w, f, __uint_as_float(y[4 * u + 3])));
        }
        tc_st16(o_col + c * 16, y);
    }
    tc_wait_st();
    tc_fence_before();
    return fmaf(held.y, f, l);
}

}  // namespace
}  // namespace svq
