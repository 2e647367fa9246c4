// sv_latent_append, sv_latent_gather: tokens' latents (512 channels) and rotary
// keys (64) into the paged pool, coded as e4m3 on the way or not, and back as
// dense bf16 rows.
//
// A warp moves one token.  Coding takes a row's max |x| by five shuffles, stores
// s = max / 448 and e4m3(x / s) (IEEE division, round to nearest even,
// saturating): the codec of the other e4m3 pools, over 512 channels.  Both calls
// are bound by HBM where they are long (1152 bytes a token on the bf16 side, 644
// on the coded one; 152489 bf16 rows read back in 60.6 us, 5.8 TB/s) and by their
// launch where they are short (4096 coded tokens 4.7 us to write, 4.2 to read).
#include <climits>

#include "svq_common.cuh"

namespace svq {

SVQ_DEFINE_ERROR_WORD(read_error_latent)

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// One token's latent and rotary key in a warp's registers: lane l holds latent channels 16 l .. 16 l + 15, and lanes
// 0-7 rotary channels 8 l .. 8 l + 7.
struct Token {
    uint4 c[2];
    uint4 r;
};

__device__ __forceinline__ Token load_rows(const __nv_bfloat16* latent, const __nv_bfloat16* rope, int lane) {
    Token t;
    t.c[0] = ld_stream_v4(latent + 16 * lane);
    t.c[1] = ld_stream_v4(latent + 16 * lane + 8);
    t.r = lane < 8 ? ld_stream_v4(rope + 8 * lane) : make_uint4(0u, 0u, 0u, 0u);
    return t;
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(unsigned char* __restrict__ pool,
                                                                 __nv_bfloat16* __restrict__ rope_pool,
                                                                 float* __restrict__ scale, int64_t num_slots,
                                                                 const __nv_bfloat16* __restrict__ latent,
                                                                 int64_t latent_stride,
                                                                 const __nv_bfloat16* __restrict__ rope,
                                                                 int64_t rope_stride,
                                                                 const int32_t* __restrict__ slot_mapping,
                                                                 int64_t num_tokens) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    pdl_wait();
    if (t >= num_tokens) return;
    const int32_t slot = slot_mapping[t];
    if (slot < 0 || slot >= num_slots) {
        if (lane == 0) svq_flag(SV_DEVERR_SLOT);
        return;
    }
    const Token x = load_rows(latent + t * latent_stride, rope + t * rope_stride, lane);
    const int64_t s = slot;
    if (lane < 8) *reinterpret_cast<uint4*>(rope_pool + s * kRopeDim + 8 * lane) = x.r;
    if (!FP8) {
        uint4* const to = reinterpret_cast<uint4*>(pool + s * (2 * kLatentDim)) + 2 * lane;
        to[0] = x.c[0];
        to[1] = x.c[1];
    } else {
        const uint32_t w[8] = {x.c[0].x, x.c[0].y, x.c[0].z, x.c[0].w, x.c[1].x, x.c[1].y, x.c[1].z, x.c[1].w};
        float f[16];
        bool odd = false;   // an infinite or NaN channel (fmaxf passes over NaN)
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[2 * e] = bf16lo(w[e]);
            f[2 * e + 1] = bf16hi(w[e]);
            amax = fmaxf(amax, fmaxf(fabsf(f[2 * e]), fabsf(f[2 * e + 1])));
            odd |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        odd = __any_sync(0xffffffffu, odd);
        const float sc = odd ? __int_as_float(0x7fffffff) : __fdiv_rn(amax, 448.f);
        uint32_t packed[4] = {0u, 0u, 0u, 0u};
        if (sc > 0.f) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const uint32_t code = __nv_cvt_float_to_fp8(__fdiv_rn(f[e], sc), __NV_SATFINITE, __NV_E4M3);
                packed[e >> 2] |= code << (8 * (e & 3));
            }
        }
        *(reinterpret_cast<uint4*>(pool + s * kLatentDim) + lane) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
        if (lane == 0) scale[s] = sc;
    }
    __threadfence();   // a kernel behind this one may read before it waits
}

// Largest i in [0, n) with a[i] <= v (a ascending).
__device__ __forceinline__ int find_row(const int32_t* a, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Rows of a warp of the read-back: one, or where they are many, kRowsEach (152489 rows: 1 67.2 us, 4 60.6, 8 62.6; 4096
// rows: 1 or 2 4.2 us, 8 5.2; 1 / 4, one request bf16 and 16 e4m3: 8192 rows 5.7 / 5.7 and 5.9 / 5.7, 24576 11.9 / 11.3 and 11.8
// / 11.7, 16 of bf16 12.4 / 13.4; from 32768 on 4 is ahead everywhere, 14.4 / 13.9 and 14.7 / 12.9, 65536 28.3 / 26.9 and 27.2 /
// 24.4).
constexpr int kRowsEach = 4, kManyRows = 32768;

struct GatherArgs {
    const unsigned char* pool;
    const __nv_bfloat16* rope_pool;
    const float* scale;
    int64_t num_pages;
    const int32_t* page_table;
    const int32_t* seq_lens;
    int batch, max_pages;
    const int32_t* row_start;
    const int32_t* first;
    int total_rows;
    __nv_bfloat16* latent;
    int64_t latent_stride;
    __nv_bfloat16* rope;
    int64_t rope_stride;
};

// R rows a warp: lane u looks up where row u is, then the rows are on their way together.
template <bool FP8, int R>
__global__ void __launch_bounds__(kThreads) latent_gather_kernel(const __grid_constant__ GatherArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * R;
    pdl_wait();
    if (blockIdx.x == 0) {   // what is wrong with the ranges and lengths
        for (int b = threadIdx.x; b < a.batch; b += kThreads) {
            const int r0 = a.row_start[b], r1 = a.row_start[b + 1];
            if (r0 < 0 || r1 < r0 || r1 > a.total_rows) {
                svq_flag(SV_DEVERR_Q_START);
            } else if (r1 > r0) {
                const int64_t len = a.seq_lens[b], f = a.first ? a.first[b] : 0;
                if (len < 0 || (len + kPage - 1) / kPage > a.max_pages || f < 0 || f + (r1 - r0) > len) svq_flag(SV_DEVERR_SEQ_LEN);
            }
        }
    }
    int64_t slot = -2;   // no request's row; -1: 0 is written
    if (lane < R && row0 + lane < a.total_rows) {
        const int r = static_cast<int>(row0) + lane;
        const int b = find_row(a.row_start, a.batch, r);
        const int r0 = a.row_start[b], r1 = a.row_start[b + 1];
        if (r0 >= 0 && r >= r0 && r < r1 && r1 <= a.total_rows) {
            slot = -1;
            const int64_t token = static_cast<int64_t>(a.first ? a.first[b] : 0) + (r - r0);
            const int64_t len = a.seq_lens[b];
            if (token >= 0 && token < len && (len + kPage - 1) / kPage <= a.max_pages) {
                const int64_t page = a.page_table[static_cast<int64_t>(b) * a.max_pages + token / kPage];
                if (page < 0 || page >= a.num_pages) svq_flag(SV_DEVERR_PAGE_TABLE);
                else slot = page * kPage + token % kPage;
            }
        }
    }
    constexpr int kAhead = R < 4 ? R : 4;   // rows on their way at a time
#pragma unroll 1
    for (int u0 = 0; u0 < R; u0 += kAhead) {
        int64_t s[kAhead];
        uint4 c0[kAhead], c1[kAhead], x[kAhead];
        float sc[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            s[u] = __shfl_sync(0xffffffffu, slot, u0 + u);
            c0[u] = c1[u] = x[u] = make_uint4(0u, 0u, 0u, 0u);
            sc[u] = 0.f;
            if (s[u] < 0) continue;
            if (lane < 8) x[u] = ld_stream_v4(a.rope_pool + s[u] * kRopeDim + 8 * lane);
            if (!FP8) {
                const unsigned char* const from = a.pool + s[u] * (2 * kLatentDim) + 32 * lane;
                c0[u] = ld_stream_v4(from);
                c1[u] = ld_stream_v4(from + 16);
            } else {
                c0[u] = ld_stream_v4(a.pool + s[u] * kLatentDim + 16 * lane);
                sc[u] = a.scale[s[u]];
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (s[u] == -2) continue;
            if (FP8 && s[u] >= 0) {
                const uint32_t w[4] = {c0[u].x, c0[u].y, c0[u].z, c0[u].w};
                uint32_t o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const __half2_raw h =
                        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((w[e >> 1] >> (16 * (e & 1))) & 0xffffu), __NV_E4M3);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                    o[e] = pack_bf16x2(f.x * sc[u], f.y * sc[u]);
                }
                c0[u] = make_uint4(o[0], o[1], o[2], o[3]);
                c1[u] = make_uint4(o[4], o[5], o[6], o[7]);
            }
            const int64_t row = row0 + u0 + u;
            uint4* const to = reinterpret_cast<uint4*>(a.latent + row * a.latent_stride) + 2 * lane;
            to[0] = c0[u];
            to[1] = c1[u];
            if (lane < 8) *reinterpret_cast<uint4*>(a.rope + row * a.rope_stride + 8 * lane) = x[u];
        }
    }
    __threadfence();
}

int launched(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

}  // namespace

int launch_latent_append(const sv_cache* c, const void* latent, int64_t latent_stride, const void* rope,
                         int64_t rope_stride, const int32_t* slot_mapping, int64_t num_tokens, cudaStream_t stream) {
    const dim3 grid(ceil_div(num_tokens, kWarps));
    const auto run = [&](auto kernel) {
        return launched(launch_pdl(kernel, grid, dim3(kThreads), 0, stream, static_cast<unsigned char*>(c->k_pool),
                                   static_cast<__nv_bfloat16*>(c->v_pool), static_cast<float*>(c->k_scale),
                                   c->num_phys_pages * kPage, static_cast<const __nv_bfloat16*>(latent), latent_stride,
                                   static_cast<const __nv_bfloat16*>(rope), rope_stride, slot_mapping, num_tokens));
    };
    return c->kv_format == SV_KV_LATENT_E4M3 ? run(latent_append_kernel<true>) : run(latent_append_kernel<false>);
}

int launch_latent_gather(const sv_cache* c, const int32_t* page_table, const int32_t* seq_lens, int batch, int max_pages,
                         const int32_t* row_start, const int32_t* first_token, int64_t total_rows, void* latent,
                         int64_t latent_stride, void* rope, int64_t rope_stride, cudaStream_t stream) {
    const GatherArgs a = {static_cast<const unsigned char*>(c->k_pool),
                          static_cast<const __nv_bfloat16*>(c->v_pool),
                          static_cast<const float*>(c->k_scale),
                          c->num_phys_pages,
                          page_table,
                          seq_lens,
                          batch,
                          max_pages,
                          row_start,
                          first_token,
                          static_cast<int>(total_rows),
                          static_cast<__nv_bfloat16*>(latent),
                          latent_stride,
                          static_cast<__nv_bfloat16*>(rope),
                          rope_stride};
    const bool fp8 = c->kv_format == SV_KV_LATENT_E4M3;
    const auto run = [&](auto kernel, int rows) {
        return launched(launch_pdl(kernel, dim3(ceil_div(total_rows, kWarps * rows)), dim3(kThreads), 0, stream, a));
    };
    if (total_rows >= kManyRows) return fp8 ? run(latent_gather_kernel<true, kRowsEach>, kRowsEach) : run(latent_gather_kernel<false, kRowsEach>, kRowsEach);
    return fp8 ? run(latent_gather_kernel<true, 1>, 1) : run(latent_gather_kernel<false, 1>, 1);
}

}  // namespace svq
