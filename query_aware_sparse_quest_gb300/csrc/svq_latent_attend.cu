// sv_latent_attention: attention in the absorbed form over the paged latents.
//
// A warp computes one row (query token, head): lane l holds latent channels
// 16 l .. 16 l + 15 and rotary channels 2 l, 2 l + 1 of the query, reads the
// tokens the row sees one by one, and keeps the running maximum, sum and average
// of the softmax in fp32.
#include <climits>

#include "svq_paged.cuh"

namespace svq {

SVQ_DEFINE_ERROR_WORD(read_error_latent_attend)

namespace {

constexpr int kQueryDim = kLatentDim + kRopeDim;
constexpr int kThreads = 256;

struct LatentArgs {
    const __nv_bfloat16* q;
    int heads;
    const int32_t* q_start;
    int total_q;
    const int32_t* page_table;
    const int32_t* seq_lens;
    int batch, max_pages;
    int64_t num_pages;
    const unsigned char* pool;
    const __nv_bfloat16* rope;
    const float* scale;
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
};

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16lo(w[e]);
        f[2 * e + 1] = bf16hi(w[e]);
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kThreads) latent_rows_kernel(const __grid_constant__ LatentArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    const int64_t rows = static_cast<int64_t>(a.total_q) * a.heads;
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < a.batch; b += kThreads) {
            const int q0 = a.q_start ? a.q_start[b] : b, q1 = a.q_start ? a.q_start[b + 1] : b + 1;
            const int len = a.seq_lens[b];
            if (q0 < 0 || q1 < q0 || q1 > a.total_q) svq_flag(SV_DEVERR_Q_START);
            else if (len < 0 || (static_cast<int64_t>(len) + kPage - 1) / kPage > a.max_pages) svq_flag(SV_DEVERR_SEQ_LEN);
            else if (len > 0 && q1 - q0 > len) svq_flag(SV_DEVERR_Q_START);
        }
    }
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); row < rows;
         row += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const int tok = static_cast<int>(row / a.heads);
        const int b = a.q_start ? find_le(a.q_start, a.batch, tok) : tok;
        const int q0 = a.q_start ? a.q_start[b] : b, q1 = a.q_start ? a.q_start[b + 1] : b + 1;
        if (q0 < 0 || tok < q0 || tok >= q1 || q1 > a.total_q) continue;
        const int len = a.seq_lens[b];
        int end = 0;   // tokens seen
        if (len > 0 && (static_cast<int64_t>(len) + kPage - 1) / kPage <= a.max_pages && q1 - q0 <= len) end = len - (q1 - tok) + 1;
        float q[18], o[16], m = -INFINITY, l = 0.f;
        const __nv_bfloat16* const qr = a.q + row * kQueryDim;
        unpack8(*reinterpret_cast<const uint4*>(qr + 16 * lane), q);
        unpack8(*reinterpret_cast<const uint4*>(qr + 16 * lane + 8), q + 8);
        const uint32_t qw = *reinterpret_cast<const uint32_t*>(qr + kLatentDim + 2 * lane);
        q[16] = bf16lo(qw);
        q[17] = bf16hi(qw);
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = 0.f;
        for (int j = 0; j < end; ++j) {
            const int64_t page = a.page_table[static_cast<int64_t>(b) * a.max_pages + j / kPage];
            if (page < 0 || page >= a.num_pages) {
                if (lane == 0) svq_flag(SV_DEVERR_PAGE_TABLE);
                continue;
            }
            const int64_t s = page * kPage + j % kPage;
            float c[16];
            if (FP8) {
                const uint4 v = *reinterpret_cast<const uint4*>(a.pool + s * kLatentDim + 16 * lane);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                const float sc = a.scale[s];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
                        static_cast<__nv_fp8x2_storage_t>((w[e >> 1] >> (16 * (e & 1))) & 0xffffu), __NV_E4M3);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
                    c[2 * e] = f.x * sc;
                    c[2 * e + 1] = f.y * sc;
                }
            } else {
                const uint4* const from = reinterpret_cast<const uint4*>(a.pool + s * (2 * kLatentDim) + 32 * lane);
                unpack8(from[0], c);
                unpack8(from[1], c + 8);
            }
            const uint32_t rw = *reinterpret_cast<const uint32_t*>(a.rope + s * kRopeDim + 2 * lane);
            float z = q[16] * bf16lo(rw) + q[17] * bf16hi(rw);
#pragma unroll
            for (int e = 0; e < 16; ++e) z = fmaf(q[e], c[e], z);
#pragma unroll
            for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            z *= a.scale_log2;
            const float mn = fmaxf(m, z), base = mn == -INFINITY ? 0.f : mn;
            const float e = ex2(m - base), p = ex2(z - base);
            m = mn;
            l = l * e + p;
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = fmaf(p, c[k], o[k] * e);
        }
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = l != 0.f ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
        uint4* const to = reinterpret_cast<uint4*>(a.out + row * kLatentDim + 16 * lane);
        to[0] = make_uint4(w[0], w[1], w[2], w[3]);
        to[1] = make_uint4(w[4], w[5], w[6], w[7]);
        if (lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
    }
    __threadfence();
}

}  // namespace

size_t latent_workspace_bytes(int, int, int) { return 256; }

int launch_latent_attention(const sv_cache* c, const void* q, int num_q_heads, const int32_t* q_start, int total_q,
                            const int32_t* page_table, const int32_t* seq_lens, int batch, int max_pages,
                            float softmax_scale, void* out, float* lse, void* /*workspace*/, int sm_count,
                            cudaStream_t stream) {
    const LatentArgs a = {static_cast<const __nv_bfloat16*>(q),
                          num_q_heads,
                          q_start,
                          total_q,
                          page_table,
                          seq_lens,
                          batch,
                          max_pages,
                          c->num_phys_pages,
                          static_cast<const unsigned char*>(c->k_pool),
                          static_cast<const __nv_bfloat16*>(c->v_pool),
                          static_cast<const float*>(c->k_scale),
                          softmax_scale * 1.4426950408889634f,
                          static_cast<__nv_bfloat16*>(out),
                          lse};
    const int64_t want = (static_cast<int64_t>(total_q) * num_q_heads + kThreads / 32 - 1) / (kThreads / 32);
    const dim3 grid(static_cast<unsigned>(want < sm_count * 8 ? want : sm_count * 8));
    const cudaError_t e = c->kv_format == SV_KV_LATENT_E4M3
                              ? launch_pdl(latent_rows_kernel<true>, grid, dim3(kThreads), 0, stream, a)
                              : launch_pdl(latent_rows_kernel<false>, grid, dim3(kThreads), 0, stream, a);
    return e == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace svq
