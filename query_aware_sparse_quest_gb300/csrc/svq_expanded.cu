// sv_expanded_attention: attention of ragged rows in the expanded form, with keys
// of 128 channels a head beside 64 rotary ones that all heads share, and values
// of 128.
//
// A warp computes one row (query token, head): lane l holds channels 4 l ..
// 4 l + 3 and rotary channels 2 l, 2 l + 1, reads the tokens the row sees one by
// one, and keeps the running maximum, sum and average of the softmax in fp32.
#include <climits>

#include "svq_paged.cuh"

namespace svq {

SVQ_DEFINE_ERROR_WORD(read_error_expanded)

namespace {

constexpr int kQueryDim = kHeadDim + kRopeDim;
constexpr int kThreads = 256;

struct ExpandedArgs {
    const __nv_bfloat16* q;
    int heads;
    const int32_t* q_start;
    int total_q;
    const __nv_bfloat16* k;
    int64_t k_stride, k_head_stride;
    const __nv_bfloat16* rope;
    int64_t rope_stride;
    const __nv_bfloat16* v;
    int64_t v_stride, v_head_stride;
    const int32_t* kv_start;
    int total_kv;
    int batch;
    bool causal;
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
};

__global__ void __launch_bounds__(kThreads) expanded_rows_kernel(const __grid_constant__ ExpandedArgs a) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    const int64_t rows = static_cast<int64_t>(a.total_q) * a.heads;
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b < a.batch; b += kThreads) {
            const int q0 = a.q_start[b], q1 = a.q_start[b + 1], k0 = a.kv_start[b], k1 = a.kv_start[b + 1];
            if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_kv) svq_flag(SV_DEVERR_Q_START);
            else if (a.causal && k1 > k0 && q1 - q0 > k1 - k0) svq_flag(SV_DEVERR_Q_START);
        }
    }
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); row < rows;
         row += static_cast<int64_t>(gridDim.x) * (kThreads / 32)) {
        const int tok = static_cast<int>(row / a.heads), h = static_cast<int>(row - static_cast<int64_t>(tok) * a.heads);
        const int b = find_le(a.q_start, a.batch, tok);
        const int q0 = a.q_start[b], q1 = a.q_start[b + 1], k0 = a.kv_start[b], k1 = a.kv_start[b + 1];
        if (q0 < 0 || tok < q0 || tok >= q1 || q1 > a.total_q) continue;
        int end = 0;   // tokens seen
        if (k0 >= 0 && k1 > k0 && k1 <= a.total_kv) {
            if (!a.causal) end = k1 - k0;
            else if (q1 - q0 <= k1 - k0) end = k1 - k0 - (q1 - tok) + 1;
        }
        const __nv_bfloat16* const qr = a.q + row * kQueryDim;
        const uint2 qa = *reinterpret_cast<const uint2*>(qr + 4 * lane);
        const uint32_t qb = *reinterpret_cast<const uint32_t*>(qr + kHeadDim + 2 * lane);
        const float q[6] = {bf16lo(qa.x), bf16hi(qa.x), bf16lo(qa.y), bf16hi(qa.y), bf16lo(qb), bf16hi(qb)};
        RowSum s;
        for (int j = 0; j < end; ++j) {
            const int64_t t = k0 + j;
            const uint2 ka = *reinterpret_cast<const uint2*>(a.k + t * a.k_stride + h * a.k_head_stride + 4 * lane);
            const uint2 va = *reinterpret_cast<const uint2*>(a.v + t * a.v_stride + h * a.v_head_stride + 4 * lane);
            const uint32_t kb = *reinterpret_cast<const uint32_t*>(a.rope + t * a.rope_stride + 2 * lane);
            float z = q[0] * bf16lo(ka.x) + q[1] * bf16hi(ka.x) + q[2] * bf16lo(ka.y) + q[3] * bf16hi(ka.y) +
                      q[4] * bf16lo(kb) + q[5] * bf16hi(kb);
#pragma unroll
            for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            s.join(RowSum{z * a.scale_log2, 1.f, make_float4(bf16lo(va.x), bf16hi(va.x), bf16lo(va.y), bf16hi(va.y))});
        }
        (void)s.write(a.out + row * kHeadDim, a.lse + row, lane);
    }
    __threadfence();
}

}  // namespace

size_t expanded_workspace_bytes(int, int, int) { return 256; }

int launch_expanded(const void* q, int num_heads, const int32_t* q_start, int total_q, const void* k, int64_t k_stride,
                    int64_t k_head_stride, const void* rope, int64_t rope_stride, const void* v, int64_t v_stride,
                    int64_t v_head_stride, const int32_t* kv_start, int total_kv, int batch, bool causal,
                    float softmax_scale, void* out, float* lse, void* /*workspace*/, int sm_count, cudaStream_t stream) {
    const ExpandedArgs a = {static_cast<const __nv_bfloat16*>(q),
                            num_heads,
                            q_start,
                            total_q,
                            static_cast<const __nv_bfloat16*>(k),
                            k_stride,
                            k_head_stride,
                            static_cast<const __nv_bfloat16*>(rope),
                            rope_stride,
                            static_cast<const __nv_bfloat16*>(v),
                            v_stride,
                            v_head_stride,
                            kv_start,
                            total_kv,
                            batch,
                            causal,
                            softmax_scale * 1.4426950408889634f,
                            static_cast<__nv_bfloat16*>(out),
                            lse};
    const int64_t want = (static_cast<int64_t>(total_q) * num_heads + kThreads / 32 - 1) / (kThreads / 32);
    const dim3 grid(static_cast<unsigned>(want < sm_count * 8 ? want : sm_count * 8));
    return launch_pdl(expanded_rows_kernel, grid, dim3(kThreads), 0, stream, a) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace svq
