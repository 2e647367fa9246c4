// Helpers shared by the window / prefix attention kernels: what a row sees, the
// pool's tensor map, and the joining of partial results.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "svq_common.cuh"

namespace svq {

// A group whose prefix the tiles work on, as the join of its rows wants it.
struct GroupRec {
    int64_t before;    // cost per kv head of the groups before it
    int tiles;         // 0: nothing is shared
    int sound;
};

// What the tiles leave of the prefixes.
struct PrefixParts {
    const GroupRec* rec;   // [groups + 1]; the last one's cost is the total
    const float* cut_o;    // partials of items that are cut
    const float2* cut_ml;
    const float* whole_o;  // those of whole items, [B Hq][128]
    const float2* whole_ml;
    int slot_rows;
    int tok_per_entry;     // requests of a row tile
    int ctas;              // that shared the work
};

namespace {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Bit t: some row at positions qlo .. qhi sees token t of the page whose first
// token is at `base`: token <= qhi, and token > qlo - window or token < sink.
__device__ __forceinline__ uint32_t union_mask(int base, int qlo, int qhi, int window, int sink) {
    const int hi = min(16, qhi - base + 1);
    if (hi <= 0) return 0u;
    const int lo = max(0, min(16, max(0, qlo - window + 1) - base));
    const int sk = max(0, min(16, sink - base));
    return ((1u << hi) - 1u) & (~((1u << lo) - 1u) | ((1u << sk) - 1u));
}
// Bit t: the row at position qpos does.
__device__ __forceinline__ uint32_t page_mask(int base, int qpos, int window, int sink) {
    return union_mask(base, qpos, qpos, window, sink);
}
// First page of a window that begins at token `lo`, and the sink pages before it.
__device__ __forceinline__ int sink_pages_of(int sink, int w0) { return min(w0, sink / kPage + (sink % kPage != 0)); }

// Largest i in [0, n) with a[i] <= v (a non-decreasing, a[0] <= v).
__device__ __forceinline__ int find_le(const int32_t* a, int n, int v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Requests in groups that share their first pages: group g is requests
// start[g] .. start[g + 1] - 1, its first pages[g] pages are shared.
struct Groups {
    const int32_t* start;   // nullptr: none
    const int32_t* pages;
    int n;
    int batch;
    int max_pages;
    // Whether group g by itself is one.
    __device__ __forceinline__ bool sound(int a, int end, int sp) const {
        return a >= 0 && a <= end && end <= batch && sp >= 0 && sp <= max_pages;
    }
};
// Groups are sound only in ascending order (none begins before a sound one
// ends), so that no row is in two of them.  By a whole warp, a group a lane:
// which of those that are sound by themselves are; `reach`: where the sound
// groups so far end.
__device__ __forceinline__ bool sound_in_order(bool ok, int a, int end, int& reach) {
    const int lane = threadIdx.x & 31;
    // The largest end of the sound groups before (an unsound one by order does not count).
    for (int round = 0; round < 32; ++round) {
        int far = ok ? end : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, far, d);
            if (lane >= d) far = max(far, y);
        }
        int prev = __shfl_up_sync(0xffffffffu, far, 1);
        if (lane == 0) prev = 0;
        const uint32_t out = __ballot_sync(0xffffffffu, ok && a < max(prev, reach));
        if (!out) {
            reach = max(reach, __shfl_sync(0xffffffffu, far, 31));
            break;
        }
        if (lane == __ffs(out) - 1) ok = false;   // the first one out of order may have hidden others
    }
    return ok;
}
// The page behind the shared ones of request b, which has `len` tokens (-1: none
// is to be read), what is wrong with it, and its group.
__device__ __forceinline__ int page_behind(const Groups& gr, int b, int len, uint32_t& fault, int& g) {
    fault = 0;
    if (b < gr.start[0] || b >= gr.start[gr.n]) return -1;
    g = find_le(gr.start, gr.n, b);
    const int a = gr.start[g], end = gr.start[g + 1], sp = gr.pages[g];
    if (!gr.sound(a, end, sp) || a > b || b >= end) fault = SV_DEVERR_GROUP;
    else if (len < 0 || (static_cast<int64_t>(len) + kPage - 1) / kPage > gr.max_pages) fault = SV_DEVERR_SEQ_LEN;
    else if (len < sp * kPage) fault = len ? SV_DEVERR_GROUP : 0u;
    else if (len > 0) return sp;
    return -1;
}

// The K or V pool bf16 [pages][kv heads][16][128] as a 4-D tensor: 64 channels,
// 8 rows (256 bytes apart), 2 channel halves (128 bytes apart), groups of 8
// rows (2 KB apart).  A box of 64 x 8 x 2 x 2 is one page's tile of one kv head
// and lands as [8-row group][half][8 rows of 128 bytes], each 1 KB block
// 128-byte swizzled: 8-row groups 2 KB apart through a whole stage, the
// uniform stride an MMA operand needs, with one copy a page.
inline bool encode_pages_map(CUtensorMap* map, const void* pool, int64_t row_groups) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_entry());
    if (!enc) return false;
    const cuuint64_t dims[4] = {64, 8, 2, static_cast<cuuint64_t>(row_groups)};
    const cuuint64_t strides[3] = {256, 128, 2048};
    const cuuint32_t box[4] = {64, 8, 2, 2};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- shares of the tiles' work
constexpr int kTilePages = 8;                       // pages of a key tile
__device__ __forceinline__ int tiles_of(int npages) { return (npages + kTilePages - 1) / kTilePages; }

// What an item costs beside its tiles (loading Q, filling the pipeline, writing
// the rows), in tiles: shares of the work count it, so that a CTA with many
// short items does not take longer than one with few long ones.  7 ragged e4m3
// requests / 32 requests behind a prefix / 61 e4m3 ones / a 4096-token chunk with
// a window, device us: 1: 96.6 / 41.2 / 43.4 / 216.4, 2: 88.6 / 41.5 / 43.9 / 215.3,
// 3: 88.3 / 41.4 / 44.3 / 215.3, 4: 87.4 / 41.8 / 44.4 / 213.5.
constexpr int kItemCost = 3;
__device__ __forceinline__ int cost_of(int tiles) { return tiles ? tiles + kItemCost : 0; }

// a / b for non-negative values that mostly fit 32 bits (a 64-bit division takes
// several times as long).
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The share of CTA c: total / ctas of the cost each, the first total % ctas one more.
struct Share {
    int64_t q, r;
    __device__ __forceinline__ Share(int64_t total, int ctas) : q(div64(total, ctas)), r(total - q * ctas) {}
    __device__ __forceinline__ int64_t start(int c) const { return c * q + (c < r ? c : r); }
    __device__ __forceinline__ int cta_of(int64_t x) const {
        const int64_t head = r * (q + 1);
        return static_cast<int>(x < head ? div64(x, q + 1) : r + div64(x - head, q));
    }
};

// An item's place in the shares: its cost begins at `begin`, its first tile
// kItemCost later.
struct Placed {
    int64_t begin;
    int tiles, c0, c1;   // the CTAs with its first and its last tile
    __device__ __forceinline__ Placed(const Share& share, int64_t at, int n)
        : begin(at), tiles(n), c0(share.cta_of(at + kItemCost)), c1(share.cta_of(at + kItemCost + n - 1)) {}
};

// Exclusive prefix sum over the block; `total` gets the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t s = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        if (lane < warps) warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[warps - 1];
    const int64_t before = warp ? warp_sums[warp - 1] : 0;
    __syncthreads();   // warp_sums may be written again
    return before + x - v;
}

// ---------------------------------------------------------------- joining partials
// A list of partials (o, (base, sum)) of one row; the base is in log2 units, o
// and the sum are relative to it.
struct Pieces {
    const float* o;
    const float2* ml;
    int64_t first;     // row of the first piece
    int64_t second;    // row of the second; the others follow `stride` apart
    int64_t stride;
    int n;
    __device__ __forceinline__ int64_t row(int k) const { return k == 0 ? first : second + (k - 1) * stride; }
};

// The partials of row r of an item that is cut: one of each of its CTAs.
__device__ __forceinline__ Pieces cut_pieces(const PrefixParts& a, const Share& share, const Placed& it, int r) {
    Pieces p;
    p.o = a.cut_o;
    p.ml = a.cut_ml;
    p.n = it.c1 - it.c0 + 1;
    p.stride = 2ll * a.slot_rows;
    p.first = (2ll * it.c0 + (share.start(it.c0) >= it.begin ? 0 : 1)) * a.slot_rows + r;
    p.second = 2ll * (it.c0 + 1) * a.slot_rows + r;
    return p;
}

// Those of a request's row in its prefix: entry e of group rec (whose entries
// come behind rec.before), row r of it, row q of the batch.
__device__ __forceinline__ Pieces prefix_pieces(const PrefixParts& a, const GroupRec& rec, int64_t total, int num_kv_heads,
                                                int h, int e, int r, int64_t q) {
    const Share share(total * num_kv_heads, a.ctas);
    const int cost = cost_of(rec.tiles);
    const Placed it(share, (rec.before + static_cast<int64_t>(e) * cost) * num_kv_heads + static_cast<int64_t>(h) * cost, rec.tiles);
    return it.c0 == it.c1 ? Pieces{a.whole_o, a.whole_ml, q, q, 0, 1} : cut_pieces(a, share, it, r);
}

// A row's running (base, sum, four channels of the output) and the pieces
// k, k + step, ... of a list, four at a time.
struct RowSum {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void add(const Pieces& p, int k, int step, int lane) {
        for (; k < p.n; k += 4 * step) {
            float2 ml[4];
            float4 x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int j = k + u * step;
                ml[u] = j < p.n ? p.ml[p.row(j)] : make_float2(-INFINITY, 0.f);
                x[u] = j < p.n ? *reinterpret_cast<const float4*>(p.o + p.row(j) * kHeadDim + 4 * lane)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mn = m;
#pragma unroll
            for (int u = 0; u < 4; ++u) mn = fmaxf(mn, ml[u].x);
            const float base = mn == -INFINITY ? 0.f : mn;   // pieces without a visible token: weights 0
            const float e = ex2(m - base);
            l *= e;
            o.x *= e, o.y *= e, o.z *= e, o.w *= e;
            m = mn;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float f = ex2(ml[u].x - base);
                l += ml[u].y * f;
                o.x += x[u].x * f;
                o.y += x[u].y * f;
                o.z += x[u].z * f;
                o.w += x[u].w * f;
            }
        }
    }
    __device__ __forceinline__ void join(const RowSum& t) {
        const float mn = fmaxf(m, t.m), base = mn == -INFINITY ? 0.f : mn;
        const float e = ex2(m - base), f = ex2(t.m - base);
        m = mn;
        l = l * e + t.l * f;
        o.x = o.x * e + t.o.x * f;
        o.y = o.y * e + t.o.y * f;
        o.z = o.z * e + t.o.z * f;
        o.w = o.w * e + t.o.w * f;
    }
    // The row of two pieces.
    __device__ __forceinline__ void add2(const float2 (&ml)[2], const float4 (&x)[2]) {
        m = fmaxf(ml[0].x, ml[1].x);
        const float base = m == -INFINITY ? 0.f : m;
        const float e = ex2(ml[0].x - base), f = ex2(ml[1].x - base);
        l = ml[0].y * e + ml[1].y * f;
        o.x = x[0].x * e + x[1].x * f;
        o.y = x[0].y * e + x[1].y * f;
        o.z = x[0].z * e + x[1].z * f;
        o.w = x[0].w * e + x[1].w * f;
    }
    // Returns whether one of the lane's channels is not finite although the sum is.  A row that sees nothing is
    // 0, whatever its tile's other rows see.
    __device__ __forceinline__ bool write(__nv_bfloat16* out, float* lse, int lane) const {
        const float inv = l > 0.f ? 1.f / l : l;
        uint2 v = make_uint2(0u, 0u);
        if (l != 0.f) {
            v.x = pack_bf16x2(o.x * inv, o.y * inv);
            v.y = pack_bf16x2(o.z * inv, o.w * inv);
        }
        *reinterpret_cast<uint2*>(out + 4 * lane) = v;
        if (lane == 0) *lse = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
        const float odd = fmaf(o.x, 0.f, fmaf(o.y, 0.f, fmaf(o.z, 0.f, o.w * 0.f)));
        return odd != 0.f && l > 0.f && l < INFINITY;
    }
};

// One row by a CTA of kWarps warps, which take the pieces in turn.  Returns what
// RowSum::write does, to the first warp.
template <int kWarps>
__device__ __forceinline__ bool join_row(const Pieces& pieces, float4 (&sm_o)[kWarps][32], float2 (&sm_ml)[kWarps],
                                         __nv_bfloat16* out, float* lse) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    bool odd = false;
    RowSum s;
    s.add(pieces, warp, kWarps, lane);
    sm_o[warp][lane] = s.o;
    if (lane == 0) sm_ml[warp] = make_float2(s.m, s.l);
    __syncthreads();
    if (warp == 0) {
        RowSum t;
#pragma unroll
        for (int u = 0; u < kWarps; ++u) t.m = fmaxf(t.m, sm_ml[u].x);
#pragma unroll
        for (int u = 0; u < kWarps; ++u) {
            const float f = ex2(sm_ml[u].x - (t.m == -INFINITY ? 0.f : t.m));
            t.l += sm_ml[u].y * f;
            t.o.x += sm_o[u][lane].x * f;
            t.o.y += sm_o[u][lane].y * f;
            t.o.z += sm_o[u][lane].z * f;
            t.o.w += sm_o[u][lane].w * f;
        }
        odd = t.write(out, lse, lane);
    }
    __syncthreads();   // the shared arrays are written again for the next row
    return odd;
}

}  // namespace
}  // namespace svq
