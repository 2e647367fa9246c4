// Decode attention of one token a request over a run of its pages: the pages a
// sliding window and its sinks leave visible, or those behind a shared prefix.
//
// One token of a kv head's query group is at most 8 rows, far fewer than a
// tcgen05 tile, and the work is bound by HBM: every visible K/V byte is read
// once (512 bytes a token and kv head in bf16, 264 in e4m3) for 8 x 512 FLOP.
// So a page is the M side of small tensor-core products that run from
// registers, S^T = K Q^T (16 tokens x 8 heads) and O^T += V^T P^T, and what
// matters is the number of pages in flight: several CTAs an SM, each with a
// ring of 8 pages that TMA fills.
//
// CTA (request x kv head, split): warp 4 loads the split's pages, warps 0-3
// take them in turn, keep a softmax of their own and join through shared
// memory.  Up to 8 splits of a row are one cluster and join through distributed
// shared memory; the partials of more are joined by a second kernel.  Behind a
// prefix a cluster also joins what the tiles left of it, so the tiles and this
// kernel, which starts while the last of them run, are the whole call (32
// requests behind 32768 tokens 38 to 40 us on the device; a kernel for the join took
// 5 us more).
//
// e4m3 pools: codes convert to f16 exactly and the products run in f16.  The
// value weight of token t is exp(z_t) s_v(t).  It is formed as
// 2^(y_t - B), y_t = log2(e) z_t + log2 s_v(t), with a running base B of its own
// beside the softmax's, so that it uses f16's range whatever the values' scale
// (exp(z_t) s_v(t) itself would fall below f16's normal numbers for values
// under 0.03 and above its largest one for values over 3e7).  P enters its
// product in the other operand's type: f16 over e4m3 pools, and two bf16 parts
// over bf16 pools (the weight's first 8 bits and the next 8), as one part's 2^-8
// would be as large an error as the output's own rounding; sums and outputs are
// fp32.
//
// Measured on a GB300 (a plain copy: 6.8 TB/s), 32 query / 4 kv heads, device
// time of a call: 8 requests with a window of 4096 tokens 16.7 us (67.5 MB, 4.0
// TB/s; 10 us at the copy's rate: 5 us are the kernel's start, the first copies
// and the join), 32 e4m3 requests with a window of 2048 22.2 us (70.5 MB, 3.2
// TB/s: 43 % of the issue slots are taken and DRAM is 34 % busy; latency within
// a page's chain of conversions and products), 32 requests at 32768 tokens without a
// window 309 us (2.15 GB, 7.0 TB/s).
#include <climits>

#include "svq_paged.cuh"

namespace svq {

SVQ_DEFINE_ERROR_WORD(read_error_window_decode)

namespace {

constexpr int kWarps = 4;                          // consumer warps; warp w takes pages w, w + 4, ...
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kParts = kWarps + 1;                 // what a CTA joins: its warps' and a prefix's part
constexpr int kStages = 8;                         // pages in flight, four producer lanes each
constexpr float kSlack = 8.f;                      // log2 units a base may lag behind the maximum
// e4m3: a value weight is 2^(y - B + kF16Lift) in f16, at most 2^15 (below f16's 65504).  Its smallest step, 2^-24,
// is then 2^-31 of a weight at the base.
constexpr float kF16Lift = 7.f;
constexpr int kMaxSplits = 64;
constexpr int kMaxCluster = 8;                     // CTAs of a cluster at most (what every launch may have)
// At least this many pages a split once every SM has work (a split costs its
// start, its merge and its partial), and at least kFewPages before that.  Device us
// with the pages in L2, 32 query / 4 kv heads: 24 pages / 12 / 48 for 8 requests of
// 256 pages 12.0 / 12.2 / 14.1, for 16 of 128 14.4 / 14.5 / 16.1; e4m3, 16 / 8 / 32
// for 8 of 128 10.4 / 11.5 / 11.5, for 32 of 32 10.3 / 10.8 / 11.0; 8 / 4 / 16 of few
// for 1 of 32 6.1 / 5.8 / 7.1, for 4 of 128 8.1 / 9.8 / 8.6, e4m3 8.8 / 10.5 / 10.2.
constexpr int kSplitPages[2] = {24, 16};           // bf16, e4m3
constexpr int kFewPages = 8;
// Rows of at most so many pages go to a cluster even where more than 8 splits would fill more SMs.
constexpr int kClusterPages = 80;
// Requests that share pages: each is read alone, shared pages and all, in one
// launch, if the batch and kv heads have at most so many pages together and a
// row so many.  Alone / shared (tiles and this kernel; a join too where more than 8
// splits read a row), 8 query heads a kv head, device us: 16 rows of 135 pages bf16
// 9.3 / 18.1, e4m3 11.0 / 21.0; 64 rows of 407 21.3 / 21.7 and 30.6 / 27.3; 128 rows
// of 200 21.0 / 23.0 and 30.0 / 26.4; 256 rows of 135 30.1 / 25.1 and 37.6 / 27.0;
// 1 row of 519 15.5 / 17.9 and 20.5 / 20.1; 1 row of 1031 24.5 / 20.5 and 34.5 /
// 22.4.  At the borders either way costs up to 2 us: 40 rows of 600 bf16 (alone)
// 22.7 / 21.5, 16 rows of 500 e4m3 (shared) 22.8 / 24.5.
constexpr int64_t kAlonePages[2] = {28000, 20000};   // bf16, e4m3
constexpr int64_t kAloneRow[2] = {640, 480};

template <bool FP8>
struct Cfg {
    static constexpr int kTile = kPage * kHeadDim * (FP8 ? 1 : 2);   // a page's K or V of one kv head
    static constexpr int kScale = FP8 ? 2 * kPage * 4 : 0;           // 16 K scales | 16 V scales
    static constexpr int kSmem = 1024 + kStages * (2 * kTile + kScale);
    static constexpr int kPerSm = FP8 ? 4 : 3;
};
static_assert(kStages * 2 * Cfg<true>::kTile >= (kParts * kMaxGroup * (kHeadDim + 3) + 2 * kMaxGroup) * 4, "the warps merge through the ring");

struct Args {
    const __nv_bfloat16* q;
    int num_q_heads, num_kv_heads, group;
    const int32_t* page_table;
    const int32_t* seq_lens;
    int max_pages;
    int64_t num_phys_pages;
    Groups groups;              // requests that share pages; none: the window's are read
    PrefixParts prefix;         // PREFIX: what a cluster joins with its part
    int window;                 // INT_MAX: none
    int sink;
    int num_splits;
    float scale_log2;           // softmax_scale * log2(e)
    const float* k_scale;
    const float* v_scale;
    __nv_bfloat16* out;         // a row's splits are a cluster, which writes its result; null: partials
    float* lse;
    float* o_part;              // [B][Hq][splits][128]
    float2* ml_part;            // [B][Hq][splits]
};

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tma_4d_hint(uint32_t dst, const void* map, int y, uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %2, %2, %3}], [%4], %5;" ::"r"(dst), "l"(map), "r"(0), "r"(y), "r"(bar), "l"(policy)
        : "memory");
}
// Two e4m3 codes (low byte first) -> f16x2 (exact).
__device__ __forceinline__ uint32_t f16x2_of(uint32_t two_codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two_codes & 0xffffu), __NV_E4M3);
    return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
// Two 16 x 16 byte tiles transposed: lane 4c + j receives bytes (rows 4j .. 4j + 3, column c) in r0 and
// (rows 4j .. 4j + 3, column c + 8) in r1 of the tile that lanes 0-15 address, and the same of that of lanes
// 16-31 in r2, r3.
__device__ __forceinline__ void ldmatrix_bytes_trans(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}
// 16-byte chunk (0 .. 15) of a row of a bf16 tile as encode_pages_map lays it out.
__device__ __forceinline__ uint32_t bf16_at(int row, int chunk) {
    return (row >> 3) * 2048 + (chunk >> 3) * 1024 + (row & 7) * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}
// 16-byte chunk (0 .. 7) of a row of an e4m3 tile (128-byte rows, 128-byte swizzle).
__device__ __forceinline__ uint32_t f8_at(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// All threads of the cluster; orders their shared accesses.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What lies at `addr` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, int rank) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
    return there;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr, int rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at_rank(addr, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, int rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at_rank(addr, rank))
                 : "memory");
    return v;
}

// The pages of a request that are read: `sinks` first ones, then w0 on.
struct View {
    int sinks, w0, count;
    int shared, row;   // the first `shared` pages are read from this row of the table
    int group;
};
// By whole warps; `report`: one of them says what is wrong.
template <bool PREFIX>
__device__ __forceinline__ View view_of(const Args& a, int len, int b, bool report) {
    View v = {0, 0, 0, 0, b, 0};
    if (a.groups.start) {
        uint32_t fault;   // of parts behind a prefix: the join reports it
        int g;
        v.w0 = page_behind(a.groups, b, len, fault, g);
        if (!PREFIX && v.w0 >= 0) {
            int reach = 0;
            bool sound = true;
            for (int g0 = 0; g0 <= g && sound; g0 += 32) {
                const int at = g0 + (threadIdx.x & 31);
                int from = 0, end = 0;
                bool ok = false;
                if (at <= g) {
                    from = a.groups.start[at];
                    end = a.groups.start[at + 1];
                    ok = a.groups.sound(from, end, a.groups.pages[at]);
                }
                ok = sound_in_order(ok, from, end, reach);
                if (g < g0 + 32) sound = __shfl_sync(0xffffffffu, ok, g - g0);
            }
            v.shared = v.w0;
            v.row = a.groups.start[g];
            v.w0 = sound ? 0 : -1;
            if (!sound) fault = SV_DEVERR_GROUP;
        }
        if (a.out && fault && report) svq_flag(fault);
        if (v.w0 < 0) return {0, 0, 0, 0, b, -1};
        v.group = g;
    } else if (len <= 0) {
        return v;
    } else {
        v.w0 = max(0, len - a.window) / kPage;
        v.sinks = sink_pages_of(a.sink, v.w0);
    }
    v.count = v.sinks + (len + kPage - 1) / kPage - v.w0;
    return v;
}

// PREFIX: requests that share pages, of which the tiles have read the shared ones:
// only those behind are read here, and the cluster joins both.
template <bool FP8, bool PREFIX>
__global__ void __launch_bounds__(kThreads, Cfg<FP8>::kPerSm)
    window_decode_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tmap_k,
                         const __grid_constant__ CUtensorMap tmap_v) {
    using C = Cfg<FP8>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint32_t s_mask[kStages];            // visible tokens of the stage's page
    __shared__ __align__(8) uint64_t full_bar[kStages];
    __shared__ __align__(8) uint64_t empty_bar[kStages];

    const int split = blockIdx.y;
    const int b = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t raw_s = smem_addr(smem_raw);
    const uint32_t ring_s = (raw_s + 1023u) & ~1023u;   // 128-byte swizzle wants 1024-byte aligned boxes
    unsigned char* const ring = smem_raw + (ring_s - raw_s);
    const float* const scale_ring = reinterpret_cast<const float*>(ring + kStages * 2 * C::kTile);
    const uint32_t full0 = smem_addr(&full_bar[0]), empty0 = smem_addr(&empty_bar[0]);

    if (threadIdx.x == 0) {
        for (int st = 0; st < kStages; ++st) {
            mbar_init(full0 + st * 8, 1);
            mbar_init(empty0 + st * 8, 1);   // stage s is read by warp s % kWarps alone
        }
        mbar_init_fence();
    }
    if (warp == kWarps) {
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    __syncthreads();

    // The inputs and pools, which the work before may still write.  Behind a prefix: the tiles have waited for it,
    // and let this kernel start when they had.
    if (!PREFIX) pdl_wait();
    int len = a.seq_lens[b];
    bool touched = true;
    if (a.groups.start) {
        touched = b >= a.groups.start[0] && b < a.groups.start[a.groups.n];
        // What is wrong with groups that hold no row.
        if (!PREFIX && blockIdx.x == 0 && split == 0)
            for (int g = threadIdx.x; g < a.groups.n; g += kThreads)
                if (!a.groups.sound(a.groups.start[g], a.groups.start[g + 1], a.groups.pages[g])) svq_flag(SV_DEVERR_GROUP);
    } else if (len < 0 || (static_cast<int64_t>(len) + kPage - 1) / kPage > a.max_pages) {
        if (threadIdx.x == 0 && split == 0) svq_flag(SV_DEVERR_SEQ_LEN);
        len = 0;
    }
    // Q^T fragments (B operand): head `row` of the group.  bf16: channels 16 k + 2 quad (+ 8).  e4m3: f16,
    // channels 16 k + 4 quad .. + 3 (a dot product does not depend on the channels' order), times a power of
    // two that puts the head's largest channel into 2^14 .. 2^15: channels down to 2^-28 of it keep all their
    // bits, whatever their size.  `back`: what undoes that for the heads of this lane's logits.
    const int quad = lane & 3, row = lane >> 2;
    uint32_t qf[8][2];
    float back[2] = {1.f, 1.f};
    if (warp < kWarps) {
        const bool hv = row < a.group;
        const __nv_bfloat16* qh =
            a.q + (static_cast<int64_t>(b) * a.num_q_heads + h * a.group + (hv ? row : 0)) * kHeadDim;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (FP8) {
                const uint2 w = hv ? *reinterpret_cast<const uint2*>(qh + 16 * k + 4 * quad) : make_uint2(0u, 0u);
                qf[k][0] = w.x;
                qf[k][1] = w.y;
            } else {
                qf[k][0] = hv ? *reinterpret_cast<const uint32_t*>(qh + 16 * k + 2 * quad) : 0u;
                qf[k][1] = hv ? *reinterpret_cast<const uint32_t*>(qh + 16 * k + 8 + 2 * quad) : 0u;
            }
        }
        if (FP8) {
            uint32_t top = 0;   // magnitudes of bf16 are in the order of their bits
#pragma unroll
            for (int k = 0; k < 8; ++k) top = __vmaxu2(top, __vmaxu2(qf[k][0] & 0x7fff7fffu, qf[k][1] & 0x7fff7fffu));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int exponent = static_cast<int>(max(top >> 16, top & 0xffffu)) >> 7;
            const int up = min(127 + 14 - exponent, 126);
            const float scale = __int_as_float((127 + up) << 23), undo = __int_as_float((127 - up) << 23);
            back[0] = __shfl_sync(0xffffffffu, undo, 8 * quad);
            back[1] = __shfl_sync(0xffffffffu, undo, 8 * quad + 4);
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) qf[k][u] = pack_half2(bf16lo(qf[k][u]) * scale, bf16hi(qf[k][u]) * scale);
        }
    }
    const View v = view_of<PREFIX>(a, len, b, split == 0 && h == 0 && threadIdx.x == 0);
    const int chunk = (v.count + a.num_splits - 1) / a.num_splits;
    const int j0 = min(v.count, split * chunk);
    const int mine = min(v.count, j0 + chunk) - j0;

    if (warp == kWarps) {
        // ---------------- loads: lanes 4u (K) and 4u + 2 (V) feed stage u with pages u, u + 8, ...
        const int32_t* const pages = a.page_table + static_cast<int64_t>(b) * a.max_pages;
        const int32_t* const first = a.page_table + static_cast<int64_t>(v.row) * a.max_pages;
        const int u = lane >> 2, part = (lane & 3) >> 1;
        const bool mover = (lane & 1) == 0;
        const uint64_t policy = l2_evict_first_policy();
        const uint32_t fb = full0 + u * 8, eb = empty0 + u * 8;
        const void* const map = part ? static_cast<const void*>(&tmap_v) : static_cast<const void*>(&tmap_k);
        // Lane l resolves the split's page i + l; the next 32 while the current ones are issued.
        auto resolve = [&](int i0, int& phys, uint32_t& mask) {
            const int i = i0 + lane;
            phys = -1;
            mask = 0;
            if (i < mine) {
                const int j = j0 + i;
                const int lp = j < v.sinks ? j : v.w0 + j - v.sinks;
                const int ph = (lp < v.shared ? first : pages)[lp];
                if (ph < 0 || ph >= a.num_phys_pages) {
                    svq_flag(SV_DEVERR_PAGE_TABLE);
                } else {
                    phys = ph;
                    mask = page_mask(lp * kPage, len - 1, a.window, a.sink);
                }
            }
        };
        int phys_c, phys_n, last = -1;
        uint32_t mask_c, mask_n;
        resolve(0, phys_c, mask_c);
        bool ok = true;
        for (int base = 0; base < mine && ok; base += 32) {
            resolve(base + 32, phys_n, mask_n);
            for (int sub = 0; sub < 32 && base + sub < mine; sub += kStages) {
                const int i = base + sub + u;
                const int phys = __shfl_sync(0xffffffffu, phys_c, sub + u);
                const uint32_t mask = __shfl_sync(0xffffffffu, mask_c, sub + u);
                bool mine_ok = true;
                if (mover && i < mine) {
                    if (i >= kStages) mine_ok = mbar_wait_bounded(eb, ((i / kStages) - 1) & 1);
                    if (mine_ok) {
                        if (part == 0) {
                            s_mask[u] = mask;
                            if (phys >= 0) mbar_arrive_expect_tx(fb, 2 * C::kTile + C::kScale);
                            else mbar_arrive(fb);
                        }
                        if (phys >= 0) {
                            const int64_t at = static_cast<int64_t>(phys) * a.num_kv_heads + h;
                            const uint32_t dst = ring_s + (2 * u + part) * C::kTile;
                            if (FP8) {
                                tma_load_2d_hint(dst, map, 0, static_cast<int>(at * kPage), fb, policy);
                                bulk_copy_g2s_hint(ring_s + kStages * 2 * C::kTile + u * C::kScale + part * (kPage * 4),
                                                   (part ? a.v_scale : a.k_scale) + at * kPage, kPage * 4, fb, policy);
                            } else {
                                tma_4d_hint(dst, map, static_cast<int>(at * 2), fb, policy);
                            }
                        }
                        last = i;
                    }
                }
                if (__any_sync(0xffffffffu, !mine_ok)) {
                    ok = false;
                    break;
                }
            }
            phys_c = phys_n;
            mask_c = mask_n;
        }
        if (!ok) svq_flag(SV_DEVERR_TIMEOUT);
        // This lane's copies land before the CTA (and its shared memory) retires.
        if (last >= 0) (void)mbar_wait_bounded(fb, (last / kStages) & 1);
        if (!a.out) {
            pdl_launch_dependents();   // (results may be inputs of what comes next)
            if (PREFIX) pdl_wait();
            return;
        }
        __syncwarp();
        cluster_sync();
        cluster_sync();
        return;
    }

    // ---------------- warps 0-3
    float o[8][4];   // channels 16 mt + row (and + 8), heads 2 quad, 2 quad + 1
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY};   // the heads' bases (log2 units)
    float mo[2] = {-INFINITY, -INFINITY};  // and those of their outputs (the same in bf16)
    float l[2] = {0.f, 0.f};               // lane-partial sums
    const int mat = lane >> 3, r8 = lane & 7;
    // Tokens of this lane's logits.  e4m3: the value product reads tokens 4 quad .. + 3 as its k slots
    // (2 quad, + 1, + 8, + 9), so rows r and r + 8 of the logit tile hold the tokens that go there.
    auto token = [](int r) { return FP8 ? 4 * ((r & 7) >> 1) + (r & 1) + 2 * (r >> 3) : r; };
    const int tok0 = token(row), tok1 = token(row + 8);
    const int krow = token(r8 + 8 * (mat & 1));   // ldmatrix row of the key tile
    const int vrow = r8 + 8 * (mat >> 1);         // and of the value tile (bf16)
    for (int i = warp; i < mine; i += kWarps) {
        const int st = i % kStages;
        if (__any_sync(0xffffffffu, !mbar_wait_bounded(full0 + st * 8, (i / kStages) & 1))) {
            if (lane == 0) svq_flag(SV_DEVERR_TIMEOUT);
            break;
        }
        const uint32_t ks_s = ring_s + 2 * st * C::kTile, vs_s = ks_s + C::kTile;
        const uint32_t mask = s_mask[st];
        if (mask != 0xffffu) {
            // Value rows of tokens that are not seen may hold anything: zero them, so that P = 0 never
            // meets a NaN.  (Keys are masked on the logits.)
            unsigned char* const vb = ring + (2 * st + 1) * C::kTile;
            constexpr int kChunks = FP8 ? 8 : 16;
            for (int c = lane; c < kPage * kChunks; c += 32) {
                const int r = c / kChunks, k = c % kChunks;
                if (!((mask >> r) & 1u))
                    *reinterpret_cast<uint4*>(vb + (FP8 ? f8_at(r, k) : bf16_at(r, k))) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
        }
        // S^T (16 tokens x 8 heads) = K Q^T, two accumulation chains.
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
        if (FP8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t r0, r1, r2, r3;
                ldmatrix_x4(ks_s + f8_at(krow, 2 * k + (mat >> 1)), r0, r1, r2, r3);
                mma_f16_16816(sa, f16x2_of(r0), f16x2_of(r1), f16x2_of(r0 >> 16), f16x2_of(r1 >> 16), qf[2 * k][0], qf[2 * k][1]);
                mma_f16_16816(sb, f16x2_of(r2), f16x2_of(r3), f16x2_of(r2 >> 16), f16x2_of(r3 >> 16), qf[2 * k + 1][0],
                              qf[2 * k + 1][1]);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t r0, r1, r2, r3;
                ldmatrix_x4(ks_s + bf16_at(krow, 2 * k + (mat >> 1)), r0, r1, r2, r3);
                if (k & 1) mma_bf16_16816(sb, r0, r1, r2, r3, qf[k][0], qf[k][1]);
                else mma_bf16_16816(sa, r0, r1, r2, r3, qf[k][0], qf[k][1]);
            }
        }
        const bool on0 = (mask >> tok0) & 1u, on1 = (mask >> tok1) & 1u;
        const float* const sc = scale_ring + st * (C::kScale / 4);
        const float f0 = FP8 && on0 ? sc[tok0] * a.scale_log2 : a.scale_log2;
        const float f1 = FP8 && on1 ? sc[tok1] * a.scale_log2 : a.scale_log2;
        const float k0 = FP8 ? back[0] : 1.f, k1 = FP8 ? back[1] : 1.f;
        const float x0 = on0 ? (sa[0] + sb[0]) * k0 * f0 : -INFINITY;   // token tok0, head 2 quad
        const float x1 = on0 ? (sa[1] + sb[1]) * k1 * f0 : -INFINITY;   // token tok0, head 2 quad + 1
        const float x2 = on1 ? (sa[2] + sb[2]) * k0 * f1 : -INFINITY;   // token tok1, head 2 quad
        const float x3 = on1 ? (sa[3] + sb[3]) * k1 * f1 : -INFINITY;   // token tok1, head 2 quad + 1
        // e4m3: the logarithm of the value weights.
        const float lv0 = FP8 && on0 ? lg2(sc[kPage + tok0]) : 0.f, lv1 = FP8 && on1 ? lg2(sc[kPage + tok1]) : 0.f;
        const float y0 = FP8 ? x0 + lv0 : x0, y1 = FP8 ? x1 + lv0 : x1, y2 = FP8 ? x2 + lv1 : x2, y3 = FP8 ? x3 + lv1 : x3;
        // A base moves only when something lies more than kSlack above it; weights stay at most 2^kSlack.
        bool grow = x0 > m[0] + kSlack || x2 > m[0] + kSlack || x1 > m[1] + kSlack || x3 > m[1] + kSlack;
        if (FP8) grow = grow || y0 > mo[0] + kSlack || y2 > mo[0] + kSlack || y1 > mo[1] + kSlack || y3 > mo[1] + kSlack;
        if (__any_sync(0xffffffffu, grow)) {
            float t0 = fmaxf(x0, x2), t1 = fmaxf(x1, x3), u0 = fmaxf(y0, y2), u1 = fmaxf(y1, y3);
#pragma unroll
            for (int s = 4; s < 32; s <<= 1) {
                t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, s));
                t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, s));
                if (FP8) {
                    u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, s));
                    u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, s));
                }
            }
            if (!FP8) u0 = t0, u1 = t1;
            const float m0 = fmaxf(m[0], t0), m1 = fmaxf(m[1], t1), n0 = fmaxf(mo[0], u0), n1 = fmaxf(mo[1], u1);
            l[0] *= ex2(m[0] - (m0 == -INFINITY ? 0.f : m0));
            l[1] *= ex2(m[1] - (m1 == -INFINITY ? 0.f : m1));
            const float c0 = ex2(mo[0] - (n0 == -INFINITY ? 0.f : n0)), c1 = ex2(mo[1] - (n1 == -INFINITY ? 0.f : n1));
            m[0] = m0, m[1] = m1, mo[0] = n0, mo[1] = n1;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                o[mt][0] *= c0;
                o[mt][1] *= c1;
                o[mt][2] *= c0;
                o[mt][3] *= c1;
            }
        }
        const float b0 = m[0] == -INFINITY ? 0.f : m[0], b1 = m[1] == -INFINITY ? 0.f : m[1];
        const float p0 = ex2(x0 - b0), p1 = ex2(x1 - b1), p2 = ex2(x2 - b0), p3 = ex2(x3 - b1);
        l[0] += p0 + p2;
        l[1] += p1 + p3;
        // P^T as the B operand: lane needs tokens 2 quad + {0, 1} (+ 8) (k slots) of head `row`.
        const int src0 = (2 * quad) * 4 + (row >> 1), src1 = (2 * quad + 1) * 4 + (row >> 1);
        const uint32_t selector = (row & 1) ? 0x7632u : 0x5410u;
        auto operand = [&](uint32_t heads) {   // tokens 2 quad, + 1 of head `row`, from the lanes with pairs of heads
            return __byte_perm(__shfl_sync(0xffffffffu, heads, src0), __shfl_sync(0xffffffffu, heads, src1), selector);
        };
        uint32_t pb0, pb1, rb0 = 0, rb1 = 0;
        if (FP8) {
            const float d0 = mo[0] == -INFINITY ? 0.f : mo[0] - kF16Lift, d1 = mo[1] == -INFINITY ? 0.f : mo[1] - kF16Lift;
            pb0 = operand(pack_half2(ex2(y0 - d0), ex2(y1 - d1)));
            pb1 = operand(pack_half2(ex2(y2 - d0), ex2(y3 - d1)));
        } else {
            // A weight cut to bf16, and what is left of it (not quite 0, so that an infinite value stays one).
            auto rest = [](float p) { return fmaxf(p - __uint_as_float(__float_as_uint(p) & 0xffff0000u), 0x1p-126f); };
            pb0 = operand(__byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x7632u));
            pb1 = operand(__byte_perm(__float_as_uint(p2), __float_as_uint(p3), 0x7632u));
            rb0 = operand(pack_bf16x2(rest(p0), rest(p1)));
            rb1 = operand(pack_bf16x2(rest(p2), rest(p3)));
        }
        // O^T (128 channels x 8) += V^T P^T.  A page's product starts from zero and is added in fp32: an MMA cuts its
        // sum off towards zero, which over a long row would take as much as the output's rounding from values of one
        // sign (a million tokens in one split: 0.2 %).
        auto add = [](float (&to)[4], const float (&d)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) to[i] += d[i];
        };
        if (FP8) {
#pragma unroll
            for (int cb = 0; cb < 4; ++cb) {
                uint32_t r0, r1, r2, r3;
                ldmatrix_bytes_trans(vs_s + f8_at(lane & 15, 2 * cb + (lane >> 4)), r0, r1, r2, r3);
                float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16_16816(d0, f16x2_of(r0), f16x2_of(r1), f16x2_of(r0 >> 16), f16x2_of(r1 >> 16), pb0, pb1);
                mma_f16_16816(d1, f16x2_of(r2), f16x2_of(r3), f16x2_of(r2 >> 16), f16x2_of(r3 >> 16), pb0, pb1);
                add(o[2 * cb], d0);
                add(o[2 * cb + 1], d1);
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
                uint32_t r0, r1, r2, r3;
                ldmatrix_x4_trans(vs_s + bf16_at(vrow, 2 * mt + (mat & 1)), r0, r1, r2, r3);
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma_bf16_16816(d, r0, r1, r2, r3, pb0, pb1);
                mma_bf16_16816(d, r0, r1, r2, r3, rb0, rb1);
                add(o[mt], d);
            }
        }
        // Every lane has read the stage before it is released, and the next copy into it stays behind these reads
        // (without the fence an arrival can overtake them where the load and store unit is busy with other stores).
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + st * 8);
    }
#pragma unroll
    for (int s = 4; s < 32; s <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], s);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], s);
    }
    // Join the warps through shared memory (every page has been consumed: no copy is in flight).
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    float* const sm_o = reinterpret_cast<float*>(ring);             // [warp, prefix][8][128]
    float* const sm_m = sm_o + kParts * kMaxGroup * kHeadDim;       // [warp, prefix][8] bases, output bases, sums
    float* const sm_d = sm_m + kParts * kMaxGroup;
    float* const sm_l = sm_d + kParts * kMaxGroup;
    float2* const sm_fin = reinterpret_cast<float2*>(sm_l + kParts * kMaxGroup);   // [8] the CTA's
    {
        float* const ow = sm_o + warp * kMaxGroup * kHeadDim;
        const int h0 = 2 * quad, h1 = 2 * quad + 1;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
            ow[h0 * kHeadDim + 16 * mt + row] = o[mt][0];
            ow[h1 * kHeadDim + 16 * mt + row] = o[mt][1];
            ow[h0 * kHeadDim + 16 * mt + row + 8] = o[mt][2];
            ow[h1 * kHeadDim + 16 * mt + row + 8] = o[mt][3];
        }
        if (row < 2) {
            const int hh = row ? h1 : h0;
            sm_m[warp * kMaxGroup + hh] = row ? m[1] : m[0];
            sm_d[warp * kMaxGroup + hh] = (row ? mo[1] : mo[0]) - (FP8 ? kF16Lift : 0.f);
            sm_l[warp * kMaxGroup + hh] = row ? l[1] : l[0];
        }
    }
    // What the tiles left of this row's prefix: the splits take the pieces in turn, warp w those of
    // heads w and w + 4.  (Partials: the join wants the tiles to have ended before this kernel does.)
    const int64_t q0 = static_cast<int64_t>(b) * a.num_q_heads + h * a.group;
    int parts = kWarps;   // what there is to join
    bool dead = false;    // the row's group is not sound
    if (PREFIX) pdl_wait();
    if (PREFIX && a.out && v.group >= 0) {
        const GroupRec rec = a.prefix.rec[v.group];
        const int64_t total = a.prefix.rec[a.groups.n].before;
        dead = !rec.sound;
        if (rec.sound && v.w0 > 0) {
            const int at = b - a.groups.start[v.group], e = at / a.prefix.tok_per_entry;
            const Pieces p = prefix_pieces(a.prefix, rec, total, a.num_kv_heads, h, e,
                                           (at - e * a.prefix.tok_per_entry) * a.group, q0);
            parts = kParts;
            const bool two = warp + kWarps < a.group;
            const int h0 = min(warp, a.group - 1), h1 = two ? warp + kWarps : h0;
            RowSum s0, s1;
            for (int k = split; k < p.n; k += 4 * a.num_splits) {
                float2 ml[8];
                float4 x[8];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int piece = k + u * a.num_splits;
                    ml[u] = ml[u + 4] = make_float2(-INFINITY, 0.f);
                    x[u] = x[u + 4] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (piece < p.n) {
                        const int64_t row = p.row(piece);
                        ml[u] = p.ml[row + h0];
                        ml[u + 4] = p.ml[row + h1];
                        x[u] = *reinterpret_cast<const float4*>(p.o + (row + h0) * kHeadDim + 4 * lane);
                        x[u + 4] = *reinterpret_cast<const float4*>(p.o + (row + h1) * kHeadDim + 4 * lane);
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    s0.join(RowSum{ml[u].x, ml[u].y, x[u]});
                    s1.join(RowSum{ml[u + 4].x, ml[u + 4].y, x[u + 4]});
                }
            }
            auto put = [&](int hh, const RowSum& s) {
                const int at = kWarps * kMaxGroup + hh;
                *reinterpret_cast<float4*>(sm_o + at * kHeadDim + 4 * lane) = s.o;
                if (lane == 0) sm_m[at] = sm_d[at] = s.m, sm_l[at] = s.l;
            };
            if (warp < a.group) put(warp, s0);
            if (two) put(warp + kWarps, s1);
        }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory");
    for (int idx = threadIdx.x; idx < a.group * kHeadDim; idx += kWarps * 32) {
        const int hh = idx / kHeadDim, d = idx % kHeadDim;
        float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < (PREFIX ? kParts : kWarps); ++w)
            if (w < parts) M = fmaxf(M, sm_m[w * kMaxGroup + hh]);
        const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < (PREFIX ? kParts : kWarps); ++w) {
            if (w >= parts) break;
            L += sm_l[w * kMaxGroup + hh] * ex2(sm_m[w * kMaxGroup + hh] - base);
            O += sm_o[(w * kMaxGroup + hh) * kHeadDim + d] * ex2(sm_d[w * kMaxGroup + hh] - base);
        }
        if (a.out) {   // over warp 0's part, which only this thread reads here
            sm_o[idx] = O;
            if (d == 0) sm_fin[hh] = make_float2(M, L);
        } else {
            a.o_part[((q0 + hh) * a.num_splits + split) * kHeadDim + d] = O;
            if (d == 0) a.ml_part[(q0 + hh) * a.num_splits + split] = make_float2(M, L);
        }
    }
    if (!a.out) return;
    __syncwarp();
    cluster_sync();
    // Four channels of a head a thread, over all CTAs of the cluster.
    for (int at = split * kWarps * 32 + threadIdx.x; at < a.group * 32; at += a.num_splits * kWarps * 32) {
        const int hh = at / 32;
        float2 ml[kMaxCluster];
        float4 x[kMaxCluster];
#pragma unroll
        for (int u = 0; u < kMaxCluster; ++u) {
            ml[u] = make_float2(-INFINITY, 0.f);
            x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (u < a.num_splits) {
                ml[u] = ld_cluster_f2(smem_addr(sm_fin + hh), u);
                x[u] = ld_cluster_f4(smem_addr(sm_o + 4 * at), u);
            }
        }
        RowSum s;
#pragma unroll
        for (int u = 0; u < kMaxCluster; ++u) s.m = fmaxf(s.m, ml[u].x);
        const float base = s.m == -INFINITY ? 0.f : s.m;
#pragma unroll
        for (int u = 0; u < kMaxCluster; ++u) {
            const float f = ex2(ml[u].x - base);
            s.l += ml[u].y * f;
            s.o.x += x[u].x * f;
            s.o.y += x[u].y * f;
            s.o.z += x[u].z * f;
            s.o.w += x[u].w * f;
        }
        if (dead) s = RowSum{};
        if (touched) (void)s.write(a.out + (q0 + hh) * kHeadDim, a.lse + q0 + hh, lane);
    }
    __syncwarp();
    cluster_sync();   // the others have read this CTA's shared memory
}

// CTA per (request, query head): joins its splits.
constexpr int kJoinThreads = 128;

__global__ void __launch_bounds__(kJoinThreads) join_splits_kernel(const float* __restrict__ o_part,
                                                                   const float2* __restrict__ ml_part, int splits,
                                                                   __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
    __shared__ float4 sm_o[kJoinThreads / 32][32];
    __shared__ float2 sm_ml[kJoinThreads / 32];
    pdl_wait();
    const int64_t q = blockIdx.x;
    const Pieces pieces = {o_part, ml_part, q * splits, q * splits + 1, 1, splits};
    (void)join_row<kJoinThreads / 32>(pieces, sm_o, sm_ml, out + q * kHeadDim, lse + q);
}

// An e4m3 pool as bytes [pages * kv heads * 16][128], in 16 x 128 boxes with the 128-byte swizzle.
bool encode_codes_map(CUtensorMap* map, const void* pool, int64_t rows) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_entry());
    if (!enc) return false;
    const cuuint64_t dims[2] = {kHeadDim, static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {kHeadDim};
    const cuuint32_t box[2] = {kHeadDim, kPage};
    const cuuint32_t ones[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(pool), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP8, bool PREFIX>
int launch(const Args& a, const CUtensorMap& tk, const CUtensorMap& tv, int batch, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    const int st = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(window_decode_kernel<FP8, PREFIX>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Cfg<FP8>::kSmem) == cudaSuccess
                   ? SV_OK
                   : SV_ERR_CUDA;
    });
    if (st) return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(batch * a.num_kv_heads, a.num_splits);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Cfg<FP8>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = a.num_splits;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.out ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, window_decode_kernel<FP8, PREFIX>, a, tk, tv) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace

// Splits of every row so that one wave of CTAs fills the GPU, of no fewer
// pages than a split is worth.  `pages`: the most a row may have.
int window_decode_splits(bool fp8, int batch, int num_kv_heads, int64_t pages, int sm_count) {
    const int rows = batch * num_kv_heads;
    const int wave = sm_count * (fp8 ? Cfg<true>::kPerSm : Cfg<false>::kPerSm) / rows;
    const int64_t coarse = (pages + kSplitPages[fp8] - 1) / kSplitPages[fp8], fine = (pages + kFewPages - 1) / kFewPages;
    const int64_t cap = coarse * rows >= sm_count ? coarse : fine;
    const int64_t s = cap < wave ? cap : wave;
    return static_cast<int>(s < 1 ? 1 : (s > kMaxSplits ? kMaxSplits : s));
}

// The same, as a cluster that joins a row without a second launch (5 us of the
// host's time; the GPU's is the same); 0: more splits than a cluster has CTAs
// are faster (`must`: never).  Device us with 8 splits / with more: 32 rows bf16 of
// 256 pages 12.0 / 12.0, 20 rows 11.2 / 10.2, of 2048 pages 63.3 / 55.7; 52 rows e4m3
// of 256 21.0 / 18.3; 1 row of 64 pages 6.3 / 6.5, of 96 6.9 / 6.7, of 512 14.2 / 9.3.
// So bf16 rows that 8 splits would not bring to one and a half CTAs an SM take
// more, e4m3 rows always, short rows never.
// bf16 CTAs, three to an SM, in clusters of 7 or 8 do not fit a part of the GPU to
// its last place: where they would take more than 85 % of all places, 6 are taken.
// Of 256 pages: 40 rows with 8 (70 %) 15.2, with 6 16.1; 52 rows with 8 (91 %) 30.3,
// with 6 22.1; 64 rows with 7 (98 %) 34.8, with 8 33.5, with 6 25.7, with 5 26.1.
int window_decode_cluster(bool fp8, int batch, int num_kv_heads, int64_t pages, int sm_count, bool must) {
    const int64_t rows = static_cast<int64_t>(batch) * num_kv_heads;
    int s = window_decode_splits(fp8, batch, num_kv_heads, pages, sm_count);
    if (s > kMaxCluster) {
        if (!must && pages > kClusterPages && (fp8 || 2 * rows * kMaxCluster < 3 * sm_count)) return 0;
        s = kMaxCluster;
    }
    if (!fp8 && s > 6 && 20 * rows * s > 17ll * sm_count * Cfg<false>::kPerSm) s = 6;
    return s;
}

// Whether requests that share pages are each read alone.
bool prefix_alone(bool fp8, int batch, int num_kv_heads, int64_t pages) {
    return batch * pages * num_kv_heads <= kAlonePages[fp8] && pages <= kAloneRow[fp8];
}

// Partial rows a call can need: a row has one split, or all rows' splits fit one wave.
int64_t window_decode_rows(int batch, int num_q_heads, int num_kv_heads) {
    const int64_t one = static_cast<int64_t>(batch) * num_q_heads;
    const int64_t wave = 160ll * Cfg<true>::kPerSm * (num_q_heads / num_kv_heads);
    return one > wave ? one : wave;
}

int launch_window_decode(const sv_cache* c, const void* q, int num_q_heads, const int32_t* page_table,
                         const int32_t* seq_lens, int batch, int max_pages, int window, int sink,
                         const int32_t* group_start, const int32_t* shared_pages, int num_groups, float softmax_scale,
                         const PrefixParts* prefix, int splits, void* out, float* lse, float* o_part, float2* ml_part,
                         cudaStream_t stream) {
    const bool fp8 = c->kv_format == SV_KV_FP8_E4M3;
    // TMA coordinates are 32-bit.
    const int64_t rows = c->num_phys_pages * c->num_kv_heads * kPage;
    if ((fp8 ? rows : rows / 8) > INT_MAX) return SV_ERR_UNSUPPORTED;
    CUtensorMap tk, tv;
    const bool ok = fp8 ? encode_codes_map(&tk, c->k_pool, rows) && encode_codes_map(&tv, c->v_pool, rows)
                        : encode_pages_map(&tk, c->k_pool, rows / 8) && encode_pages_map(&tv, c->v_pool, rows / 8);
    if (!ok) return SV_ERR_CUDA;
    Args a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = c->num_kv_heads;
    a.group = num_q_heads / c->num_kv_heads;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.max_pages = max_pages;
    a.num_phys_pages = c->num_phys_pages;
    a.groups = Groups{group_start, shared_pages, num_groups, batch, max_pages};
    a.window = window > 0 ? window : INT_MAX;
    a.sink = sink;
    a.prefix = prefix ? *prefix : PrefixParts{};
    a.num_splits = splits;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.k_scale = static_cast<const float*>(c->k_scale);
    a.v_scale = static_cast<const float*>(c->v_scale);
    a.o_part = o_part;
    a.ml_part = ml_part;
    if (prefix) return fp8 ? launch<true, true>(a, tk, tv, batch, stream) : launch<false, true>(a, tk, tv, batch, stream);
    return fp8 ? launch<true, false>(a, tk, tv, batch, stream) : launch<false, false>(a, tk, tv, batch, stream);
}

int launch_join_splits(const float* o_part, const float2* ml_part, int splits, int64_t rows, void* out, float* lse,
                       cudaStream_t stream) {
    return launch_pdl(join_splits_kernel, dim3(static_cast<unsigned>(rows)), dim3(kJoinThreads), 0, stream, o_part, ml_part,
                      splits, static_cast<__nv_bfloat16*>(out), lse) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

}  // namespace svq
