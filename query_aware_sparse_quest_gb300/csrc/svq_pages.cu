// sv_pages_*: who holds which page of the pool.  Copying, forking, reserving,
// freeing and compacting pages, for all layers that share one page table.
//
// The only state beside the page table and the lengths is one int32 reference
// count a page; a page is free when its count is zero, and the lowest free
// page is always taken first, so that results depend on nothing but the
// arguments.  Finding free pages is a scan of the counts (4 bytes a page: 64 KB
// for a pool of 16384 pages) instead of a free list that every call would have
// to keep in order.
//
// A call that takes pages is planned by one cluster of 8 CTAs: each scans an
// eighth of the counts, the CTAs' sums are exchanged through distributed
// shared memory, and the cluster barrier orders its phases, so that a scan
// over the whole pool and what depends on it are one launch.  Moving page
// data is a second launch over the whole GPU, one CTA at a time per page and
// layer (34 KB for 4 kv heads), bound by HBM.  Measured on a GB300 (a plain copy:
// 6.8 TB/s): packing a pool of 16384 pages held to 60 per cent, 4 layers of 4 kv
// heads, 181 us for 1.10 GB read and written (6.1 TB/s); fork, reserve and free
// for 64 children of 16 parents in 8 layers 25 us on the device and 25.5 as calls,
// for 8 of 1 in one layer 18.6 and 22 to 23: four launches and three calls of the
// host, with 34 MB and 0.1 MB moved.
//
// Kernels are launched to overlap the end of the one before (a beam step of
// three calls 33 -> 24 us), but each waits for it before its first access and
// lets none after it start early: tables, lengths and slots are inputs that
// later kernels (append, page selection) read as soon as they start, without a
// wait of their own.  So every thread ends with a fence behind what it wrote.
#include <climits>

#include "svq_common.cuh"

namespace svq {

SVQ_DEFINE_ERROR_WORD(read_error_pages)

namespace {

constexpr int kCluster = 8;
constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;

struct CacheDesc {
    unsigned char* k;
    unsigned char* v;
    unsigned char* meta;
    unsigned char* k_scale;   // null for bf16 pools
    unsigned char* v_scale;   // null for latents too
    int k_chunks, v_chunks;   // 16-byte chunks of a page
    int meta_chunks;          // 0 for latents
    int scale_chunks;
};
struct CacheSet {
    CacheDesc c[SV_MAX_CACHES];
    int n;
};

// The rows of a page table.
struct Rows {
    int32_t* table;
    int32_t* lens;
    int num_rows;
    int max_pages;
    int32_t* counts;
    int num_pages;            // of the pool
};

// The last thing a thread does that has written tables, lengths or slots.
__device__ __forceinline__ void release_writes() { __threadfence(); }

__device__ __forceinline__ int cluster_rank() {
    int r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster; orders their global and shared accesses.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Writes v to the same shared variable of every CTA of the cluster (one thread).
__device__ __forceinline__ void cluster_store(const int* where, int v) {
    const uint32_t mine = smem_addr(where);
    for (int r = 0; r < kCluster; ++r) {
        uint32_t there;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(r));
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(there), "r"(v) : "memory");
    }
}

// Exclusive prefix sum over the block; `total` gets the sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T s = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    total = warp_sums[31];
    const T before = warp ? warp_sums[warp - 1] : T(0);
    __syncthreads();   // warp_sums may be written again
    return before + x - v;
}

// This CTA's part of the pool: [lo, hi).
__device__ __forceinline__ void slice(int num_pages, int rank, int& lo, int& hi) {
    const int per = (num_pages + kCluster - 1) / kCluster;
    lo = min(num_pages, rank * per);
    hi = min(num_pages, lo + per);
}

// Sum of `v` over the CTA, published to every CTA of the cluster as out[rank]
// (visible after the next cluster_sync).
__device__ __forceinline__ void publish(int v, int rank, int* warp_sums, int* out) {
    int total;
    (void)block_scan(v, warp_sums, total);
    if (threadIdx.x == 0) cluster_store(out + rank, total);
}

// Free pages of this CTA's part, in order: emit(rank over the pool, page) for ranks below `most`.
template <typename F>
__device__ __forceinline__ void each_free(const int32_t* counts, int lo, int hi, int before, int most, int* warp_sums, F&& emit) {
    for (int base = lo; base < hi && before < most; base += kPlanThreads) {
        const int p = base + threadIdx.x;
        const int free = p < hi && counts[p] <= 0;
        int total;
        const int rank = before + block_scan(free, warp_sums, total);
        if (free && rank < most) emit(rank, p);
        before += total;
    }
}

__device__ __forceinline__ int count_free(const int32_t* counts, int lo, int hi) {
    int n = 0;
    for (int p = lo + threadIdx.x; p < hi; p += kPlanThreads) n += counts[p] <= 0;
    return n;
}

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

__device__ __forceinline__ bool len_ok(const Rows& t, int len) {
    return len >= 0 && (static_cast<int64_t>(len) + kPage - 1) / kPage <= t.max_pages;
}

// One page of one layer, by the whole CTA: 16-byte chunks, eight loads a
// thread in flight before their stores.
__device__ __forceinline__ void copy_span(unsigned char* base, int64_t src, int64_t dst, int chunks) {
    const uint4* s = reinterpret_cast<const uint4*>(base) + src * chunks;
    uint4* d = reinterpret_cast<uint4*>(base) + dst * chunks;
    for (int i = threadIdx.x; i < chunks; i += kMoveThreads) d[i] = ld_stream_v4(s + i);
}
__device__ __forceinline__ void copy_page(const CacheDesc& c, int64_t src, int64_t dst) {
    if (c.v_chunks != c.k_chunks) {   // latents and their rotary keys
        copy_span(c.k, src, dst, c.k_chunks);
        copy_span(c.v, src, dst, c.v_chunks);
        if (c.k_scale) copy_span(c.k_scale, src, dst, c.scale_chunks);
        return;
    }
    const int chunks = c.k_chunks;
    const uint4* ks = reinterpret_cast<const uint4*>(c.k) + src * chunks;
    const uint4* vs = reinterpret_cast<const uint4*>(c.v) + src * chunks;
    uint4* kd = reinterpret_cast<uint4*>(c.k) + dst * chunks;
    uint4* vd = reinterpret_cast<uint4*>(c.v) + dst * chunks;
    for (int i0 = threadIdx.x; i0 < chunks; i0 += 4 * kMoveThreads) {
        uint4 k[4], v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kMoveThreads;
            if (i < chunks) {
                k[u] = ld_stream_v4(ks + i);
                v[u] = ld_stream_v4(vs + i);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kMoveThreads;
            if (i < chunks) {
                kd[i] = k[u];
                vd[i] = v[u];
            }
        }
    }
    copy_span(c.meta, src, dst, c.meta_chunks);
    if (c.k_scale) {
        copy_span(c.k_scale, src, dst, c.scale_chunks);
        copy_span(c.v_scale, src, dst, c.scale_chunks);
    }
}

// ---------------------------------------------------------------- copy
// CTA (i, layer): page src[i] -> dst[i].
__global__ void __launch_bounds__(kMoveThreads) copy_pages_kernel(const __grid_constant__ CacheSet set,
                                                                  const int32_t* __restrict__ src,
                                                                  const int32_t* __restrict__ dst, int num_pages) {
    pdl_wait();
    const int s = src[blockIdx.x], d = dst[blockIdx.x];
    if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) {
        if (threadIdx.x == 0) svq_flag(SV_DEVERR_PAGE_TABLE);
        return;
    }
    if (s != d) copy_page(set.c[blockIdx.y], s, d);
}

// ---------------------------------------------------------------- fork
struct ForkArgs {
    Rows t;
    const int32_t* parents;
    const int32_t* children;
    int n;
    int32_t* owner;      // [num_rows] first fork of a child row (large tables)
    int32_t* is_parent;  // [num_rows]
    int32_t* who;        // [n] the forks that take a page, in order
    int32_t* rank;       // [n] a fork's place among those, -1: it takes none
    int32_t* take;       // [n] page the fork got, kNone: needs none, kSkip: not made
    uint32_t* wrong;     // [n] what is wrong with its parent's pages (error bits)
};
constexpr int kNone = -1, kSkip = -2;
// Rows listed twice are found by letting every list entry name itself at its
// row and the lowest win: for tables up to this many rows in the shared memory
// of the CTA that walks the list, for others in global memory by the whole
// cluster (two more of its barriers).
constexpr int kRowsHere = 4096;

__device__ __forceinline__ bool row_ok(const Rows& t, int r) { return r >= 0 && r < t.num_rows; }
// What a CTA that finds something wrong adds to its count of free pages (at most 2^24 of them).
constexpr int kWrong = 1 << 25;
// What is wrong with the pages that row p of `len` tokens lists, by a warp (a lane's share): full ones may be -1,
// let go of behind a window.  Spans `part`, part + parts, ... of them.
__device__ __forceinline__ uint32_t pages_fault(const Rows& t, int p, int len, int part, int parts) {
    constexpr int kLoads = 8;   // in flight
    if (!row_ok(t, p) || !len_ok(t, len)) return 0u;
    const int full = len / kPage, pages = (len + kPage - 1) / kPage;
    const int32_t* row = t.table + static_cast<int64_t>(p) * t.max_pages;
    uint32_t wrong = 0;
    for (int p0 = part * kLoads * 32 + threadIdx.x % 32; p0 < pages; p0 += parts * kLoads * 32) {
        int e[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) e[u] = p0 + 32 * u < pages ? row[p0 + 32 * u] : -1;
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            if (e[u] < 0 || e[u] >= t.num_pages) {
                if (e[u] != -1 || (p0 + 32 * u == full && full < pages)) wrong |= SV_DEVERR_PAGE_TABLE;
            } else if (t.counts[e[u]] <= 0) {
                wrong |= SV_DEVERR_REF_COUNT;
            }
        }
    }
    return wrong;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    fork_plan_kernel(const __grid_constant__ ForkArgs a) {
    __shared__ int warp_sums[32];
    __shared__ int frees[kCluster];
    __shared__ int needed;
    __shared__ int owner[kRowsHere];
    __shared__ uint32_t is_parent[kRowsHere / 32];
    const int rank = cluster_rank();
    const int me = rank * kPlanThreads + threadIdx.x;
    constexpr int kAll = kCluster * kPlanThreads;
    const bool here = a.t.num_rows <= kRowsHere;
    pdl_wait();
    cluster_sync();   // every CTA of the cluster is there before another writes its shared memory
    if (!here) {
        for (int i = me; i < a.n; i += kAll) {
            const int c = a.children[i], p = a.parents[i];
            if (row_ok(a.t, c)) a.owner[c] = INT_MAX, a.is_parent[c] = 0;
            if (row_ok(a.t, p)) a.is_parent[p] = 0;
        }
        cluster_sync();
        for (int i = me; i < a.n; i += kAll) {
            const int c = a.children[i], p = a.parents[i];
            if (row_ok(a.t, c)) atomicMin(&a.owner[c], i);
            if (row_ok(a.t, p)) a.is_parent[p] = 1;
        }
        cluster_sync();
    }
    int lo, hi;
    slice(a.t.num_pages, rank, lo, hi);
    // The other CTAs look at the parents' pages while the first walks the list (no count changes before it is done).
    const int checker = rank > 0 ? (threadIdx.x / 32) * (kCluster - 1) + rank - 1 : 0;
    constexpr int kCheckers = (kCluster - 1) * (kPlanThreads / 32);
    int parent = a.parents[checker % a.n], parent_len = row_ok(a.t, parent) ? a.t.lens[parent] : 0;   // (early)
    publish(count_free(a.t.counts, lo, hi), rank, warp_sums, frees);
    if (rank == 0) {
        if (here) {
            for (int r = threadIdx.x; r < a.t.num_rows; r += kPlanThreads) owner[r] = INT_MAX;
            for (int r = threadIdx.x; r < kRowsHere / 32; r += kPlanThreads) is_parent[r] = 0;
            __syncthreads();
            for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
                const int c = a.children[i], p = a.parents[i];
                if (row_ok(a.t, c)) atomicMin(&owner[c], i);
                if (row_ok(a.t, p)) atomicOr(&is_parent[p / 32], 1u << (p % 32));
            }
            __syncthreads();
        }
        int base = 0;
        for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
            const int i = i0 + threadIdx.x;
            int need = 0, take = kSkip;
            if (i < a.n) {
                const int c = a.children[i], p = a.parents[i];
                bool fine = row_ok(a.t, c) && row_ok(a.t, p);
                if (fine)
                    fine = here ? owner[c] == i && !((is_parent[c / 32] >> (c % 32)) & 1u) : a.owner[c] == i && !a.is_parent[c];
                if (!fine) {
                    svq_flag(SV_DEVERR_ROW);
                } else {
                    const int len = a.t.lens[p];
                    if (!len_ok(a.t, len)) {
                        svq_flag(SV_DEVERR_SEQ_LEN);
                    } else {
                        take = kNone;
                        need = len % kPage != 0;
                    }
                }
            }
            int total;
            const int r = base + block_scan(need, warp_sums, total);
            if (i < a.n) {
                a.take[i] = take;
                a.rank[i] = need ? r : -1;
                if (need) a.who[r] = i;
            }
            base += total;
        }
        if (threadIdx.x == 0) cluster_store(&needed, base);
    } else {
        uint32_t found = 0;
        const int parts = max(1, kCheckers / a.n);
        for (int w = checker; w < a.n * parts; w += kCheckers) {
            if (w != checker) parent = a.parents[w % a.n], parent_len = row_ok(a.t, parent) ? a.t.lens[parent] : 0;
            found |= pages_fault(a.t, parent, parent_len, w / a.n, parts);
        }
        if (__syncthreads_or(found) && threadIdx.x == 0) cluster_store(frees + rank, frees[rank] + kWrong);
    }
    cluster_sync();
    int before = 0, all = 0;
    bool wrong = false;
    for (int r = 0; r < kCluster; ++r) {
        const int free = frees[r] % kWrong;
        if (r < rank) before += free;
        all += free;
        wrong |= frees[r] >= kWrong;
    }
    if (wrong) {   // which forks
        for (int i = me; i < a.n; i += kAll) a.wrong[i] = 0;
        cluster_sync();
        for (int i = me / 32; i < a.n; i += kAll / 32) {
            parent = a.parents[i];
            const uint32_t fault = pages_fault(a.t, parent, row_ok(a.t, parent) ? a.t.lens[parent] : 0, 0, 1);
            if (fault) atomicOr(&a.wrong[i], fault);
        }
        cluster_sync();
    }
    // The r-th free page goes to the r-th fork that takes one (a CTA's scan is past the counts it changes).  It
    // stays free if something is wrong with the pages of that fork's parent.
    each_free(a.t.counts, lo, hi, before, needed, warp_sums, [&](int r, int p) {
        const int i = a.who[r];
        if (wrong && a.wrong[i]) return;
        a.take[i] = p;
        a.t.counts[p] = 1;
    });
    for (int i = me; i < a.n; i += kAll) {
        if (wrong && a.wrong[i]) {
            if (a.rank[i] >= 0 || a.take[i] == kNone) {
                a.take[i] = kSkip;
                svq_flag(a.wrong[i]);
            }
        } else if (a.rank[i] >= all) {
            a.take[i] = kSkip;
            svq_flag(SV_DEVERR_NO_PAGE);
        }
    }
}

// CTAs below n: the child's row and the counts of the pages it shares.  The
// others: the partial page of fork i in one layer.
__global__ void __launch_bounds__(kMoveThreads) fork_move_kernel(const __grid_constant__ CacheSet set,
                                                                 const __grid_constant__ ForkArgs a) {
    pdl_wait();
    const int i = blockIdx.x;
    const int take = a.take[i];
    if (take == kSkip) return;
    const int parent = a.parents[i];
    const int len = a.t.lens[parent];
    const int full = len / kPage;
    const int32_t* from = a.t.table + static_cast<int64_t>(parent) * a.t.max_pages;
    if (blockIdx.y > 0) {
        if (take >= 0) copy_page(set.c[blockIdx.y - 1], from[full], take);
        return;
    }
    int32_t* to = a.t.table + static_cast<int64_t>(a.children[i]) * a.t.max_pages;
    for (int p = threadIdx.x; p < full; p += kMoveThreads) {
        const int e = from[p];
        to[p] = e;
        if (e >= 0) atomicAdd(&a.t.counts[e], 1);   // (the plan has looked at them)
    }
    if (threadIdx.x == 0) {
        if (len % kPage) to[full] = take;
        a.t.lens[a.children[i]] = len;
    }
    release_writes();
}

// ---------------------------------------------------------------- reserve
struct ReserveArgs {
    Rows t;
    const int32_t* rows;
    const int32_t* add;
    int n;
    int32_t* slots;
    int num_slots;
    int32_t* owner;     // [num_rows] (large tables)
    int32_t* need;      // [n + 1] pages taken before each request
    int32_t* tok;       // [n + 1] tokens before each request
    int32_t* len;       // [n] the row's length, -1: refused
    int32_t* free;      // [num_pages]
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    reserve_kernel(const __grid_constant__ ReserveArgs a) {
    __shared__ int warp_sums[32];
    __shared__ int frees[kCluster];
    __shared__ int needed, tokens;
    __shared__ int64_t wide_sums[32];
    __shared__ int owner[kRowsHere];
    constexpr int64_t kMost = INT_MAX;
    const int rank = cluster_rank();
    const int me = rank * kPlanThreads + threadIdx.x;
    constexpr int kAll = kCluster * kPlanThreads;
    const bool here = a.t.num_rows <= kRowsHere;
    pdl_wait();
    cluster_sync();   // every CTA of the cluster is there before another writes its shared memory
    if (!here) {
        for (int i = me; i < a.n; i += kAll)
            if (row_ok(a.t, a.rows[i])) a.owner[a.rows[i]] = INT_MAX;
        cluster_sync();
        for (int i = me; i < a.n; i += kAll)
            if (row_ok(a.t, a.rows[i])) atomicMin(&a.owner[a.rows[i]], i);
        cluster_sync();
    }
    int lo, hi;
    slice(a.t.num_pages, rank, lo, hi);
    publish(count_free(a.t.counts, lo, hi), rank, warp_sums, frees);
    if (rank == 0) {
        if (here) {
            for (int r = threadIdx.x; r < a.t.num_rows; r += kPlanThreads) owner[r] = INT_MAX;
            __syncthreads();
            for (int i = threadIdx.x; i < a.n; i += kPlanThreads)
                if (row_ok(a.t, a.rows[i])) atomicMin(&owner[a.rows[i]], i);
            __syncthreads();
        }
        // 64-bit sums; what is stored saturates past everything that can be served.
        int64_t pages = 0, toks = 0, total;
        for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
            const int i = i0 + threadIdx.x;
            int need = 0, add = 0, ok = 0, len = 0;
            if (i < a.n) {
                const int r = a.rows[i];
                add = max(0, a.add[i]);
                bool fine = row_ok(a.t, r) && a.add[i] >= 0;
                if (fine) fine = (here ? owner[r] : a.owner[r]) == i;
                if (!fine) {
                    svq_flag(SV_DEVERR_ROW);
                } else {
                    len = a.t.lens[r];
                    const int64_t end = static_cast<int64_t>(len) + add;
                    if (!len_ok(a.t, len) || (end + kPage - 1) / kPage > a.t.max_pages) {
                        svq_flag(SV_DEVERR_SEQ_LEN);
                    } else {
                        ok = 1;
                        need = static_cast<int>((end + kPage - 1) / kPage) - (len + kPage - 1) / kPage;
                        if (len % kPage && add > 0) {   // the page that is written on has to be the row's own
                            const int e = a.t.table[static_cast<int64_t>(r) * a.t.max_pages + len / kPage];
                            const bool in = e >= 0 && e < a.t.num_pages;
                            if (!in || a.t.counts[e] != 1) {
                                svq_flag(in ? SV_DEVERR_REF_COUNT : SV_DEVERR_PAGE_TABLE);
                                ok = need = 0;
                            }
                        }
                    }
                }
            }
            const int64_t t0 = toks + block_scan(static_cast<int64_t>(add), wide_sums, total);
            toks += total;
            if (ok && t0 + add > a.num_slots) {
                svq_flag(SV_DEVERR_SLOT);
                ok = need = 0;
            }
            const int64_t p0 = pages + block_scan(static_cast<int64_t>(need), wide_sums, total);
            pages += total;
            if (i < a.n) {
                a.len[i] = ok ? len : -1;
                a.tok[i] = static_cast<int>(min(t0, kMost));
                a.need[i] = static_cast<int>(min(p0, kMost));
            }
        }
        if (threadIdx.x == 0) {
            a.need[a.n] = static_cast<int>(min(pages, kMost));
            a.tok[a.n] = static_cast<int>(min(toks, kMost));
            cluster_store(&needed, a.need[a.n]);
            cluster_store(&tokens, a.tok[a.n]);
        }
    }
    cluster_sync();
    int before = 0, all = 0;
    for (int r = 0; r < kCluster; ++r) {
        if (r < rank) before += frees[r];
        all += frees[r];
    }
    // A request gets its pages if all that it and those before it need are there.
    auto granted = [&](int i) { return a.len[i] >= 0 && (a.need[i + 1] == a.need[i] || a.need[i + 1] <= all); };
    // The k-th free page (a CTA's scan is past the counts it changes).
    each_free(a.t.counts, lo, hi, before, min(needed, all), warp_sums, [&](int k, int p) {
        a.free[k] = p;
        const int i = find_le(a.need, a.n, k);
        if (!granted(i)) return;
        const int at = (a.len[i] + kPage - 1) / kPage + k - a.need[i];
        a.t.table[static_cast<int64_t>(a.rows[i]) * a.t.max_pages + at] = p;
        a.t.counts[p] = 1;
    });
    for (int i = me; i < a.n; i += kAll) {
        if (granted(i)) a.t.lens[a.rows[i]] = a.len[i] + a.add[i];
        else if (a.len[i] >= 0) svq_flag(SV_DEVERR_NO_PAGE);
    }
    cluster_sync();
    const int ntok = min(tokens, a.num_slots);
    for (int64_t at = me; at < ntok; at += kAll) {   // (a list may have all the entries that 32 bits count)
        const int k = static_cast<int>(at), i = find_le(a.tok, a.n, k);
        int slot = -1;
        if (granted(i)) {
            const int pos = a.len[i] + k - a.tok[i], fresh = pos / kPage - (a.len[i] + kPage - 1) / kPage;
            const int page = fresh >= 0 ? a.free[a.need[i] + fresh]
                                        : a.t.table[static_cast<int64_t>(a.rows[i]) * a.t.max_pages + pos / kPage];
            slot = page * kPage + pos % kPage;
        }
        a.slots[k] = slot;
    }
    release_writes();
}

// ---------------------------------------------------------------- free
// CTA i: pages [first, end) of row rows[i], or the whole row.  An entry is
// exchanged for -1 before its page's count goes down, so a row that is listed
// twice, or a page range freed twice, lets go of every page once.
__global__ void __launch_bounds__(kMoveThreads) free_kernel(const __grid_constant__ Rows t, const int32_t* __restrict__ rows,
                                                            const int32_t* __restrict__ first,
                                                            const int32_t* __restrict__ end) {
    pdl_wait();
    const int i = blockIdx.x;
    const int r = rows[i];
    if (!row_ok(t, r)) {
        if (threadIdx.x == 0) svq_flag(SV_DEVERR_ROW);
        return;
    }
    int len = t.lens[r];
    if (!len_ok(t, len)) {
        if (threadIdx.x == 0) svq_flag(SV_DEVERR_SEQ_LEN);
        return;
    }
    const int pages = (len + kPage - 1) / kPage;
    const int hi = end ? min(pages, end[i]) : pages;
    const int lo = first ? min(max(0, first[i]), pages) : 0;   // (so that lo + a thread's number does not wrap)
    int32_t* row = t.table + static_cast<int64_t>(r) * t.max_pages;
    for (int p = lo + threadIdx.x; p < hi; p += kMoveThreads) {
        const int e = atomicExch(&row[p], -1);
        if (e >= 0 && e < t.num_pages) {
            if (atomicSub(&t.counts[e], 1) <= 0) {
                atomicAdd(&t.counts[e], 1);
                svq_flag(SV_DEVERR_REF_COUNT);
            }
        } else if (e != -1) {
            svq_flag(SV_DEVERR_PAGE_TABLE);
        }
    }
    __syncthreads();   // every thread has read the length
    if (!first && threadIdx.x == 0) t.lens[r] = 0;
    release_writes();
}

// ---------------------------------------------------------------- compact
struct CompactArgs {
    Rows t;                 // table, lens and counts are only read
    int32_t* table_out;
    int32_t* counts_out;
    int32_t* live;          // [1]
    int32_t* src;           // [num_pages] pages that move, ascending
    int32_t* dst;           // [num_pages] where they go
    int32_t* to;            // [num_pages] new place of a page, -1: free
    int32_t* moves;         // [1]
};

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const __grid_constant__ CompactArgs a) {
    __shared__ int warp_sums[32];
    __shared__ int frees[kCluster], holes[kCluster];
    const int rank = cluster_rank();
    const int n = a.t.num_pages;
    int lo, hi;
    slice(n, rank, lo, hi);
    pdl_wait();
    cluster_sync();   // every CTA of the cluster is there before another writes its shared memory
    publish(count_free(a.t.counts, lo, hi), rank, warp_sums, frees);
    cluster_sync();
    int live = n;
    for (int r = 0; r < kCluster; ++r) live -= frees[r];
    // Free pages below `live` are filled from the live pages above it; there are as many.
    publish(lo < live ? count_free(a.t.counts, lo, min(hi, live)) : 0, rank, warp_sums, holes);
    cluster_sync();
    int hole = 0, moves = 0, mover = 0;
    for (int r = 0; r < kCluster; ++r) {
        int l, h;
        slice(n, r, l, h);
        if (r < rank) {
            hole += holes[r];
            // live pages at or above `live` in that part
            mover += max(0, h - max(l, live)) - (frees[r] - holes[r]);
        }
        moves += holes[r];
    }
    for (int base = lo; base < hi; base += kPlanThreads) {
        const int p = base + threadIdx.x;
        const int c = p < hi ? a.t.counts[p] : 0;
        const bool in = p < hi, is_live = in && c > 0;
        const bool is_hole = in && !is_live && p < live, moves_up = is_live && p >= live;
        int nh, nm;
        const int rh = hole + block_scan(static_cast<int>(is_hole), warp_sums, nh);
        const int rm = mover + block_scan(static_cast<int>(moves_up), warp_sums, nm);
        if (is_hole) a.dst[rh] = p;
        if (moves_up) a.src[rm] = p;
        if (in && !moves_up) {
            a.to[p] = is_live ? p : -1;
            if (!is_hole) a.counts_out[p] = is_live ? c : 0;
        }
        hole += nh;
        mover += nm;
    }
    cluster_sync();
    for (int k = rank * kPlanThreads + threadIdx.x; k < moves; k += kCluster * kPlanThreads) a.to[a.src[k]] = a.dst[k];
    if (rank == 0 && threadIdx.x == 0) {
        *a.live = live;
        *a.moves = moves;
    }
}

// Page copies (unit u: page u / layers in layer u % layers), counts of the
// moved pages, and the rewritten tables, each spread over the grid.
__global__ void __launch_bounds__(kMoveThreads) compact_move_kernel(const __grid_constant__ CacheSet set,
                                                                    const __grid_constant__ CompactArgs a) {
    pdl_wait();
    const int moves = *a.moves;
    const int64_t units = static_cast<int64_t>(moves) * set.n;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int k = static_cast<int>(u / set.n);
        copy_page(set.c[u - static_cast<int64_t>(k) * set.n], a.src[k], a.dst[k]);
    }
    const int64_t me = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x;
    const int64_t all = static_cast<int64_t>(gridDim.x) * kMoveThreads;
    for (int64_t k = me; k < moves; k += all) {
        const int s = a.src[k];
        const int c = a.t.counts[s];
        a.counts_out[a.dst[k]] = c;
        a.counts_out[s] = 0;
    }
    const int64_t entries = static_cast<int64_t>(a.t.num_rows) * a.t.max_pages;
    for (int64_t i = me; i < entries; i += all) {
        const int r = static_cast<int>(i / a.t.max_pages);
        const int p = static_cast<int>(i - static_cast<int64_t>(r) * a.t.max_pages);
        const int len = a.t.lens[r];
        int e = a.t.table[i];
        if (p == 0 && !len_ok(a.t, len)) svq_flag(SV_DEVERR_SEQ_LEN);
        if (len > 0 && p < (len - 1) / kPage + 1) {
            if (e >= 0 && e < a.t.num_pages) {
                e = a.to[e];
                if (e < 0) svq_flag(SV_DEVERR_REF_COUNT);   // a free page in a table
            } else if (e != -1) {
                svq_flag(SV_DEVERR_PAGE_TABLE);
            }
        }
        a.table_out[i] = e;
    }
    release_writes();
}

void fill_set(CacheSet* set, const sv_cache* caches, int n) {
    set->n = n;
    for (int i = 0; i < n; ++i) {
        const sv_cache& c = caches[i];
        const bool fp8 = c.kv_format == SV_KV_FP8_E4M3 || c.kv_format == SV_KV_LATENT_E4M3;
        CacheDesc& d = set->c[i];
        d = CacheDesc{};
        d.k = static_cast<unsigned char*>(c.k_pool);
        d.v = static_cast<unsigned char*>(c.v_pool);
        d.scale_chunks = c.num_kv_heads * 4;
        if (fp8) d.k_scale = static_cast<unsigned char*>(c.k_scale);
        if (is_latent(&c)) {
            d.k_chunks = kPage * kLatentDim * (fp8 ? 1 : 2) / 16;
            d.v_chunks = kPage * kRopeDim * 2 / 16;
        } else {
            d.k_chunks = d.v_chunks = c.num_kv_heads * (fp8 ? 128 : 256);
            d.meta = static_cast<unsigned char*>(c.meta);
            d.meta_chunks = c.num_kv_heads * 32;
            if (fp8) d.v_scale = static_cast<unsigned char*>(c.v_scale);
        }
    }
}

int launched(cudaError_t e) { return e == cudaSuccess ? SV_OK : SV_ERR_CUDA; }

size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// owner, is_parent, then four lists of n + 1 (fork: who, rank, take, wrong;
// reserve: need, tok, len), then three of num_pages (reserve: free; compact: src, dst,
// to) and a word.
size_t pages_workspace_bytes(int64_t num_pages, int num_rows, int n) {
    return 2 * up(4ull * num_rows) + 4 * up(4ull * (static_cast<size_t>(n) + 1)) + 3 * up(4ull * num_pages) + 256;
}

namespace {
struct Carve {
    int32_t *owner, *is_parent, *a, *b, *c, *d, *p, *q, *r, *word;
    Carve(void* ws, int64_t num_pages, int num_rows, int n) {
        unsigned char* at = static_cast<unsigned char*>(ws);
        auto take = [&](size_t ints) { int32_t* x = reinterpret_cast<int32_t*>(at); at += up(4 * ints); return x; };
        owner = take(num_rows);
        is_parent = take(num_rows);
        a = take(static_cast<size_t>(n) + 1);
        b = take(static_cast<size_t>(n) + 1);
        c = take(static_cast<size_t>(n) + 1);
        d = take(static_cast<size_t>(n) + 1);
        p = take(num_pages);
        q = take(num_pages);
        r = take(num_pages);
        word = take(1);
    }
};
}  // namespace

int launch_pages_copy(const sv_cache* caches, int num_caches, const int32_t* src, const int32_t* dst, int n,
                      cudaStream_t stream) {
    CacheSet set;
    fill_set(&set, caches, num_caches);
    return launched(launch_pdl(copy_pages_kernel, dim3(n, num_caches), dim3(kMoveThreads), 0, stream, set, src, dst,
                               static_cast<int>(caches[0].num_phys_pages)));
}

int launch_pages_fork(const sv_cache* caches, int num_caches, int32_t* table, int32_t* lens, int num_rows, int max_pages,
                      int32_t* counts, const int32_t* parents, const int32_t* children, int n, void* ws,
                      cudaStream_t stream) {
    CacheSet set;
    fill_set(&set, caches, num_caches);
    const int num_pages = static_cast<int>(caches[0].num_phys_pages);
    const Carve w(ws, num_pages, num_rows, n);
    ForkArgs a = {{table, lens, num_rows, max_pages, counts, num_pages}, parents, children, n, w.owner, w.is_parent,
                  w.a, w.b, w.c, reinterpret_cast<uint32_t*>(w.d)};
    const int st = launched(launch_pdl(fork_plan_kernel, dim3(kCluster), dim3(kPlanThreads), 0, stream, a));
    if (st) return st;
    return launched(launch_pdl(fork_move_kernel, dim3(n, num_caches + 1), dim3(kMoveThreads), 0, stream, set, a));
}

int launch_pages_reserve(int32_t* table, int32_t* lens, int num_rows, int max_pages, int32_t* counts, int num_pages,
                         const int32_t* rows, const int32_t* add, int n, int32_t* slots, int num_slots, void* ws,
                         cudaStream_t stream) {
    const Carve w(ws, num_pages, num_rows, n);
    ReserveArgs a = {{table, lens, num_rows, max_pages, counts, num_pages}, rows, add, n, slots, num_slots, w.owner,
                     w.a, w.b, w.c, w.p};
    return launched(launch_pdl(reserve_kernel, dim3(kCluster), dim3(kPlanThreads), 0, stream, a));
}

int launch_pages_free(int32_t* table, int32_t* lens, int num_rows, int max_pages, int32_t* counts, int num_pages,
                      const int32_t* rows, const int32_t* first, const int32_t* end, int n, cudaStream_t stream) {
    const Rows t = {table, lens, num_rows, max_pages, counts, num_pages};
    return launched(launch_pdl(free_kernel, dim3(n), dim3(kMoveThreads), 0, stream, t, rows, first, end));
}

int launch_pages_compact(const sv_cache* caches, int num_caches, const int32_t* table, const int32_t* lens, int num_rows,
                         int max_pages, const int32_t* counts, int32_t* table_out, int32_t* counts_out, int32_t* live,
                         int32_t* page_map, void* ws, int sm_count, cudaStream_t stream) {
    CacheSet set;
    fill_set(&set, caches, num_caches);
    const int num_pages = static_cast<int>(caches[0].num_phys_pages);
    const Carve w(ws, num_pages, num_rows, 0);
    CompactArgs a = {{const_cast<int32_t*>(table), const_cast<int32_t*>(lens), num_rows, max_pages,
                      const_cast<int32_t*>(counts), num_pages},
                     table_out, counts_out, live, w.p, w.q, page_map ? page_map : w.r, w.word};
    const int st = launched(launch_pdl(compact_plan_kernel, dim3(kCluster), dim3(kPlanThreads), 0, stream, a));
    if (st) return st;
    return launched(launch_pdl(compact_move_kernel, dim3(sm_count * 6), dim3(kMoveThreads), 0, stream, set, a));
}

}  // namespace svq
