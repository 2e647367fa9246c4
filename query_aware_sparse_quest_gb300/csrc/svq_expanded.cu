// sv_expanded_attention: attention of ragged rows in the expanded form on the
// tcgen05 tensor cores, with keys of 128 channels a head beside 64 rotary ones
// that all heads share, and values of 128.
//
// Mathematics.  A row tile is up to 256 query tokens of one head, two streams of
// 128 rows.  With Q (128 x 192), a key tile K (128 tokens x 192: the head's 128
// channels and the shared rotary ones) and a value tile V,
//   S = Q K^T                  (fp32 in TMEM, 12 MMAs of k = 16 channels)
//   P = exp2(S * scale - base) (bf16 in TMEM over S; base = a running maximum)
//   O = O * 2^(old - new base) + P V   (fp32 in TMEM, 8 MMAs of k = 16 tokens)
// and at the end out = O / sum P, lse = ln 2 * (base + log2 sum P), as the tiles of
// the paged calls do.  P is rounded to bf16 because one MMA takes both operands in
// one type; the sum is taken of the unrounded weights, in fp32.
//
// Work.  An entry is a row tile with the tokens it sees, an item an entry of one
// head.  Every CTA takes an equal run of the (request, head, entry, key tile)
// sequence; a run that starts or ends inside an item leaves a partial (O, base,
// sum), joined by a second kernel.  Where the keys and values do not fit the L2 and
// a head has several row tiles, CTAs take whole items first, in step with one another
// (see ExpandedArgs), and such runs of the rest.
//
// Roles of a CTA (one per SM; TMEM holds S0, S1, O0, O1 of 128 columns each):
//   warp 0       loads keys, warp 3 values: a ring of 8 blocks of 16 KB (TMA), of
//                64 channels x 128 tokens (keys) and 128 channels x 64 tokens
//                (values), so that each is freed when its products are done
//   warp 1       issues the MMAs
//   warp 2       walks the plan
//   warps 4-7    softmax of stream 0, one row a thread; warps 8-11 of stream 1
// Two streams keep the tensor cores busy while the other's softmax runs: the two
// 128-row halves of a tile, each over every key tile; or, for up to 128 rows, the
// even and the odd key tiles of the same rows, joined at the end.
//
// What bounds it (GB300): long chunks, the tensor pipe at the card's power limit (4096
// tokens of 32 heads at 32768 1533 us, 1.68 PFLOP/s, where the library's product
// sustains 1.73); short ones, the filling and emptying of the pipeline once an item and
// the three kernels' start (300 tokens of 16 heads 20.6 us, 5 ragged requests 62 us).
// 256 rows an item because K and V are read once for them: with 128 the ring would
// carry twice the bytes a product.
#include <climits>

#include "svq_fold.cuh"

namespace svq {

SVQ_DEFINE_ERROR_WORD(read_error_expanded)

namespace {

constexpr int kQueryDim = kHeadDim + kRopeDim;
constexpr int kTileTok = 128;
constexpr int kBlock = 16384;                       // bytes of a ring block
constexpr int kBlocks = 8;
constexpr int kRowTile = 256;                       // query tokens of an entry at most
constexpr int kMaxCtas = 160;                       // partial slots in the workspace
constexpr float kSlack = 8.f;                       // log2 units the base may lag behind the maximum
constexpr int kFoldTiles = 512;                     // key tiles of a stream after which its O moves into fp32 sums
constexpr int kColS = 0, kColO = 256;               // TMEM columns of S0 and O0; S1 and O1 lie 128 further
constexpr int kThreads = 384;
// 128 x 88 + 256 x 208 = 384 x 168.
constexpr int kOtherRegs = 88, kSoftmaxRegs = 208;
constexpr int kQBytes = 128 * kQueryDim * 2;        // a stream's rows
constexpr int kControlBytes = 3 * 1024;
constexpr int kSmem = kBlocks * kBlock + 2 * kQBytes + kControlBytes;
static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");

constexpr int kAllVisible = 1 << 30;

struct __align__(16) Entry {
    int row0;    // first query token (row of q)
    int ntok;
    int pos0;    // position of the first one; kAllVisible: no mask
    int kv0;     // first token (row of k)
    int len;     // tokens that some row of it sees
    int tiles;   // key tiles of those
    int pad[2];
};

// Waves: CTAs that start items at the same time, in the items' order, read the keys and values of the same heads at the
// same time, which then come from L2 (equal runs of the whole sequence have every CTA at a head of its own: each item's
// keys and values come from HBM).  A 4096-token chunk of 32 heads at 32768 tokens 1855 -> 1533 us.  Not worth it where
// the L2 holds them anyway (tokens times heads, 512 bytes each; 5 ragged requests of 60 MB 62.5 us, in waves 63.6), nor for
// many requests, as the plan looks up items one by one, nor where a head has few row tiles, which a CTA with an equal run
// takes one after the other.  Fresh prompts of 32 requests and 64 heads, equal runs / waves, us: 512 tokens 281 / 313, 1024
// 718 / 784, 1280 1013 / 1021, 1536 1431 / 1403, 1792 1832 / 1747, 3000 5291 / 5084; 300-token chunks of 16 requests and 16
// heads at 4096 tokens 215 / 252.  So from a mean of kWaveRows query tokens a request on.
constexpr int kMaxWaves = 64, kWaveBatch = 32, kWaveRows = 1536;
constexpr int64_t kWaveTokens = 128 << 10;
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
    // Plan
    Entry* entries;
    int64_t* cum;         // [E + 1] cost per head of the entries before each
    int* req_first;       // [batch + 1] first entry of each request
    int64_t* req_cum;     // [batch + 1] cost per head of the requests before each
    int max_entries;
    int* waves;           // whole items that a CTA takes first: c, c + CTAs, ...
    int64_t* starts;      // [CTAs + 1] cost before each CTA's share of the others
    int ctas;
    bool in_step;         // waves pay
    // Partials
    float* cut_o;         // [2 CTAs][slot_rows][128]
    float2* cut_ml;
    int4* cut_item;       // [CTAs][2]: row0, ntok, head, pieces; slots of the first piece and the second, entry
    uint32_t* odd;        // 32-row parts of whole items that are not finite: (entry * heads + head) * 8 + part
    int* num_odd;
    int slot_rows;
};

// S (+)= Q K^T over 64 channels: 16 of them are 32 bytes further in the rows.  By the whole warp, as the others.
__device__ __forceinline__ void mma_qk4(uint32_t d, uint32_t q_lo, uint32_t k_lo, uint32_t idesc, uint32_t acc, uint32_t go) {
    asm volatile(
        "{\n\t.reg .pred acc, yes, go;\n\t.reg .b32 al, bl;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.u32 acc, %6, 0;\n\tsetp.ne.u32 go, %7, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\t"
        SVQ_MMA_SS_IF(0, 0, acc) SVQ_MMA_SS_IF(2, 2, yes) SVQ_MMA_SS_IF(4, 4, yes) SVQ_MMA_SS_IF(6, 6, yes)
        "}" ::"r"(d), "r"(q_lo), "r"(k_lo), "r"(desc_hi(1024)), "r"(desc_hi(1024)), "r"(idesc), "r"(acc), "r"(go)
        : "memory");
}
// O (+)= P V over 64 tokens: 16 of them are 8 TMEM columns and 2 KB.
__device__ __forceinline__ void mma_pv4(uint32_t d, uint32_t p, uint32_t v_lo, uint32_t idesc, uint32_t acc, uint32_t go) {
    asm volatile(
        "{\n\t.reg .pred acc, yes, go;\n\t.reg .b32 al, bl;\n\t.reg .b64 bd;\n\t"
        "setp.ne.u32 acc, %5, 0;\n\tsetp.ne.u32 go, %6, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\t"
        SVQ_MMA_TS_IF(0, 0, acc) SVQ_MMA_TS_IF(8, 128, yes) SVQ_MMA_TS_IF(16, 256, yes) SVQ_MMA_TS_IF(24, 384, yes)
        "}" ::"r"(d), "r"(p), "r"(v_lo), "r"(desc_hi(1024)), "r"(idesc), "r"(acc), "r"(go)
        : "memory");
}
__device__ __forceinline__ void mma_pv1(uint32_t d, uint32_t p, uint32_t v_lo, uint32_t idesc, uint32_t acc, uint32_t go) {
    asm volatile(
        "{\n\t.reg .pred acc, go;\n\t.reg .b32 al, bl;\n\t.reg .b64 bd;\n\tsetp.ne.u32 acc, %5, 0;\n\tsetp.ne.u32 go, %6, 0;\n\t"
        SVQ_MMA_TS_IF(0, 0, acc)
        "}" ::"r"(d), "r"(p), "r"(v_lo), "r"(desc_hi(1024)), "r"(idesc), "r"(acc), "r"(go)
        : "memory");
}
// bf16 x bf16 -> fp32, M = 128, N = 128, A K-major; B K-major (keys) or N-major (values).
constexpr uint32_t kIdescQK = (1u << 4) | (1u << 7) | (1u << 10) | ((128u / 8) << 17) | ((128u / 16) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

// A run of key tiles of one item (entry, head); none: the CTA's work is over.
struct __align__(16) Seg {
    Entry en;
    int h;
    int t0, t1;
    int slot;         // where a partial goes; -1 - (entry * heads + head): the segment is the whole item
};
constexpr int kSegs = 4;

struct Control {
    uint64_t full[kBlocks], empty[kBlocks];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t s_full[2], p_full[2], o_full[2], q_full[2];
    uint64_t join[2];                 // both streams have published their statistics / have read O0 and O1
    uint64_t part, drain;
    uint32_t tmem;
    int gave_up;
    Seg seg[kSegs];
    float2 ml[2][128];                // stream statistics of a joined tile
};
static_assert(sizeof(Control) <= kControlBytes, "control block");

// The ring blocks of a segment of n tiles, three a key tile and two a value tile, in the order of their use.  Two row
// halves: K0 V0 K1 V1 ..; even and odd tiles: K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ uint32_t k_block(bool two, int t) { return two ? 5u * t : (t == 0 ? 0u : 5u * t - 2u); }
__device__ __forceinline__ uint32_t v_block(bool two, int t, int n) { return two ? 5u * t + 3u : (t == n - 1 ? 5u * n - 2u : 5u * t + 6u); }

__device__ __forceinline__ void gave_up(Control* ct) {
    svq_flag(SV_DEVERR_TIMEOUT);
    *static_cast<volatile int*>(&ct->gave_up) = 1;
}
constexpr int kSegRounds = 128;   // of kPolls: what the plan waits for a slot whose segment may be long

// Largest i in [0, n) with a[i] <= v (a ascending), by the whole warp (32 probes a round trip).
__device__ __forceinline__ int warp_find_le(const int64_t* a, int n, int64_t v) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane * step < len && a[at] <= v;
        const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;
        const int nlo = lo + max(k, 0) * step;
        len = min(step, lo + len - nlo);
        lo = nlo;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads, 1)
    expanded_kernel(const __grid_constant__ ExpandedArgs a, const __grid_constant__ CUtensorMap tmap_q,
                    const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_r,
                    const __grid_constant__ CUtensorMap tmap_v) {
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const ring = smem;
    unsigned char* const qs = smem + kBlocks * kBlock;
    Control* const ct = reinterpret_cast<Control*>(qs + 2 * kQBytes);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        ct->gave_up = 0;
        for (int i = 0; i < kBlocks; ++i) {
            mbar_init(smem_addr(&ct->full[i]), 1);
            mbar_init(smem_addr(&ct->empty[i]), 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_addr(&ct->s_full[w]), 1);
            mbar_init(smem_addr(&ct->p_full[w]), 4);
            mbar_init(smem_addr(&ct->o_full[w]), 1);
            mbar_init(smem_addr(&ct->q_full[w]), 1);
            mbar_init(smem_addr(&ct->join[w]), 256);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(smem_addr(&ct->seg_full[i]), 1);
            mbar_init(smem_addr(&ct->seg_empty[i]), 3 + 8);   // loads, MMAs, softmax
        }
        mbar_init(smem_addr(&ct->part), 1);
        mbar_init(smem_addr(&ct->drain), 1);
        mbar_init_fence();
        prefetch_tmap(&tmap_q);
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_r);
        prefetch_tmap(&tmap_v);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&ct->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    if (gridDim.x > 1) pdl_launch_dependents();   // the join, which waits (without one: the next call, which may not)
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(ct->tmem);
    // Every role takes the segments in order: the k-th is in slot k % kSegs.
    auto seg_done = [&](uint32_t k) {   // once a warp
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ct->seg_empty[k % kSegs]));
    };

    {
        if (warp == 0) {
            // ---------------- keys: three blocks a tile
            reg_dec<kOtherRegs>();
            uint32_t base = 0, issued = 0;   // blocks before the segment; the last one loaded here, plus 1
            for (uint32_t k = 0;; ++k) {
                TEST_WAIT(ct->seg_full[k % kSegs], (k / kSegs) & 1, keys_end);
                const Seg& s = ct->seg[k % kSegs];
                const int n = s.t1 - s.t0;
                if (n == 0) break;
                const bool two = s.en.ntok > 128;
                for (int i = 0; i < n; ++i) {
                    const int tok = s.en.kv0 + (s.t0 + i) * kTileTok;
#pragma unroll
                    for (int c = 0; c < 3; ++c) {
                        const uint32_t at = base + k_block(two, i) + c, st = at % kBlocks;
                        TEST_WAIT(ct->empty[st], ((at / kBlocks) & 1) ^ 1, keys_end);
                        if (lane == 0) {
                            const uint32_t bar = smem_addr(&ct->full[st]), dst = smem_addr(ring) + st * kBlock;
                            mbar_arrive_expect_tx(bar, kBlock);
                            if (c < 2) tma_load_3d(dst, &tmap_k, c * 64, tok, s.h, bar);
                            else tma_load_2d(dst, &tmap_r, 0, tok, bar);
                        }
                        issued = at + 1;
                    }
                }
                base += 5 * n;
                seg_done(k);
            }
            goto keys_done;   // every load has been waited for by the MMAs
        keys_end:
            // Gave up: the copies still in flight land before the CTA (and its shared memory) retires.  This warp's
            // last kBlocks blocks are waited for, in any case.
            for (uint32_t x = issued > kBlocks ? issued - kBlocks : 0; x < issued; ++x)
                (void)bar_wait(smem_addr(&ct->full[x % kBlocks]), (x / kBlocks) & 1);
        keys_done:;
        } else if (warp == 3) {
            // ---------------- values: two blocks of 64 tokens a tile
            reg_dec<kOtherRegs>();
            uint32_t base = 0, issued = 0, part_ph = 0;
            for (uint32_t k = 0;; ++k) {
                TEST_WAIT(ct->seg_full[k % kSegs], (k / kSegs) & 1, values_end);
                const Seg& s = ct->seg[k % kSegs];
                const int n = s.t1 - s.t0;
                if (n == 0) break;
                const bool two = s.en.ntok > 128;
                for (int i = 0; i < n; ++i) {
                    for (int c = 0; c < 2; ++c) {
                        const int first = (s.t0 + i) * kTileTok + c * 64;
                        const int here = s.en.len - first;          // tokens from here on
                        const uint32_t at = base + v_block(two, i, n) + c, st = at % kBlocks;
                        const uint32_t bar = smem_addr(&ct->full[st]), dst = smem_addr(ring) + st * kBlock;
                        TEST_WAIT(ct->empty[st], ((at / kBlocks) & 1) ^ 1, values_end);
                        const bool whole = here >= 64, some = here > 0;
                        const uint32_t on = whole ? bar : smem_addr(&ct->part);
                        if (lane == 0 && some) {
                            mbar_arrive_expect_tx(on, kBlock);
                            tma_load_3d(dst, &tmap_v, 0, s.en.kv0 + first, s.h, on);
                            tma_load_3d(dst + kBlock / 2, &tmap_v, 64, s.en.kv0 + first, s.h, on);
                        }
                        issued = at + 1;
                        if (!whole) {
                            // Rows behind the last token may hold anything; those that its product reads become
                            // zeros (P = 0 must not meet a NaN).
                            if (some) {
                                TEST_WAIT(ct->part, part_ph, values_end);
                                part_ph ^= 1;
                                const int end = (here + 15) / 16 * 16;
                                for (int x = here * 16 + lane; x < end * 16; x += 32)
                                    *reinterpret_cast<uint4*>(ring + st * kBlock + (x & 8) * (kBlock / 16) + (x >> 4) * 128 + (x & 7) * 16) =
                                        make_uint4(0u, 0u, 0u, 0u);
                                fence_proxy_async_smem();
                                __syncwarp();
                            }
                            if (lane == 0) mbar_arrive(bar);
                        }
                    }
                }
                base += 5 * n;
                seg_done(k);
            }
            goto values_done;
        values_end:
            for (uint32_t x = issued > kBlocks ? issued - kBlocks : 0; x < issued; ++x)
                (void)bar_wait(smem_addr(&ct->full[x % kBlocks]), (x / kBlocks) & 1);
        values_done:;
        } else if (warp == 1) {
            // ---------------- MMAs: the whole warp, in step
            reg_dec<kOtherRegs>();
            {
                const uint32_t go = elected();
                uint32_t ld = 0;
                uint32_t q_ph = 0, p_ph = 0;   // bit w: stream w's phase
                const uint32_t ring_s = smem_addr(ring), qs_s = smem_addr(qs);
                auto wait = [&](uint64_t& bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_ready(smem_addr(&bar), parity)) != 0; };
                auto commit = [&](uint64_t& bar) {
                    if (go) mma_commit(smem_addr(&bar));
                };
                auto ready = [&](uint32_t i) { return wait(ct->full[i % kBlocks], (i / kBlocks) & 1); };
                auto block = [&](uint32_t i) { return ring_s + i % kBlocks * kBlock; };
                auto release = [&](uint32_t i) { commit(ct->empty[i % kBlocks]); };
                // Blocks are waited for where a stream is the first to read them, and freed where one is the last.
                auto qk = [&](int w, uint32_t i, bool first, bool last) {
#pragma unroll
                    for (int c = 0; c < 3; ++c) {
                        if (first && !ready(i + c)) return false;
                        mma_qk4(tmem + kColS + w * 128, desc_lo(qs_s + w * kQBytes + c * kBlock, 16), desc_lo(block(i + c), 16),
                                kIdescQK, c != 0, go);
                        if (last) release(i + c);
                    }
                    commit(ct->s_full[w]);
                    return true;
                };
                // P V of stream w with the values in blocks i, i + 1, of which `steps` groups of 16 tokens count.
                auto pv = [&](int w, uint32_t i, int steps, bool acc, bool first, bool last) {
                    const uint32_t o = tmem + kColO + w * 128, p = tmem + kColS + w * 128;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (first && !ready(i + c)) return false;
                        const uint32_t v_lo = desc_lo(block(i + c), kBlock / 2);
                        if (steps >= 4 * c + 4) {
                            mma_pv4(o, p + c * 32, v_lo, kIdescPV, acc || c, go);
                        } else {
                            for (int u = 0; u < steps - 4 * c; ++u) mma_pv1(o, p + c * 32 + u * 8, v_lo + u * 128, kIdescPV, acc || c || u, go);
                        }
                        if (last) release(i + c);
                    }
                    return true;
                };
                auto p_ready = [&](int w) {
                    const bool r = wait(ct->p_full[w], (p_ph >> w) & 1);
                    p_ph ^= 1u << w;
                    tc_fence_after();
                    return r;
                };
                bool ok = true;
                for (uint32_t k = 0; ok; ++k) {
                    ok = wait(ct->seg_full[k % kSegs], (k / kSegs) & 1);
                    const Seg& s = ct->seg[k % kSegs];
                    const int n = uniform(s.t1 - s.t0);
                    if (!ok || n == 0) break;
                    const bool two = uniform(s.en.ntok) > 128;   // two row halves; else even and odd tiles
                    for (int w = 0; w < 2 && ok; ++w) {
                        const int t = two ? 0 : w;
                        if (t >= n) break;
                        ok = wait(ct->q_full[w], (q_ph >> w) & 1);
                        q_ph ^= 1u << w;
                        if (!ok) break;
                        tc_fence_after();
                        ok = qk(w, ld + k_block(two, t), !two || w == 0, !two || w == 1);
                    }
                    int steps = uniform((s.en.len - s.t0 * kTileTok + 15) / 16);   // groups of 16 tokens from the tile on
                    if (two) {
                        for (int t = 0; t < n && ok; ++t, steps -= 8) {
                            const bool next = t + 1 < n;
                            const uint32_t vl = ld + v_block(true, t, n), kl = ld + k_block(true, t + 1);
                            const bool acc = (t & (kFoldTiles - 1)) != 0;
                            ok = p_ready(0) && pv(0, vl, steps, acc, true, false);
                            if (!ok) break;
                            if (next) ok = qk(0, kl, true, false);
                            else commit(ct->o_full[0]);
                            ok = ok && p_ready(1);
                            if (!ok) break;
                            pv(1, vl, steps, acc, false, true);
                            if (next) qk(1, kl, false, true);
                            else commit(ct->o_full[1]);
                        }
                    } else {
                        for (int t = 0; t < n && ok; ++t, steps -= 8) {
                            const int w = t & 1;
                            ok = p_ready(w) && pv(w, ld + v_block(false, t, n), steps, ((t >> 1) & (kFoldTiles - 1)) != 0, true, true);
                            if (!ok) break;
                            if (t + 2 < n) ok = qk(w, ld + k_block(false, t + 2), true, true);
                            else commit(ct->o_full[w]);
                        }
                    }
                    ld += 5 * n;
                    if (ok && go) mbar_arrive(smem_addr(&ct->seg_empty[k % kSegs]));
                }
                if (!ok && go) gave_up(ct);
                commit(ct->drain);   // nothing of this CTA's is in flight when TMEM is freed
                (void)wait(ct->drain, 0);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ---------------- the CTA's share of the plan, segment by segment
            reg_dec<kOtherRegs>();
            const int waves = *a.waves;
            const int64_t first = a.starts[blockIdx.x];
            int64_t left = a.starts[blockIdx.x + 1] - first;
            int b = 0, h = 0, e = 0, e0 = 0, e1 = 0;   // request, head, entry, the request's entries
            int64_t off = 0, into = 0;                 // into the item's cost; where the share begins
            bool first_item = true;
            Entry en;
            uint32_t k = 0;
            auto fetch = [&](int e) {
                const int4* p = reinterpret_cast<const int4*>(a.entries + e);
                const int4 x = p[0], y = p[1];
                return Entry{x.x, x.y, x.z, x.w, y.x, y.y, {0, 0}};
            };
            auto publish = [&](int t0, int t1, int slot) {   // false: gave up
                for (int round = 0;; ++round) {
                    if (!__any_sync(0xffffffffu, !bar_wait(smem_addr(&ct->seg_empty[k % kSegs]), ((k / kSegs) & 1) ^ 1))) break;
                    if (__any_sync(0xffffffffu, *static_cast<volatile int*>(&ct->gave_up)) || round == kSegRounds) {
                        if (lane == 0) gave_up(ct);
                        return false;
                    }
                }
                if (lane == 0) {
                    Seg& s = ct->seg[k % kSegs];
                    s.en = en;
                    s.h = h;
                    s.t0 = t0;
                    s.t1 = t1;
                    s.slot = slot;
                    mbar_arrive(smem_addr(&ct->seg_full[k % kSegs]));
                }
                ++k;
                return true;
            };
            // (A CTA that gives up in its waves names no item for the join.)
            if (lane == 0) a.cut_item[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
            for (int64_t j = 0, i = blockIdx.x; j < waves; ++j, i += gridDim.x) {
                while (i >= static_cast<int64_t>(a.heads) * a.req_first[b + 1]) ++b;
                e0 = a.req_first[b];
                const int64_t in = i - static_cast<int64_t>(a.heads) * e0, n = a.req_first[b + 1] - e0;
                h = static_cast<int>(div64(in, n));
                e = e0 + static_cast<int>(in - h * n);
                en = fetch(e);
                if (en.tiles && !publish(0, en.tiles, -1 - (e * a.heads + h))) goto plan_end;
            }
            if (left > 0) {
                const int64_t u = div64(first, a.heads);
                b = warp_find_le(a.req_cum, a.batch, u);
                e0 = a.req_first[b];
                e1 = a.req_first[b + 1];
                const int64_t c0 = a.req_cum[b], in = first - c0 * a.heads, one = a.req_cum[b + 1] - c0;
                h = static_cast<int>(div64(in, one));
                off = in - h * one;
                e = e0 + warp_find_le(a.cum + e0, e1 - e0, c0 + off);
                off -= a.cum[e] - c0;
                into = off;
                en = fetch(e);
            }
            {
                // The CTA after the one with an item's first tile names the item for the join.
                int4 what = make_int4(0, 0, 0, 0), where = make_int4(0, 0, 0, 0);
                if (into > 0) {
                    const int64_t begin = first - into;
                    const int c0 = warp_find_le(a.starts, gridDim.x, begin + kItemCost);
                    if (static_cast<int>(blockIdx.x) == c0 + 1) {
                        const int c1 = warp_find_le(a.starts, gridDim.x, begin + kItemCost + en.tiles - 1);
                        what = make_int4(en.row0, en.ntok, h, c1 - c0 + 1);
                        where.x = 2 * c0 + (a.starts[c0] >= begin ? 0 : 1);
                        where.y = 2 * (c0 + 1);
                        where.z = e;
                    }
                }
                if (lane == 0) {
                    a.cut_item[2 * blockIdx.x] = what;
                    a.cut_item[2 * blockIdx.x + 1] = where;
                }
            }
            for (;;) {
                int t0 = 0, t1 = 0;
                if (left > 0) {
                    const int64_t take = min(left, cost_of(en.tiles) - off);
                    t0 = static_cast<int>(max(static_cast<int64_t>(0), off - kItemCost));
                    t1 = static_cast<int>(max(static_cast<int64_t>(0), off + take - kItemCost));
                    left -= take;
                    off += take;
                }
                if (t1 > t0 || left <= 0) {
                    const bool whole = t0 == 0 && t1 == en.tiles;
                    if (!publish(t0, t1, whole ? -1 - (e * a.heads + h) : static_cast<int>(blockIdx.x) * 2 + (first_item ? 0 : 1))) break;
                    if (t1 == t0) break;
                }
                first_item = false;
                if (left > 0 && off == cost_of(en.tiles)) {
                    off = 0;
                    if (++e == e1) {   // the next head, or the next request with tokens
                        e = e0;
                        if (++h == a.heads) {
                            h = 0;
                            do ++b;
                            while (a.req_cum[b + 1] == a.req_cum[b]);
                            e = e0 = a.req_first[b];
                            e1 = a.req_first[b + 1];
                        }
                    }
                    en = fetch(e);
                }
            }
        plan_end:;
        } else {
            // ---------------- softmax: warps 4-7 stream 0, warps 8-11 stream 1
            reg_inc<kSoftmaxRegs>();
            const int w = (warp - 4) >> 2;
            const int row = (warp & 3) * 32 + lane;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t s_col = tmem + lanes + kColS + w * 128;
            const uint32_t o_col = tmem + lanes + kColO + w * 128;
            uint32_t s_ph = 0, o_ph0 = 0, o_ph1 = 0, join_ph = 0, q_loads = 0;
            auto stream_tiles = [&](const Seg& g) {
                const int n = g.t1 - g.t0;
                return g.en.ntok > 128 ? n : (n - w + 1) / 2;
            };
            // The stream's 128 rows of Q: three blocks of 64 channels.
            auto load_q = [&](const Seg& g) {
                if (row == 0) {
                    const uint32_t bar = smem_addr(&ct->q_full[w]), dst = smem_addr(qs) + w * kQBytes;
                    const int tok = g.en.row0 + (g.en.ntok > 128 ? w * 128 : 0);
                    mbar_arrive_expect_tx(bar, kQBytes);
                    ++q_loads;
#pragma unroll
                    for (int c = 0; c < 3; ++c) tma_load_3d(dst + c * kBlock, &tmap_q, c * 64, g.h, tok, bar);
                }
            };
            for (uint32_t k = 0;; ++k) {
                const Seg& s = ct->seg[k % kSegs];
                if (k == 0) {
                    TEST_WAIT(ct->seg_full[0], 0, softmax_end);
                    if (stream_tiles(s) > 0) load_q(s);
                }
                const int n = s.t1 - s.t0;
                if (n == 0) break;
                TEST_WAIT(ct->seg_full[(k + 1) % kSegs], ((k + 1) / kSegs) & 1, softmax_end);
                const Seg& nx = ct->seg[(k + 1) % kSegs];
                const bool next_q = stream_tiles(nx) > 0;
                const int rows = s.en.ntok;
                const bool two = rows > 128;
                const int nt = stream_tiles(s);
                const int off = two ? w * 128 : 0;
                const int r = off + row;
                const bool valid = r < rows;
                const bool warp_on = off + (warp & 3) * 32 < rows;
                const bool all = s.en.pos0 == kAllVisible;
                // Tokens that this row sees, and that every row of the warp's stream half does.
                const int see = all ? s.en.len : s.en.pos0 + min(r, rows - 1) + 1;
                const int see_all = all ? s.en.len : s.en.pos0 + off + 1;
                float m = -INFINITY, l = 0.f;
                // The row's place for what is folded: that of the segment's partial; a whole item's CTA has not
                // written its second one yet.  (Base, sum) are kept in ct->ml.
                auto folded = [&] {
                    const int slot = s.slot >= 0 ? s.slot : 2 * static_cast<int>(blockIdx.x) + 1;
                    return a.cut_o + (static_cast<int64_t>(slot) * a.slot_rows + (two ? r : w * (a.slot_rows / 2) + row)) * kHeadDim;
                };
                for (int j0 = 0; j0 < nt; j0 += kFoldTiles) {
                    if (j0 > 0) {
                        TEST_WAIT(ct->s_full[w], s_ph, softmax_end);   // O is complete, and the next product into it starts anew
                        if (warp_on) fold_out(o_col, folded(), valid, j0 > kFoldTiles, ct->ml[w][row], m, l);
                        l = 0.f;
                    }
                    for (int j = j0; j < min(nt, j0 + kFoldTiles); ++j) {
                        const int ti = two ? j : 2 * j + w;          // tile of the segment
                        const int base_tok = (s.t0 + ti) * kTileTok;
                        TEST_WAIT(ct->s_full[w], s_ph, softmax_end);
                        s_ph ^= 1;
                        tc_fence_after();
                        if (j == nt - 1 && next_q) load_q(nx);       // the stream's last use of Q is over
                        if (warp_on) {
                            float x[128];
#pragma unroll
                            for (int c = 0; c < 4; ++c) tc_ld32(s_col + c * 32, reinterpret_cast<uint32_t(&)[32]>(x[c * 32]));
                            tc_wait_ld();
                            if (base_tok + kTileTok > see_all) {
                                const int lim = see - base_tok;
#pragma unroll
                                for (int c = 0; c < 128; ++c)
                                    if (c >= lim) x[c] = -INFINITY;
                            }
                            float mx[4];
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                mx[c] = fmaxf(x[c], x[c + 4]);
#pragma unroll
                                for (int u = 8; u < 128; u += 8) mx[c] = fmaxf(fmaxf(mx[c], x[u + c]), x[u + c + 4]);
                            }
                            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                            // The base moves only when the maximum is more than kSlack above it; weights stay at most
                            // 2^kSlack, and sums and outputs share the base.  Threads without a row have no say.
                            if (__any_sync(0xffffffffu, valid && top > m + kSlack)) {
                                const float mn = fmaxf(m, top);
                                const float alpha = mn == -INFINITY ? 1.f : ex2(m - mn);
                                m = mn;
                                l *= alpha;
                                if (j > 0) {   // S of this tile is complete, so the MMAs into O before it are
#pragma unroll 1
                                    for (int c = 0; c < 8; ++c) {
                                        uint32_t y[16];
                                        tc_ld16(o_col + c * 16, y);
                                        tc_wait_ld();
#pragma unroll
                                        for (int u = 0; u < 16; ++u) y[u] = __float_as_uint(__uint_as_float(y[u]) * alpha);
                                        tc_st16(o_col + c * 16, y);
                                    }
                                }
                            }
                            const float base = m == -INFINITY ? 0.f : m;
                            // Weights and their sum, two at a time, and P in bf16 over S (read already).
                            const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), base2 = pack2(-base, -base);
                            uint64_t sum[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                uint32_t p[16];
#pragma unroll
                                for (int u = 0; u < 16; ++u) {
                                    float e0, e1;
                                    unpack2(fma2(pack2(x[c * 32 + 2 * u], x[c * 32 + 2 * u + 1]), scale2, base2), e0, e1);
                                    e0 = ex2(e0);
                                    e1 = ex2(e1);
                                    sum[u & 3] = add2(sum[u & 3], pack2(e0, e1));
                                    p[u] = pack_bf16x2(e0, e1);
                                }
                                tc_st16(s_col + c * 16, p);
                            }
                            float s0, s1;
                            unpack2(add2(add2(sum[0], sum[2]), add2(sum[1], sum[3])), s0, s1);
                            l += s0 + s1;
                            tc_wait_st();
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&ct->p_full[w]));
                    }
                }
                if (nt == 0 && next_q) load_q(nx);

                // ---------------- the segment's end
                float* po = nullptr;        // this row's fp32 partial
                float2* pml = nullptr;
                const int64_t qrow = static_cast<int64_t>(s.en.row0 + r) * a.heads + s.h;
                if (s.slot >= 0) {
                    const int64_t at = static_cast<int64_t>(s.slot) * a.slot_rows + r;
                    po = a.cut_o + at * kHeadDim;
                    pml = a.cut_ml + at;
                }
                float f0 = 1.f, f1 = 0.f;   // factors of O0 and O1 (f0: of the own O when there are two row halves)
                float M = m, L = l;
                if (two) {
                    TEST_WAIT(ct->o_full[w], w ? o_ph1 : o_ph0, softmax_end);
                    o_ph0 ^= 1;
                    o_ph1 ^= 1;
                    if (nt > kFoldTiles && warp_on) L = l = fold_in(o_col, folded(), valid, ct->ml[w][row], m, l);
                } else {
                    TEST_WAIT(ct->o_full[0], o_ph0, softmax_end);
                    o_ph0 ^= 1;
                    if (n > 1) {
                        TEST_WAIT(ct->o_full[1], o_ph1, softmax_end);
                        o_ph1 ^= 1;
                    }
                    if (nt > kFoldTiles && warp_on) l = fold_in(o_col, folded(), valid, ct->ml[w][row], m, l);
                    ct->ml[w][row] = make_float2(m, l);
                    mbar_arrive(smem_addr(&ct->join[0]));
                    TEST_WAIT(ct->join[0], join_ph, softmax_end);
                    const float2 other = ct->ml[1 - w][row];
                    M = fmaxf(m, other.x);
                    const float mine = M == -INFINITY ? 0.f : ex2(m - M), theirs = M == -INFINITY ? 0.f : ex2(other.x - M);
                    L = l * mine + other.y * theirs;
                    f0 = w == 0 ? mine : theirs;
                    f1 = w == 0 ? theirs : mine;
                }
                tc_fence_after();
                if (warp_on) {
                    const float inv = po ? 1.f : (L > 0.f ? 1.f / L : L);
                    f0 *= inv;
                    f1 *= inv;
                    float odd = 0.f;   // NaN once a channel of the row is not finite
                    // Two halves: the whole row of the own stream.  Joined: 64 channels of both.
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        if (!two && (c >> 1) != w) continue;
                        uint32_t x[32];
                        tc_ld32(tmem + lanes + (two ? kColO + w * 128 : kColO) + c * 32, x);
                        tc_wait_ld();
#pragma unroll
                        for (int u = 0; u < 32; ++u) x[u] = __float_as_uint(__uint_as_float(x[u]) * f0);
                        if (!two && n > 1) {
                            uint32_t y[32];
                            tc_ld32(tmem + lanes + kColO + 128 + c * 32, y);
                            tc_wait_ld();
#pragma unroll
                            for (int u = 0; u < 32; ++u)
                                x[u] = __float_as_uint(fmaf(__uint_as_float(y[u]), f1, __uint_as_float(x[u])));
                        }
                        if (valid) {
                            if (po) {
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    st_v8(po + c * 32 + 8 * u, x[8 * u], x[8 * u + 1], x[8 * u + 2], x[8 * u + 3], x[8 * u + 4],
                                          x[8 * u + 5], x[8 * u + 6], x[8 * u + 7]);
                            } else {
                                uint32_t v[16];
#pragma unroll
                                for (int u = 0; u < 32; ++u) odd = fmaf(__uint_as_float(x[u]), 0.f, odd);
#pragma unroll
                                for (int u = 0; u < 16; ++u)   // (a row that sees nothing is 0, whatever the others see)
                                    v[u] = L == 0.f ? 0u : pack_bf16x2(__uint_as_float(x[2 * u]), __uint_as_float(x[2 * u + 1]));
#pragma unroll
                                for (int u = 0; u < 2; ++u)
                                    st_v8(a.out + qrow * kHeadDim + c * 32 + 16 * u, v[8 * u], v[8 * u + 1], v[8 * u + 2],
                                          v[8 * u + 3], v[8 * u + 4], v[8 * u + 5], v[8 * u + 6], v[8 * u + 7]);
                            }
                        }
                    }
                    if (!po && __any_sync(0xffffffffu, odd != 0.f && L > 0.f && L < INFINITY) && lane == 0)
                        a.odd[atomicAdd(a.num_odd, 1)] = static_cast<uint32_t>(~s.slot) * 8 + (warp - 4 - (two ? 0 : w * 4));
                    if (valid && (two || w == 0)) {
                        if (po) *pml = make_float2(M, L);
                        else a.lse[qrow] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : (L == 0.f ? -INFINITY : L);
                    }
                }
                // Joined tiles: both halves of the CTA have read O0 and O1 before either is written again.
                tc_fence_before();
                if (!two) {
                    mbar_arrive(smem_addr(&ct->join[1]));
                    TEST_WAIT(ct->join[1], join_ph, softmax_end);
                    join_ph ^= 1;
                }
                seg_done(k);
            }
        softmax_end:
            // (Gave up: the rows in flight land before the CTA retires.)
            if (row == 0 && q_loads) (void)bar_wait(smem_addr(&ct->q_full[w]), (q_loads - 1) & 1);
        }
    }
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------- plan
// Few threads where a thread each is enough: 1024 of them take 0.7 us longer to start and to meet (300 tokens 21.4 -> 20.7).
constexpr int kPlanThreads = 1024, kFewPlanThreads = 256;
static_assert(kMaxCtas <= kFewPlanThreads, "a thread a CTA");

// The tokens of request b's range: false for ranges that are none.
__device__ __forceinline__ bool kv_range(const ExpandedArgs& a, int b, int size, int& k0, int& n) {
    k0 = a.kv_start[b];
    const int k1 = a.kv_start[b + 1];
    n = 0;
    if (k0 < 0 || k1 < k0 || k1 > a.total_kv) return false;
    if (a.causal && k1 > k0 && size > k1 - k0) return false;
    n = k1 - k0;
    return true;
}

// One CTA: the list of entries, and the running sums of their costs.
__global__ void __launch_bounds__(kPlanThreads) expanded_plan_kernel(const __grid_constant__ ExpandedArgs a) {
    __shared__ int64_t warp_sums[32];
    __shared__ int most_waves;
    const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
    int64_t total;
    pdl_wait();   // the workspace may still be read by the call before
    if (a.total_kv > 0) pdl_launch_dependents();   // the tiles, which wait (else this kernel's rows are the results)
    int n = 0;
    for (int i0 = 0; i0 < a.batch; i0 += threads) {
        const int i = i0 + tid;
        int count = 0;
        if (i < a.batch) {
            const int q0 = a.q_start[i], q1 = a.q_start[i + 1];
            if (q0 < 0 || q1 < q0 || q1 > a.total_q) svq_flag(SV_DEVERR_Q_START);
            else count = (q1 - q0 + kRowTile - 1) / kRowTile;
        }
        const int64_t before = n + block_scan(count, warp_sums, total);
        // (Broken starts that overlap could list more entries than the workspace holds.)
        if (i < a.batch) a.req_first[i] = static_cast<int>(min(before, static_cast<int64_t>(a.max_entries)));
        n = static_cast<int>(min(n + total, static_cast<int64_t>(INT_MAX / 2)));
    }
    if (n > a.max_entries) {
        if (tid == 0) svq_flag(SV_DEVERR_Q_START);
        n = a.max_entries;
    }
    if (tid == 0) a.req_first[a.batch] = n;
    __syncthreads();
    int64_t base = 0;
    for (int e0 = 0; e0 < n; e0 += threads) {
        const int e = e0 + tid;
        Entry en = {0, 0, 0, 0, 0, 0, {0, 0}};
        bool empty = false;   // rows that see nothing
        if (e < n) {
            const int b = find_le(a.req_first, a.batch, e);
            const int start = a.q_start[b], size = a.q_start[b + 1] - start;
            const int at = (e - a.req_first[b]) * kRowTile;
            int tokens;
            if (!kv_range(a, b, size, en.kv0, tokens)) svq_flag(SV_DEVERR_Q_START);
            en.row0 = start + at;
            en.ntok = min(kRowTile, size - at);
            en.pos0 = a.causal ? tokens - size + at : kAllVisible;
            en.len = a.causal && tokens ? en.pos0 + en.ntok : tokens;
            empty = tokens == 0;
        }
        en.tiles = (en.len + kTileTok - 1) / kTileTok;
        const int64_t before = base + block_scan(cost_of(en.tiles), warp_sums, total);
        base += total;
        if (e < n) {
            a.entries[e] = en;
            a.cum[e] = before;
        }
        for (uint32_t rest = __ballot_sync(0xffffffffu, empty); rest; rest &= rest - 1) {
            const int src = __ffs(rest) - 1;
            const int64_t r0 = static_cast<int64_t>(__shfl_sync(0xffffffffu, en.row0, src)) * a.heads;
            const int64_t r1 = r0 + static_cast<int64_t>(__shfl_sync(0xffffffffu, en.ntok, src)) * a.heads;
            uint4* o = reinterpret_cast<uint4*>(a.out + r0 * kHeadDim);
            for (int64_t i = lane; i < (r1 - r0) * (kHeadDim / 8); i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int64_t i = r0 + lane; i < r1; i += 32) a.lse[i] = -INFINITY;
        }
    }
    if (tid == 0) {
        a.cum[n] = base;
        *a.num_odd = 0;
    }
    __syncthreads();
    for (int i = tid; i <= a.batch; i += threads) a.req_cum[i] = a.cum[a.req_first[i]];

    // Thread c: the shares of CTA c.  Whole items first, the waves, and of the others what makes its share equal.
    const int64_t cost = base * a.heads, items = static_cast<int64_t>(n) * a.heads;
    const Share share(cost, a.ctas);
    const int64_t equal = tid < a.ctas ? share.start(tid + 1) - share.start(tid) : 0;
    int waves = a.in_step ? static_cast<int>(min(items / a.ctas, static_cast<int64_t>(kMaxWaves))) : 0;
    if (!waves) {
        if (tid < a.ctas) a.starts[tid] = share.start(tid);
        if (tid == 0) {
            a.starts[a.ctas] = cost;
            *a.waves = 0;
        }
        __threadfence();
        return;
    }
    // Costs only add up, so the waves that fit are the fewest that fit a thread's share, each thread going through its own
    // items once.  (Looking from the most waves down, each time through all of them, took 140 us of 930 for 32 requests of
    // 1024 tokens and 64 heads.)
    auto first_items = [&](int most, int64_t limit, int64_t& sum) {   // how many of them stay within the limit; their cost
        int b = 0, j = 0;
        sum = 0;
        for (int64_t i = tid; j < most; ++j, i += a.ctas) {
            while (i >= static_cast<int64_t>(a.heads) * a.req_first[b + 1]) ++b;
            const int e0 = a.req_first[b];
            const int64_t in = i - static_cast<int64_t>(a.heads) * e0, entries = a.req_first[b + 1] - e0;
            const int e = e0 + static_cast<int>(in - div64(in, entries) * entries);
            const int64_t more = sum + a.cum[e + 1] - a.cum[e];
            if (more > limit) break;
            sum = more;
        }
        return j;
    };
    int64_t mine = 0, whole;          // of the thread's waves; of all
    if (tid == 0) most_waves = waves;
    __syncthreads();
    if (tid < a.ctas) {
        const int fit = first_items(waves, equal - 1, mine);
        if (fit < waves) atomicMin(&most_waves, fit);
    }
    __syncthreads();
    waves = most_waves;
    if (tid < a.ctas) (void)first_items(waves, equal, mine);
    const int64_t len = equal - mine;
    (void)block_scan(mine, warp_sums, whole);
    const int64_t before = whole + block_scan(len, warp_sums, total);
    if (tid < a.ctas) a.starts[tid] = before;
    if (tid == 0) {
        a.starts[a.ctas] = cost;
        *a.waves = waves;
    }
    __threadfence();
}

// ---------------------------------------------------------------- joining partials
// A row of an entry whose outputs may not be finite, by one warp.  The tile's
// product multiplies every value of the tile with a weight, and a weight 0 does
// not hide an infinite or NaN value from the rows that do not see its token.  So
// if the row's logits are finite, its outputs are not, and a token that other
// rows of the entry see and this one does not holds such a value, the row is
// computed again from its own tokens alone.
__device__ __noinline__ void look_at_row(const ExpandedArgs& a, int entry, int h, int r) {
    const int lane = threadIdx.x & 31;
    const Entry en = a.entries[entry];
    if (en.pos0 == kAllVisible) return;   // its rows see the same tokens
    const int end = en.pos0 + r + 1;
    const int64_t qrow = static_cast<int64_t>(en.row0 + r) * a.heads + h;
    const uint2 w = *reinterpret_cast<const uint2*>(a.out + qrow * kHeadDim + 4 * lane);
    const float4 got = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
    {
        const float odd = fmaf(got.x, 0.f, fmaf(got.y, 0.f, fmaf(got.z, 0.f, got.w * 0.f)));
        if (!(fabsf(a.lse[qrow]) < INFINITY) || !__any_sync(0xffffffffu, odd != 0.f)) return;
    }
    auto value = [&](int t) {
        const uint2 x = *reinterpret_cast<const uint2*>(a.v + (en.kv0 + static_cast<int64_t>(t)) * a.v_stride + h * a.v_head_stride + 4 * lane);
        return make_float4(bf16lo(x.x), bf16hi(x.x), bf16lo(x.y), bf16hi(x.y));
    };
    {
        // The row's own token is NaN wherever the row is not finite (all tokens are NaN): so is the result.
        const float4 v = value(end - 1);
        const bool known = (v.x != v.x || got.x * 0.f == 0.f) && (v.y != v.y || got.y * 0.f == 0.f) &&
                           (v.z != v.z || got.z * 0.f == 0.f) && (v.w != v.w || got.w * 0.f == 0.f);
        if (__all_sync(0xffffffffu, known)) return;
    }
    float odd = 0.f;   // of the tokens that other rows see and this one does not
    for (int t = end; t < en.len; ++t) {
        const float4 v = value(t);
        odd = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, odd))));
    }
    if (!__any_sync(0xffffffffu, odd != 0.f)) return;   // the row's own tokens gave it
    const __nv_bfloat16* const qr = a.q + qrow * kQueryDim;
    const uint2 qa = *reinterpret_cast<const uint2*>(qr + 4 * lane);
    const uint32_t qb = *reinterpret_cast<const uint32_t*>(qr + kHeadDim + 2 * lane);
    RowSum s;
    for (int j = 0; j < end; ++j) {
        const int64_t t = en.kv0 + static_cast<int64_t>(j);
        const uint2 ka = *reinterpret_cast<const uint2*>(a.k + t * a.k_stride + h * a.k_head_stride + 4 * lane);
        const uint32_t kb = *reinterpret_cast<const uint32_t*>(a.rope + t * a.rope_stride + 2 * lane);
        float z = bf16lo(qa.x) * bf16lo(ka.x) + bf16hi(qa.x) * bf16hi(ka.x) + bf16lo(qa.y) * bf16lo(ka.y) +
                  bf16hi(qa.y) * bf16hi(ka.y) + bf16lo(qb) * bf16lo(kb) + bf16hi(qb) * bf16hi(kb);
#pragma unroll
        for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        s.join(RowSum{z * a.scale_log2, 1.f, value(j)});
    }
    (void)s.write(a.out + qrow * kHeadDim, a.lse + qrow, lane);
}

// CTA (c, y) joins the item that CTA c + 1 of the tiles goes on with; rows y,
// y + gridDim.y, ... (of 8 warps each, when the pieces are few).  Then the parts
// of whole items with rows that are not finite.
constexpr int kCutThreads = 256;

__global__ void __launch_bounds__(kCutThreads, 4) expanded_join_kernel(const __grid_constant__ ExpandedArgs a) {
    constexpr int kWarps = kCutThreads / 32;
    __shared__ float4 sm_o[kWarps][32];
    __shared__ float2 sm_ml[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const int4 what = a.cut_item[2 * (blockIdx.x + 1)];
    const int num_odd = *a.num_odd;
    const int n = what.w;
    if (n == 0 && num_odd == 0) return;
    const int4 where = n ? a.cut_item[2 * (blockIdx.x + 1) + 1] : what;
    const int rows = n ? what.y : 0;
    auto at_row = [&](int r) { return static_cast<int64_t>(what.x + r) * a.heads + what.z; };
    auto pieces = [&](int r) {
        return Pieces{a.cut_o, a.cut_ml, static_cast<int64_t>(where.x) * a.slot_rows + r,
                      static_cast<int64_t>(where.y) * a.slot_rows + r, 2ll * a.slot_rows, n};
    };
    bool odd = false;
    if (n <= 8) {   // few pieces: a warp a row
        for (int r = blockIdx.y * kWarps + warp; r < rows; r += gridDim.y * kWarps) {
            RowSum s;
            s.add(pieces(r), 0, 1, lane);
            odd |= s.write(a.out + at_row(r) * kHeadDim, a.lse + at_row(r), lane);
        }
    } else {
        for (int r = blockIdx.y; r < rows; r += gridDim.y)
            odd |= join_row<kWarps>(pieces(r), sm_o, sm_ml, a.out + at_row(r) * kHeadDim, a.lse + at_row(r));
    }
    if (__any_sync(0xffffffffu, odd)) {   // of the rows this warp wrote
        __syncwarp();                     // (their lse by its first lane)
        for (int r = n <= 8 ? blockIdx.y * kWarps + warp : blockIdx.y; r < rows; r += n <= 8 ? gridDim.y * kWarps : gridDim.y)
            look_at_row(a, where.z, what.z, r);
    }
    constexpr int kTurns = 32 / kWarps;   // a warp a row
    for (int64_t i = blockIdx.y * gridDim.x + blockIdx.x; i < static_cast<int64_t>(num_odd) * kTurns; i += gridDim.x * gridDim.y) {
        const uint32_t part = a.odd[i / kTurns];
        const int e = part / 8 / a.heads, h = part / 8 % a.heads;
        const int r = part % 8 * 32 + static_cast<int>(i % kTurns) * kWarps + warp;
        if (r < a.entries[e].ntok) look_at_row(a, e, h, r);
    }
    __threadfence();
}

// ---------------------------------------------------------------- host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
    size_t entries, cum, waves, starts, req_first, req_cum, cut_item, cut_o, cut_ml, odd, num_odd, total;
    int max_entries, item_rows, slot_rows;
    Layout(int64_t batch, int64_t rows, int heads) {
        const int64_t e = rows / kRowTile + batch;
        max_entries = static_cast<int>(e);
        item_rows = static_cast<int>(rows < kRowTile ? rows : kRowTile);
        slot_rows = 2 * item_rows < kRowTile ? 2 * item_rows : kRowTile;   // (both streams of up to 128 rows fold theirs)
        size_t at = 0;
        auto take = [&](size_t bytes) { const size_t r = at; at += up(bytes); return r; };
        entries = take(e * sizeof(Entry));
        cum = take((e + 1) * sizeof(int64_t));
        waves = take(sizeof(int));
        starts = take((kMaxCtas + 1) * sizeof(int64_t));
        req_first = take((batch + 1) * sizeof(int));
        req_cum = take((batch + 1) * sizeof(int64_t));
        cut_item = take(2 * kMaxCtas * sizeof(int4));
        cut_o = take(2ull * kMaxCtas * slot_rows * kHeadDim * sizeof(float));
        cut_ml = take(2ull * kMaxCtas * slot_rows * sizeof(float2));
        odd = take(8ull * e * heads * sizeof(uint32_t));
        num_odd = take(sizeof(int));
        total = at + 256;   // the parts begin at the workspace's first multiple of 256 (rows are written 32 bytes at a time)
    }
};

// bf16 rows in blocks of 64 channels, 128-byte swizzled: dims (channels, n1, n2), strides in elements of n1 and n2, box
// (64, b1, b2).  n2 == 0: two dimensions.
bool encode_rows(CUtensorMap* map, const void* p, int channels, int64_t n1, int64_t s1, int b1, int64_t n2, int64_t s2, int b2) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_entry());
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(channels), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
    const cuuint32_t ones[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n2 ? 3 : 2, const_cast<void*>(p), dims, strides, box, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t expanded_workspace_bytes(int batch, int num_heads, int total_q) { return Layout(batch, total_q, num_heads).total; }

int launch_expanded(const void* q, int num_heads, const int32_t* q_start, int total_q, const void* k, int64_t k_stride,
                    int64_t k_head_stride, const void* rope, int64_t rope_stride, const void* v, int64_t v_stride,
                    int64_t v_head_stride, const int32_t* kv_start, int total_kv, int batch, bool causal,
                    float softmax_scale, void* out, float* lse, void* workspace, int sm_count, cudaStream_t stream) {
    const Layout lay(batch, total_q, num_heads);
    unsigned char* const ws =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
    ExpandedArgs a = {};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.heads = num_heads;
    a.q_start = q_start;
    a.total_q = total_q;
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.k_stride = k_stride;
    a.k_head_stride = k_head_stride;
    a.rope = static_cast<const __nv_bfloat16*>(rope);
    a.rope_stride = rope_stride;
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.v_stride = v_stride;
    a.v_head_stride = v_head_stride;
    a.kv_start = kv_start;
    a.total_kv = total_kv;
    a.batch = batch;
    a.causal = causal;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.entries = reinterpret_cast<Entry*>(ws + lay.entries);
    a.cum = reinterpret_cast<int64_t*>(ws + lay.cum);
    a.waves = reinterpret_cast<int*>(ws + lay.waves);
    a.starts = reinterpret_cast<int64_t*>(ws + lay.starts);
    a.ctas = sm_count < kMaxCtas ? sm_count : kMaxCtas;
    a.in_step = batch <= kWaveBatch && total_q >= static_cast<int64_t>(kWaveRows) * batch &&
                static_cast<int64_t>(total_kv) * num_heads >= kWaveTokens;
    a.req_first = reinterpret_cast<int*>(ws + lay.req_first);
    a.req_cum = reinterpret_cast<int64_t*>(ws + lay.req_cum);
    a.max_entries = lay.max_entries;
    a.cut_o = reinterpret_cast<float*>(ws + lay.cut_o);
    a.cut_ml = reinterpret_cast<float2*>(ws + lay.cut_ml);
    a.cut_item = reinterpret_cast<int4*>(ws + lay.cut_item);
    a.odd = reinterpret_cast<uint32_t*>(ws + lay.odd);
    a.num_odd = reinterpret_cast<int*>(ws + lay.num_odd);
    a.slot_rows = lay.slot_rows;
    const int plan_threads = lay.max_entries <= kFewPlanThreads ? kFewPlanThreads : kPlanThreads;
    if (launch_pdl(expanded_plan_kernel, dim3(1), dim3(plan_threads), 0, stream, a) != cudaSuccess) return SV_ERR_CUDA;
    if (total_kv == 0) return SV_OK;   // (the plan has written every row)
    CUtensorMap tq, tk, tr, tv;
    if (!encode_rows(&tq, q, kQueryDim, num_heads, kQueryDim, 1, total_q, static_cast<int64_t>(num_heads) * kQueryDim, 128) ||
        !encode_rows(&tk, k, kHeadDim, total_kv, k_stride, 128, num_heads, k_head_stride, 1) ||
        !encode_rows(&tr, rope, kRopeDim, total_kv, rope_stride, 128, 0, 0, 0) ||
        !encode_rows(&tv, v, kHeadDim, total_kv, v_stride, 64, num_heads, v_head_stride, 1))
        return SV_ERR_CUDA;
    static std::atomic<bool> attr_set[64];
    const int st = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess
                   ? SV_OK
                   : SV_ERR_CUDA;
    });
    if (st) return st;
    const int ctas = a.ctas;
    if (launch_pdl(expanded_kernel, dim3(ctas), dim3(kThreads), kSmem, stream, a, tq, tk, tr, tv) != cudaSuccess)
        return SV_ERR_CUDA;
    if (ctas < 2) return SV_OK;
    const int y = lay.item_rows < 32 ? lay.item_rows : (lay.item_rows < 128 ? 32 : 8);
    return launch_pdl(expanded_join_kernel, dim3(ctas - 1, y), dim3(kCutThreads), 0, stream, a) == cudaSuccess ? SV_OK
                                                                                                             : SV_ERR_CUDA;
}

}  // namespace svq
