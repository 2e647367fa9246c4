// Attention of many query rows over ranges of cached pages on the tcgen05
// tensor cores: chunks of query tokens with a sliding window and sinks, and the
// shared prefix of a decode batch.
//
// Mathematics.  A row tile is up to 256 (query token, query head) pairs that
// read the same pages of one kv head; 128 of them are one MMA's M side, so the
// group's query heads share every key and value.  With Q (128 x 128), a key
// tile K (128 tokens x 128) and a value tile V,
//   S = Q K^T                  (fp32 in TMEM, 8 MMAs of k = 16 channels)
//   P = exp2(S * scale - base) (bf16 in TMEM over S; base = a running maximum)
//   O = O * 2^(old - new base) + P V   (fp32 in TMEM, one MMA of k = 16 per page;
//                               every kFoldTiles tiles it moves into sums in memory)
// and at the end out = O / sum P, lse = ln 2 * (base + log2 sum P).  The sums and
// bases are fp32.  P is rounded to bf16 because one MMA takes both operands in
// one type and V is bf16; the sum is taken of the unrounded weights.  That is off
// by at most 2^-8 of each weight (outputs are 0.0023 from 64 bits where the
// output's own rounding alone is 0.0017); P in two parts would be half as much
// tensor work again.
//
// Work.  An entry is a row tile with its page range: a plan kernel lists those
// of chunks, those of prefixes follow from the groups.  Every CTA takes an
// equal run of the
// (entry, kv head, tile) sequence, so ragged batches, short windows and long
// contexts all fill the GPU without a choice of splits; a run that starts or
// ends inside an item leaves a partial (O, base, sum) in the workspace, joined
// by a second kernel.  A CTA has at most two such partials, so their traffic
// does not grow with the problem.
//
// Roles of a CTA (one per SM; TMEM holds S0, S1, O0, O1 of 128 columns each):
//   warps 0, 3   load key and value pages through a ring of 32 KB stages (TMA, one
//                box a page)
//   warp 1       issues the MMAs (one thread)
//   warps 4-7    softmax of stream 0, one row a thread
//   warps 8-11   softmax of stream 1
//   warps 12-19  (e4m3 pools) widen the codes to bf16 tiles
// Two streams keep the tensor cores busy while the other's softmax runs: the
// two 128-row halves of a tile of more than 128 rows, each over every key
// tile; or, for up to 128 rows, the even and the odd key tiles of the same
// rows, joined at the end.
//
// What bounds it.  bf16, long runs: the tensor pipe and the softmax between its
// products (8 MMAs of 64 cycles a product; 128 exponentials a row and tile on
// 16 lanes a cycle take as long).  e4m3: instructions, of the softmax (the
// scales, two passes over S) and of widening every tile's codes.  Few rows or
// short runs: the start, the first copies, and partials.  Measured on GB300s
// (copy 6.8 TB/s, library bf16 product 1895 TFLOP/s), 32 query / 4 kv heads, on the
// device in a graph and as a call in a run of calls: a 4096-token chunk at 32768
// tokens, causal, 1.24 to 1.28 ms and 1.33 to 1.38, by the card's power (1490 to
// 1650 TFLOP/s, 79 to 87 % of the product's), with a window of 4096 tokens 216 us
// and 220 to 224 (1250 TFLOP/s of visible work; 12 % of the tiles' work is masked
// or item cost); 7 ragged e4m3 requests of up to 4000 tokens 87 us and 92 (48 % of
// the issue slots, the tensor pipe 18 %); 32 requests behind 32768 shared tokens
// 38 to 40 us and 42 to 44, of which these tiles 21 to 25.
#include <climits>

#include "svq_paged.cuh"

namespace svq {

SVQ_DEFINE_ERROR_WORD(read_error_attend)

int window_decode_splits(bool fp8, int batch, int num_kv_heads, int64_t pages, int sm_count);
int window_decode_cluster(bool fp8, int batch, int num_kv_heads, int64_t pages, int sm_count, bool must);
bool prefix_alone(bool fp8, int batch, int num_kv_heads, int64_t pages);
int64_t window_decode_rows(int batch, int num_q_heads, int num_kv_heads);
int launch_window_decode(const sv_cache* c, const void* q, int num_q_heads, const int32_t* page_table,
                         const int32_t* seq_lens, int batch, int max_pages, int window, int sink,
                         const int32_t* group_start, const int32_t* shared_pages, int num_groups, float softmax_scale,
                         const PrefixParts* prefix, int splits, void* out, float* lse, float* o_part, float2* ml_part,
                         cudaStream_t stream);
int launch_join_splits(const float* o_part, const float2* ml_part, int splits, int64_t rows, void* out, float* lse,
                       cudaStream_t stream);

namespace {

constexpr int kTileTok = kTilePages * kPage;        // 128 tokens
constexpr int kPageBytes = kPage * kHeadDim * 2;    // a page's bf16 tile of one kv head: 4 KB
constexpr int kStageBytes = kTilePages * kPageBytes;
constexpr int kRowTile = 256;                       // rows of an entry at most
constexpr int kInfoSlots = 8;                       // tiles whose page faults / scales are kept (loads run at most 5 tiles ahead)
constexpr int kMaxCtas = 160;                       // partial slots in the workspace
constexpr float kSlack = 8.f;                       // log2 units the base may lag behind the maximum
// A stream's key tiles after which its O and sum move into fp32 sums of their own and start again from zero.  The
// MMAs cut their sums off at fp32's last bit, eight times a tile, always towards zero: values of one sign lose 2^-20.4
// of their sum a tile (0.4 % over a million tokens, 5 % over 8 million, measured).  512 tiles lose 2^-11.4.
constexpr int kFoldTiles = 512;
constexpr int kColS = 0, kColO = 256;               // TMEM columns of S0 and O0; S1 and O1 lie 128 further

// One row tile and the pages that some row of it sees: the first `sink_pages`
// logical pages, then pages from w0 on.
struct __align__(16) Entry {
    int row0;         // first query token (row of q)
    int ntok;         // query tokens
    int pos0;         // position of the first one; kAllVisible: no mask
    int req;          // page table row
    int sink_pages;
    int w0;
    int npages;       // pages in the list
    int tiles;        // key tiles of npages
};
constexpr int kAllVisible = 1 << 30;

struct Plan {
    Entry* entries;
    int64_t* cum;      // [E + 1] cost per kv head of the entries before each
    int* num_entries;
    int* req_offset;   // first entry of each request
};

struct AttendArgs {
    const __nv_bfloat16* q;
    int num_q_heads, num_kv_heads, group;
    const int32_t* page_table;
    int max_pages;
    int64_t num_phys_pages;
    const unsigned char* k_pool;
    const unsigned char* v_pool;
    const float* k_scale;
    const float* v_scale;
    Plan plan;         // chunks
    Groups groups;     // prefixes
    int tok_per_entry; // query tokens of a row tile: kRowTile / group
    const int32_t* seq_lens;   // prefixes
    int window;        // INT_MAX: none
    int sink;
    float scale_log2;  // softmax_scale * log2(e)
    __nv_bfloat16* out;
    float* lse;
    float* cut_o;      // [2 CTAs][slot_rows][128] partials of items that are cut
    float2* cut_ml;    // [2 CTAs][slot_rows] (base in log2 units, sum)
    GroupRec* group_rec;   // prefixes: [groups + 1], for the join; the last one's cost is the total
    int4* cut_item;    // chunks: [CTAs][2] the item that goes on in a CTA: row0, ntok, kv head, pieces (0: none is to
                       // be joined here); slot of the first piece, of the second, and the entry
    uint32_t* odd;     // chunks: 32-row parts of whole items with a channel that is not finite:
                       // (entry * kv heads + kv head) * 8 + part
    int* num_odd;
    bool fp8;
    int slot_rows;
    float* whole_o;    // prefixes: the parts of whole items, [B Hq][128]; else null
    float2* whole_ml;
    float* split_o;    // prefixes: the parts behind the prefix, [B Hq][splits][128]
    float2* split_ml;
    int splits;
};

// Largest e in [0, n) with cum[e] <= u, by the whole warp (32 probes a round trip).
__device__ __forceinline__ int warp_find(const int64_t* cum, int n, int64_t u) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) / 32;
        const int at = lo + lane * step;
        const bool le = lane * step < len && cum[at] <= u;
        const int k = __popc(__ballot_sync(0xffffffffu, le)) - 1;   // cum is non-decreasing: a prefix of the lanes
        const int nlo = lo + max(k, 0) * step;
        len = min(step, lo + len - nlo);
        lo = nlo;
    }
    return lo;
}

// Prefixes: a group has `entries` row tiles of `tiles` key tiles each.
struct GroupAt {
    int g, a, entries, tiles;
    int64_t before;   // cost per kv head of the groups before it
};
// By the whole warp, 32 groups a round from group `from` on, before which lie groups of cost `total` per kv head that
// end at request `reach`: the group for which pick(before, cost) holds, if any (else g < 0), and the cost up to the
// last group looked at (all of them unless `stop`: the search ends with the group).  rec: where the groups are written
// down, and what is wrong with them reported.
template <typename F>
__device__ __forceinline__ GroupAt warp_groups(const Groups& gr, int tok_per_entry, int from, int reach, int64_t& total,
                                               bool stop, GroupRec* rec, F&& pick) {
    const int lane = threadIdx.x & 31;
    GroupAt found = {-1, 0, 0, 0, 0};
    for (int g0 = from; g0 < gr.n && !(stop && found.g >= 0); g0 += 32) {
        const int g = g0 + lane;
        int a = 0, end = 0, sp = 0;
        bool ok = false;
        if (g < gr.n) {
            a = gr.start[g];
            end = gr.start[g + 1];
            sp = gr.pages[g];
            ok = gr.sound(a, end, sp);
        }
        ok = sound_in_order(ok, a, end, reach);
        const int entries = ok && sp > 0 ? (end - a + tok_per_entry - 1) / tok_per_entry : 0;
        const int64_t cost = static_cast<int64_t>(entries) * cost_of(tiles_of(sp));
        int64_t x = cost;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        const int64_t before = total + x - cost;
        if (rec && g < gr.n) {
            if (!ok) svq_flag(SV_DEVERR_GROUP);
            rec[g] = GroupRec{before, ok ? tiles_of(sp) : 0, ok};
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, ok && pick(before, cost));
        if (hit && found.g < 0) {
            const int src = __ffs(hit) - 1;
            found = {g0 + src, __shfl_sync(0xffffffffu, a, src), __shfl_sync(0xffffffffu, entries, src),
                     __shfl_sync(0xffffffffu, tiles_of(sp), src), __shfl_sync(0xffffffffu, before, src)};
        }
        total += __shfl_sync(0xffffffffu, x, 31);
    }
    if (rec && lane == 0) rec[gr.n].before = total;
    return found;
}

// ---------------------------------------------------------------- tcgen05
// bf16 x bf16 -> fp32, M = 128, N = 128, A K-major; B K-major (keys) or N-major (values).
constexpr uint32_t kIdescQK = (1u << 4) | (1u << 7) | (1u << 10) | ((128u / 8) << 17) | ((128u / 16) << 24);
constexpr uint32_t kIdescPV = kIdescQK | (1u << 16);

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
// S = Q K^T: channels 16 k .. of both operands are 32 bytes further in a half's
// rows (2 in the descriptor); the second half is 16 KB (Q) and 1 KB (K) on.
__device__ __forceinline__ void mma_qk(uint32_t d, uint32_t q_lo, uint32_t k_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred no, yes;\n\t.reg .b32 al, bl;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.u32 no, 0, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\t"
        SVQ_MMA_SS(0, 0, no) SVQ_MMA_SS(2, 2, yes) SVQ_MMA_SS(4, 4, yes) SVQ_MMA_SS(6, 6, yes)
        SVQ_MMA_SS(1024, 64, yes) SVQ_MMA_SS(1026, 66, yes) SVQ_MMA_SS(1028, 68, yes) SVQ_MMA_SS(1030, 70, yes)
        "}" ::"r"(d), "r"(q_lo), "r"(k_lo), "r"(desc_hi(1024)), "r"(desc_hi(2048)), "r"(idesc)
        : "memory");
}
#define SVQ_MMA_TS(ao, bo, acc)                                                  \
    "add.u32 al, %1, " #ao ";\n\tadd.u32 bl, %2, " #bo ";\n\t"                   \
    "mov.b64 bd, {bl, %3};\n\t"                                                  \
    "tcgen05.mma.cta_group::1.kind::f16 [%0], [al], bd, %4, " #acc ";\n\t"
// O (+)= P V over a whole tile: one step a page (8 TMEM columns, 4 KB).
__device__ __forceinline__ void mma_pv8(uint32_t d, uint32_t p, uint32_t v_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred acc, yes;\n\t.reg .b32 al, bl;\n\t.reg .b64 bd;\n\t"
        "setp.ne.u32 acc, %5, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\t"
        SVQ_MMA_TS(0, 0, acc) SVQ_MMA_TS(8, 256, yes) SVQ_MMA_TS(16, 512, yes) SVQ_MMA_TS(24, 768, yes)
        SVQ_MMA_TS(32, 1024, yes) SVQ_MMA_TS(40, 1280, yes) SVQ_MMA_TS(48, 1536, yes) SVQ_MMA_TS(56, 1792, yes)
        "}" ::"r"(d), "r"(p), "r"(v_lo), "r"(desc_hi(2048)), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void mma_pv1(uint32_t d, uint32_t p, uint32_t v_lo, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred acc;\n\t.reg .b32 al, bl;\n\t.reg .b64 bd;\n\tsetp.ne.u32 acc, %5, 0;\n\t"
        SVQ_MMA_TS(0, 0, acc)
        "}" ::"r"(d), "r"(p), "r"(v_lo), "r"(desc_hi(2048)), "r"(idesc), "r"(acc)
        : "memory");
}
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
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], [%4];"
        ::"r"(dst), "l"(tmap), "r"(0), "r"(y), "r"(bar)
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
// ---------------------------------------------------------------- shared memory
template <bool FP8>
struct Cfg {
    static constexpr int kStages = FP8 ? 3 : 5;
    static constexpr int kCodeStages = FP8 ? 3 : 0;             // 16 KB of e4m3 codes each
    static constexpr int kWiden = FP8 ? 8 : 0;                  // widening warps
    static constexpr int kThreads = 384 + 32 * kWiden;
    static constexpr int kRing = kStages * kStageBytes;
    static constexpr int kQ = 2 * 128 * kHeadDim * 2;           // one 128-row tile a stream
    static constexpr int kCodes = kCodeStages * kTileTok * kHeadDim;
    static constexpr int kScales = FP8 ? kInfoSlots * 2 * kTileTok * 4 : 0;
    static constexpr int kControl = 3072;
    // Registers a thread after the start (the block is launched with 168 or 96 for each);
    // bf16 softmax rows keep their 128 logits in them:
    // 128 x 88 + 256 x 208 = 384 x 168; 384 x 72 + 256 x 128 < 640 x 96.
    static constexpr int kOtherRegs = FP8 ? 72 : 88;
    static constexpr int kSoftmaxRegs = FP8 ? 128 : 208;
    static constexpr int kSmem = kRing + kQ + kCodes + kScales + kControl;
};
static_assert(Cfg<false>::kSmem <= 227 * 1024 && Cfg<true>::kSmem <= 227 * 1024, "shared memory of one CTA");

// A run of tiles of one item (entry, kv head); none: the CTA's work is over.
struct __align__(16) Seg {
    Entry en;
    int h;            // kv head
    int t0, t1;       // tiles of the item
    int slot;         // where a partial goes; -1 - (entry * kv heads + kv head): the segment is the whole item
};
constexpr int kSegs = 4;

struct Control {
    uint64_t full[5], empty[5];       // ring stages
    uint64_t code_full[3], code_empty[3];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t s_full[2], p_full[2], o_full[2], q_full[2];
    uint64_t join[2];                 // both streams have published their statistics / have read O0 and O1
    uint64_t drain;
    uint32_t tmem;
    int gave_up;                      // a role's wait ran out
    int fault[kInfoSlots];            // pages of a tile that the table does not give
    Seg seg[kSegs];
    float2 ml[2][128];                // stream statistics of a joined tile
};
static_assert(sizeof(Control) <= 3072, "control block");

__device__ __forceinline__ int logical_page(const Entry& en, int i) {
    return i < en.sink_pages ? i : en.w0 + i - en.sink_pages;
}
__device__ __forceinline__ int last_pos(const Entry& en) {
    return en.pos0 == kAllVisible ? kAllVisible : en.pos0 + en.ntok - 1;
}

// The loads of a segment of n tiles, in order: K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1):
// the place of a tile's keys and values, and which load a place is.
__device__ __forceinline__ uint32_t k_load(int t) { return t == 0 ? 0u : 2u * t - 1u; }
__device__ __forceinline__ uint32_t v_load(int t, int n) { return t == n - 1 ? 2u * n - 1u : 2u * t + 2u; }
__device__ __forceinline__ bool load_is_k(int i, int n) { return i == 0 || (i != 2 * n - 1 && (i & 1)); }
__device__ __forceinline__ int load_tile(int i, int n) {
    return load_is_k(i, n) ? (i + 1) / 2 : (i == 2 * n - 1 ? n - 1 : i / 2 - 1);
}

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
// Bit 7 of every byte of c that is a NaN code (0x7f or 0xff).
__device__ __forceinline__ uint32_t has_nan(uint32_t c) { return ((c & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ void keep_nan(uint32_t c, uint32_t& lo, uint32_t& hi) {
    const uint32_t n = has_nan(c);
    if (n & 0x00000080u) lo |= 0x00007fffu;
    if (n & 0x00008000u) lo |= 0x7fff0000u;
    if (n & 0x00800000u) hi |= 0x00007fffu;
    if (n & 0x80000000u) hi |= 0x7fff0000u;
}

// Waits for a phase of an mbarrier, at most kPolls polls; false when it gave up.
// A poll that finds the phase open takes 4 us on a GB300 (3.95 measured, whatever
// time limit the instruction is given; with none named a chunk of 4096 tokens at
// 32768 takes 1348 us instead of 1255), so that is after half a second; the waits
// that this bounds are for copies and for other warps' work on a few tiles,
// microseconds.  Few instructions, as every role's loop has several: the roles of
// a CTA share the instruction caches.
constexpr uint32_t kPolls = 1u << 17;
constexpr uint32_t kPollNs = 1000;
// The one wait that may be long is the scheduler's, for a slot whose segment is
// done: 1.7 us a key tile, so 14 s for the 2^30 tokens that a row may have.  It
// ends when another role gave up, and after so many rounds of kPolls (a minute).
constexpr int kSegRounds = 128;
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
__device__ __forceinline__ void gave_up(Control* ct) {
    svq_flag(SV_DEVERR_TIMEOUT);
    *static_cast<volatile int*>(&ct->gave_up) = 1;
}
// The same by a whole warp; all of it leaves for `out` when it gave up.
#define SVQ_WAIT(bar, parity, out)                                                        \
    do {                                                                                  \
        if (__any_sync(0xffffffffu, !bar_wait(smem_addr(&(bar)), (parity)))) {   \
            if (lane == 0) gave_up(ct);                                                   \
            goto out;                                                                     \
        }                                                                                 \
    } while (0)

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

template <bool FP8>
__global__ void __launch_bounds__(Cfg<FP8>::kThreads, 1)
    attend_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v) {
    using C = Cfg<FP8>;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const ring = smem;
    unsigned char* const qs = smem + C::kRing;
    unsigned char* const codes = qs + C::kQ;
    float* const scales = reinterpret_cast<float*>(codes + C::kCodes);   // [slot][K | V][128]
    Control* const ct = reinterpret_cast<Control*>(codes + C::kCodes + C::kScales);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.group;

    if (threadIdx.x == 0) {
        ct->gave_up = 0;
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_addr(&ct->full[i]), FP8 ? C::kWiden : 1);
            mbar_init(smem_addr(&ct->empty[i]), 1);
        }
        for (int i = 0; i < C::kCodeStages; ++i) {
            mbar_init(smem_addr(&ct->code_full[i]), 1);
            mbar_init(smem_addr(&ct->code_empty[i]), C::kWiden);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_addr(&ct->s_full[w]), 1);
            mbar_init(smem_addr(&ct->p_full[w]), 4);
            mbar_init(smem_addr(&ct->o_full[w]), 1);
            mbar_init(smem_addr(&ct->q_full[w]), 128);
        }
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(smem_addr(&ct->seg_full[i]), 1);
            mbar_init(smem_addr(&ct->seg_empty[i]), 3 + 8 + C::kWiden);   // loads, MMAs, softmax, widening warps
        }
        mbar_init(smem_addr(&ct->join[0]), 256);
        mbar_init(smem_addr(&ct->join[1]), 256);
        mbar_init(smem_addr(&ct->drain), 1);
        mbar_init_fence();
        if (!FP8) {
            prefetch_tmap(&tmap_k);
            prefetch_tmap(&tmap_v);
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&ct->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // Prefixes: what is behind them shares nothing with this kernel but the join at its end, and may
    // start when all CTAs are past this wait.
    pdl_wait();
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ct->tmem;
    // Every role takes the segments in order: the k-th is in slot k % kSegs.
    auto seg_wait = [&](uint32_t k) { return bar_wait(smem_addr(&ct->seg_full[k % kSegs]), (k / kSegs) & 1); };
    auto seg_done = [&](uint32_t k) {   // once a warp
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&ct->seg_empty[k % kSegs]));
    };

    {
        if (warp == 0 || warp == 3) {
            // ---------------- loads: warp 0 keys, warp 3 values
            reg_dec<C::kOtherRegs>();
            const bool is_v = warp == 3;
            const void* const map = is_v ? static_cast<const void*>(&tmap_v) : static_cast<const void*>(&tmap_k);
            const unsigned char* const pool = is_v ? a.v_pool : a.k_pool;
            constexpr uint32_t kDepth = FP8 ? C::kCodeStages : C::kStages;
            uint64_t* const full = FP8 ? ct->code_full : ct->full;
            uint64_t* const empty = FP8 ? ct->code_empty : ct->empty;
            const uint32_t to = FP8 ? smem_addr(codes) : smem_addr(ring);
            constexpr uint32_t kTo = FP8 ? kTileTok * kHeadDim : kStageBytes;   // bytes of a stage, of a page
            constexpr uint32_t kToPage = kTo / kTilePages;
            uint32_t base = 0, tile = 0;   // loads and key tiles before the segment
            uint32_t last[3] = {0, 0, 0};  // the last loads issued here, each plus 1
            // Lane l resolves page i + l of a segment's list (four tiles at a time), well before
            // the loads that need it.
            auto fetch = [&](const Seg& g, int i0) {
                const int i = i0 + lane;
                int ph = -2;               // behind the segment's pages
                if (i < min(g.en.npages, g.t1 * kTilePages))
                    ph = a.page_table[static_cast<int64_t>(g.en.req) * a.max_pages + logical_page(g.en, i)];
                return ph;
            };
            int cur = -2, nxt = -2;
            for (uint32_t k = 0;; ++k) {
                const Seg& s = ct->seg[k % kSegs];
                if (k == 0) {
                    SVQ_WAIT(ct->seg_full[0], 0, loads_end);
                    nxt = fetch(s, s.t0 * kTilePages);
                }
                const int n = s.t1 - s.t0;
                if (n == 0) break;
                const int qlo = s.en.pos0, qhi = last_pos(s.en);
                for (int i = 0; i < n; ++i) {
                    if (i % 4 == 0) {
                        cur = nxt;
                        if (i + 4 < n) nxt = fetch(s, (s.t0 + i + 4) * kTilePages);
                    }
                    if (i == n - 1) {      // the next segment's first pages
                        SVQ_WAIT(ct->seg_full[(k + 1) % kSegs], ((k + 1) / kSegs) & 1, loads_end);
                        const Seg& g = ct->seg[(k + 1) % kSegs];
                        nxt = fetch(g, g.t0 * kTilePages);
                    }
                    const uint32_t at = base + (is_v ? v_load(i, n) : k_load(i));
                    const uint32_t st = at % kDepth;
                    int ph = __shfl_sync(0xffffffffu, cur, (i % 4) * kTilePages + (lane & 7));
                    if (lane >= kTilePages) ph = -2;
                    const bool bad = ph != -2 && (ph < 0 || ph >= a.num_phys_pages);
                    uint32_t seen = 0xffffu;
                    if (!FP8 && is_v && ph != -2) {
                        seen = union_mask(logical_page(s.en, (s.t0 + i) * kTilePages + lane) * kPage, qlo, qhi, a.window, a.sink);
                        if (bad) seen = 0u;
                    }
                    const uint32_t faults = __ballot_sync(0xffffffffu, bad);
                    const uint32_t parts = __ballot_sync(0xffffffffu, seen != 0xffffu);
                    const bool load = ph != -2 && !bad && seen == 0xffffu;
                    const uint32_t loads = __ballot_sync(0xffffffffu, load);
                    const int64_t from = (static_cast<int64_t>(bad ? 0 : ph) * a.num_kv_heads + s.h);
                    // Value pages with tokens that no row sees: those tokens may hold anything, so
                    // the warp copies such a page with zeros in their place (P = 0 must not meet a
                    // NaN).  At most three pages of an item: the sinks' last, the window's first,
                    // the last; and pages that the table does not give.  The first one's data are
                    // requested before the stage is free.
                    uint4 v[8];
                    auto request = [&](int p) {
                        const uint32_t m = __shfl_sync(0xffffffffu, seen, p);
                        const uint4* src = reinterpret_cast<const uint4*>(a.v_pool + __shfl_sync(0xffffffffu, from, p) * kPageBytes);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int r = 2 * k + (lane >> 4);
                            v[k] = (m >> r) & 1u ? src[r * 16 + (lane & 15)] : make_uint4(0u, 0u, 0u, 0u);
                        }
                    };
                    if (!FP8 && parts) request(__ffs(parts) - 1);
                    SVQ_WAIT(empty[st], ((at / kDepth) & 1) ^ 1, loads_end);
                    if (faults && !is_v && lane == 0) svq_flag(SV_DEVERR_PAGE_TABLE);
                    if (!is_v && lane == 0) ct->fault[(tile + i) % kInfoSlots] = static_cast<int>(faults);
                    if (!FP8 && parts) {
                        for (uint32_t rest = parts; rest;) {
                            unsigned char* const o = ring + st * kStageBytes + (__ffs(rest) - 1) * kPageBytes;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const int r = 2 * k + (lane >> 4), c = lane & 15;
                                *reinterpret_cast<uint4*>(o + (r >> 3) * 2048 + (c >> 3) * 1024 + (r & 7) * 128 +
                                                          (((c & 7) ^ (r & 7)) << 4)) = v[k];
                            }
                            rest &= rest - 1;
                            if (rest) request(__ffs(rest) - 1);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    const uint32_t bar = smem_addr(&full[st]);
                    if (lane == 0) {
                        const uint32_t bytes = __popc(loads) * (kToPage + (FP8 && !is_v ? 2 * kPage * 4 : 0));
                        if (bytes) mbar_arrive_expect_tx(bar, bytes);
                        else mbar_arrive(bar);
                    }
                    __syncwarp();
                    if (load) {
                        const uint32_t dst = to + st * kTo + lane * kToPage;
                        if (FP8) {
                            bulk_copy_g2s(dst, pool + from * kToPage, kToPage, bar);
                            if (!is_v) {
                                const uint32_t sc = smem_addr(scales + (tile + i) % kInfoSlots * 2 * kTileTok + lane * kPage);
                                bulk_copy_g2s(sc, a.k_scale + from * kPage, kPage * 4, bar);
                                bulk_copy_g2s(sc + kTileTok * 4, a.v_scale + from * kPage, kPage * 4, bar);
                            }
                        } else {
                            tma_load_4d(dst, map, static_cast<int>(from * 2), bar);
                        }
                    }
                    last[2] = last[1];
                    last[1] = last[0];
                    last[0] = at + 1;
                }
                base += 2 * n;
                tile += n;
                seg_done(k);
            }
            goto loads_done;   // every load has been waited for by the MMAs or the widening warps
        loads_end:
            // Gave up: the copies still in flight land before the CTA (and its shared memory)
            // retires; at most three of the ring's loads are this warp's.
            for (int k = 0; k < 3; ++k)
                if (last[k]) (void)bar_wait(smem_addr(&full[(last[k] - 1) % kDepth]), ((last[k] - 1) / kDepth) & 1);
        loads_done:;
        } else if (warp == 1) {
            // ---------------- MMAs (one thread)
            reg_dec<C::kOtherRegs>();
            if (lane == 0) {
                uint32_t ld = 0;
                uint32_t q_ph = 0, p_ph = 0;   // bit w: stream w's phase
                const uint32_t ring_s = smem_addr(ring), qs_s = smem_addr(qs);
                auto load_ready = [&](uint32_t i) {
                    return bar_wait(smem_addr(&ct->full[i % C::kStages]), (i / C::kStages) & 1);
                };
                auto stage = [&](uint32_t i) { return ring_s + i % C::kStages * kStageBytes; };
                auto release = [&](uint32_t i) { mma_commit(smem_addr(&ct->empty[i % C::kStages])); };
                auto qk = [&](int w, uint32_t ks) {
                    mma_qk(tmem + kColS + w * 128, desc_lo(qs_s + w * (128 * kHeadDim * 2), 16), desc_lo(ks, 16), kIdescQK);
                    mma_commit(smem_addr(&ct->s_full[w]));
                };
                bool ok = true;
                for (uint32_t k = 0; ok; ++k) {
                    ok = seg_wait(k);
                    const Seg& s = ct->seg[k % kSegs];
                    const int n = s.t1 - s.t0;
                    if (!ok || n == 0) break;
                    const bool two = s.en.ntok * group > 128;   // two row halves; else even and odd tiles
                    const int first_page = s.t0 * kTilePages, npages = s.en.npages;
                    for (int w = 0; w < 2 && ok; ++w) {
                        const int t = two ? 0 : w;
                        if (t >= n) break;
                        const uint32_t kl = ld + k_load(t);
                        ok = load_ready(kl) && bar_wait(smem_addr(&ct->q_full[w]), (q_ph >> w) & 1);
                        q_ph ^= 1u << w;
                        if (!ok) break;
                        tc_fence_after();
                        qk(w, stage(kl));
                        if (!two || w == 1) release(kl);
                    }
                    // P V of (stream w, tile t), whose values are in stage vl.
                    auto pv = [&](int w, uint32_t vs, int pages, bool acc) {
                        // The two 64-channel halves of a value tile are 1 KB apart (N-major operand).
                        const uint32_t v_lo = desc_lo(vs, 1024);
                        const uint32_t o = tmem + kColO + w * 128, p = tmem + kColS + w * 128;
                        if (pages >= kTilePages) {
                            mma_pv8(o, p, v_lo, kIdescPV, acc);
                        } else {
                            for (int u = 0; u < pages; ++u)
                                mma_pv1(o, p + u * 8, v_lo + u * (kPageBytes >> 4), kIdescPV, acc || u != 0);
                        }
                    };
                    auto p_ready = [&](int w) {
                        const bool r = bar_wait(smem_addr(&ct->p_full[w]), (p_ph >> w) & 1);
                        p_ph ^= 1u << w;
                        tc_fence_after();
                        return r;
                    };
                    // The tensor pipe queues only a few MMAs, so what lies between the last of one
                    // (tile, stream) pair and the first of the next is kept short: loads are waited
                    // for once a tile, stages follow one another.
                    int pages = npages - first_page;
                    if (two) {
                        for (int t = 0; t < n && ok; ++t, pages -= kTilePages) {
                            const bool next = t + 1 < n;
                            const uint32_t vl = ld + v_load(t, n), kl = ld + k_load(t + 1);
                            const uint32_t vs = stage(vl), ks = stage(kl);
                            ok = load_ready(vl) && (!next || load_ready(kl)) && p_ready(0);
                            if (!ok) break;
                            pv(0, vs, pages, (t & (kFoldTiles - 1)) != 0);
                            if (next) qk(0, ks);
                            else mma_commit(smem_addr(&ct->o_full[0]));
                            ok = p_ready(1);
                            if (!ok) break;
                            pv(1, vs, pages, (t & (kFoldTiles - 1)) != 0);
                            if (next) qk(1, ks);
                            else mma_commit(smem_addr(&ct->o_full[1]));
                            release(vl);
                            if (next) release(kl);
                        }
                    } else {
                        for (int t = 0; t < n && ok; ++t, pages -= kTilePages) {
                            const int w = t & 1;
                            const bool next = t + 2 < n;
                            const uint32_t vl = ld + v_load(t, n), kl = ld + k_load(t + 2);
                            ok = load_ready(vl) && (!next || load_ready(kl)) && p_ready(w);
                            if (!ok) break;
                            pv(w, stage(vl), pages, ((t >> 1) & (kFoldTiles - 1)) != 0);
                            if (next) qk(w, stage(kl));
                            else mma_commit(smem_addr(&ct->o_full[w]));
                            release(vl);
                            if (next) release(kl);
                        }
                    }
                    ld += 2 * n;
                    if (ok) mbar_arrive(smem_addr(&ct->seg_empty[k % kSegs]));
                }
                if (!ok) gave_up(ct);
                mma_commit(smem_addr(&ct->drain));   // nothing of this CTA's is in flight when TMEM is freed
                (void)bar_wait(smem_addr(&ct->drain), 0);
            }
            __syncwarp();
        } else if (warp == 2) {
            // ---------------- the CTA's share of the plan, segment by segment
            reg_dec<C::kOtherRegs>();
            const bool prefix = a.groups.start != nullptr;
            int num_entries = 0;
            int64_t total = 0;
            GroupAt grp;
            if (prefix) {
                grp = warp_groups(a.groups, a.tok_per_entry, 0, 0, total, false, blockIdx.x == 0 ? a.group_rec : nullptr,
                                  [](int64_t, int64_t) { return false; });
            } else {
                num_entries = *a.plan.num_entries;
                total = a.plan.cum[num_entries];
            }
            const Share share(total * a.num_kv_heads, gridDim.x);
            const int64_t first = share.start(blockIdx.x);
            int64_t left = share.start(blockIdx.x + 1) - first;
            int e = 0, h = 0;                // entry (prefixes: of the group)
            int64_t off = 0;                 // into the item's cost
            if (left > 0) {
                const int64_t u = div64(first, a.num_kv_heads);
                int64_t before;
                int cost;
                if (prefix) {
                    int64_t passed = 0;
                    grp = warp_groups(a.groups, a.tok_per_entry, 0, 0, passed, true, nullptr,
                                      [u](int64_t b, int64_t c) { return b <= u && u < b + c; });
                    cost = cost_of(grp.tiles);
                    e = static_cast<int>(div64(u - grp.before, cost));
                    before = grp.before + static_cast<int64_t>(e) * cost;
                } else {
                    e = warp_find(a.plan.cum, num_entries, u);
                    before = a.plan.cum[e];
                    cost = cost_of(a.plan.entries[e].tiles);
                }
                const int64_t in = first - before * a.num_kv_heads;
                h = static_cast<int>(div64(in, cost));
                off = in - static_cast<int64_t>(h) * cost;
            }
            const bool go_on = off > 0;      // the share begins inside an item
            if (left <= 0 && !prefix && lane == 0) a.cut_item[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
            bool first_item = true;
            Entry en;
            int held = -1;
            for (uint32_t k = 0;;) {
                int t0 = 0, t1 = 0;
                if (left > 0) {
                    if (prefix && held != e) {
                        if (e == grp.entries) {   // the next group with something to read
                            int64_t passed = grp.before + static_cast<int64_t>(grp.entries) * cost_of(grp.tiles);
                            grp = warp_groups(a.groups, a.tok_per_entry, grp.g + 1, a.groups.start[grp.g + 1], passed, true,
                                              nullptr, [](int64_t, int64_t c) { return c > 0; });
                            e = 0;
                        }
                        const int row0 = grp.a + e * a.tok_per_entry;
                        const int pages = a.groups.pages[grp.g];
                        en = Entry{row0, min(a.tok_per_entry, a.groups.start[grp.g + 1] - row0), kAllVisible, grp.a, 0, 0, pages,
                                   grp.tiles};
                        held = e;
                    }
                    while (!prefix && held != e) {
                        const int4* p = reinterpret_cast<const int4*>(a.plan.entries + e);
                        const int4 x = p[0], y = p[1];
                        en = Entry{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                        held = e;
                        if (en.tiles == 0) ++e;   // rows that see nothing
                    }
                    if (first_item && !prefix && lane == 0) {
                        // The CTA after the one with an item's first tile names the item for the join.
                        int4 what = make_int4(0, 0, 0, 0), where = make_int4(0, 0, 0, 0);
                        if (go_on) {
                            const Placed it(share, first - off, en.tiles);
                            if (static_cast<int>(blockIdx.x) == it.c0 + 1) {
                                what = make_int4(en.row0, en.ntok, h, it.c1 - it.c0 + 1);
                                where.x = 2 * it.c0 + (share.start(it.c0) >= it.begin ? 0 : 1);
                                where.y = 2 * (it.c0 + 1);
                                where.z = e;
                            }
                        }
                        a.cut_item[2 * blockIdx.x] = what;
                        a.cut_item[2 * blockIdx.x + 1] = where;
                    }
                    const int64_t take = min(left, cost_of(en.tiles) - off);
                    t0 = static_cast<int>(max(static_cast<int64_t>(0), off - kItemCost));
                    t1 = static_cast<int>(max(static_cast<int64_t>(0), off + take - kItemCost));
                    left -= take;
                    off += take;
                }
                if (t1 > t0 || left <= 0) {
                    for (int round = 0;; ++round) {
                        if (!__any_sync(0xffffffffu, !bar_wait(smem_addr(&ct->seg_empty[k % kSegs]), ((k / kSegs) & 1) ^ 1))) break;
                        if (__any_sync(0xffffffffu, *static_cast<volatile int*>(&ct->gave_up)) || round == kSegRounds) {
                            if (lane == 0) gave_up(ct);
                            goto plan_end;
                        }
                    }
                    if (lane == 0) {
                        Seg& s = ct->seg[k % kSegs];
                        s.en = en;
                        s.h = h;
                        s.t0 = t0;
                        s.t1 = t1;
                        s.slot = t0 == 0 && t1 == en.tiles ? -1 - (e * a.num_kv_heads + h) : static_cast<int>(blockIdx.x) * 2 + (first_item ? 0 : 1);
                        mbar_arrive(smem_addr(&ct->seg_full[k % kSegs]));
                    }
                    ++k;
                    if (t1 == t0) break;
                }
                first_item = false;
                if (off == cost_of(en.tiles)) {
                    off = 0;
                    if (++h == a.num_kv_heads) {
                        h = 0;
                        ++e;
                        held = -1;
                    }
                }
            }
        plan_end:;
        } else if (warp < 12) {
            // ---------------- softmax: warps 4-7 stream 0, warps 8-11 stream 1
            reg_inc<C::kSoftmaxRegs>();
            const int w = (warp - 4) >> 2;
            const int row = (warp & 3) * 32 + lane;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const uint32_t s_col = tmem + lanes + kColS + w * 128;
            const uint32_t o_col = tmem + lanes + kColO + w * 128;
            uint32_t s_ph = 0, o_ph0 = 0, o_ph1 = 0, join_ph = 0;
            uint32_t tile0 = 0;          // key tiles of the CTA before the segment
            auto stream_tiles = [&](const Seg& g) {
                const int n = g.t1 - g.t0;
                return g.en.ntok * group > 128 ? n : (n - w + 1) / 2;
            };
            // The stream's 128 rows of Q, 128-byte swizzled, two halves of 64 channels.
            auto load_q = [&](const Seg& g) {
                const int rows = g.en.ntok * group;
                const int off = rows > 128 ? w * 128 : 0;
                const int tid = row, c = tid & 15;
                const uint32_t dst = smem_addr(qs) + w * (128 * kHeadDim * 2) + (c >> 3) * 16384;
                for (int r = tid >> 4; r < 128 && off + r < rows; r += 8) {
                    const int tok = (off + r) / group, head = (off + r) - tok * group;
                    const __nv_bfloat16* src =
                        a.q + (static_cast<int64_t>(g.en.row0 + tok) * a.num_q_heads + g.h * group + head) * kHeadDim + c * 8;
                    cp_async16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4), src, 16);
                }
                cp_async_commit();
            };
            auto q_ready = [&] {
                cp_async_wait<0>();
                fence_proxy_async_smem();
                mbar_arrive(smem_addr(&ct->q_full[w]));
            };
            for (uint32_t k = 0;; ++k) {
                const Seg& s = ct->seg[k % kSegs];
                if (k == 0) {
                    SVQ_WAIT(ct->seg_full[0], 0, softmax_end);
                    if (stream_tiles(s) > 0) {
                        load_q(s);
                        q_ready();
                    }
                }
                const int n = s.t1 - s.t0;
                if (n == 0) break;
                SVQ_WAIT(ct->seg_full[(k + 1) % kSegs], ((k + 1) / kSegs) & 1, softmax_end);
                const Seg& nx = ct->seg[(k + 1) % kSegs];
                const bool next_q = stream_tiles(nx) > 0;
                const int rows = s.en.ntok * group;
                const bool two = rows > 128;
                const int nt = stream_tiles(s);
                const int off = two ? w * 128 : 0;
                const int r = off + row;
                const bool valid = r < rows;
                const bool warp_on = off + (warp & 3) * 32 < rows;
                const int tok = r / group;
                const bool all = s.en.pos0 == kAllVisible;
                const int qpos = all ? kAllVisible : s.en.pos0 + min(tok, s.en.ntok - 1);
                const int qlo = all ? kAllVisible : s.en.pos0 + off / group;
                const int qhi = all ? kAllVisible : s.en.pos0 + (min(rows, off + 128) - 1) / group;
                float m = -INFINITY, l = 0.f;
                // The row's place for what is folded: that of the segment's partial; a whole item's CTA has not
                // written its second one yet.  (Base, sum) are kept in ct->ml.
                auto folded = [&] {
                    const int slot = s.slot >= 0 ? s.slot : 2 * static_cast<int>(blockIdx.x) + 1;
                    return a.cut_o + (static_cast<int64_t>(slot) * a.slot_rows + (two ? r : w * (a.slot_rows / 2) + row)) * kHeadDim;
                };
                for (int j0 = 0; j0 < nt; j0 += kFoldTiles) {
                    if (j0 > 0) {
                        SVQ_WAIT(ct->s_full[w], s_ph, softmax_end);   // O is complete, and the next product into it starts anew
                        if (warp_on) fold_out(o_col, folded(), valid, j0 > kFoldTiles, ct->ml[w][row], m, l);
                        l = 0.f;
                    }
                    for (int j = j0; j < min(nt, j0 + kFoldTiles); ++j) {
                        const int ti = two ? j : 2 * j + w;          // tile of the segment
                        const int i0 = (s.t0 + ti) * kTilePages;     // first page of the tile in the list
                        const int slot = (tile0 + ti) % kInfoSlots;
                        const int base0 = logical_page(s.en, i0) * kPage, base7 = logical_page(s.en, i0 + 7) * kPage;
                        bool plain = i0 + kTilePages <= s.en.npages && base7 - base0 == 7 * kPage && base7 + 15 <= qlo &&
                                     (base0 > qhi - a.window || base7 + 15 < a.sink);
                        SVQ_WAIT(ct->s_full[w], s_ph, softmax_end);
                        s_ph ^= 1;
                        tc_fence_after();
                        if (j == nt - 1 && next_q) load_q(nx);       // the stream's last use of Q is over
                        if (warp_on) {
                            const int fault = ct->fault[slot];
                            plain = plain && !fault;
                            // Visible columns, 32 a word (two pages).
                            uint32_t bits0 = ~0u, bits1 = ~0u, bits2 = ~0u, bits3 = ~0u;
                            if (!plain) {
                                auto two_pages = [&](int c) {
                                    uint32_t bits = 0;
#pragma unroll
                                    for (int u = 0; u < 2; ++u) {
                                        const int i = i0 + 2 * c + u;
                                        if (i < s.en.npages && !((fault >> (2 * c + u)) & 1))
                                            bits |= page_mask(logical_page(s.en, i) * kPage, qpos, a.window, a.sink) << (16 * u);
                                    }
                                    return bits;
                                };
                                bits0 = two_pages(0);
                                bits1 = two_pages(1);
                                bits2 = two_pages(2);
                                bits3 = two_pages(3);
                            }
                            // Pairs of tokens: key scales times scale_log2, value scales.
                            const ulonglong2* ks = reinterpret_cast<const ulonglong2*>(scales + slot * 2 * kTileTok);
                            const ulonglong2* vs = ks + kTileTok / 4;
                            // The row's logits.  bf16: all 128 stay in registers from here to P (a causal chunk
                            // 1268 us; with the exponentials in a rolled loop 1363).  e4m3 (fewer registers a
                            // thread, and the widening warps' code beside it in the instruction cache): rolled
                            // loops over 32 columns that read S from TMEM twice (ragged chunks 89.0 us; logits in
                            // registers, with half the widening warps, 90.7).  Scales act on pairs of tokens,
                            // the keys' with scale_log2 in them.
                            float x[FP8 ? 1 : 128];
                            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                            if constexpr (FP8) {
#pragma unroll 1
                                for (int c = 0; c < 4; ++c) {
                                    float x[32];
                                    tc_ld32(s_col + c * 32, reinterpret_cast<uint32_t(&)[32]>(x));
                                    tc_wait_ld();
#pragma unroll
                                    for (int u = 0; u < 8; ++u) {
                                        const ulonglong2 k4 = ks[c * 8 + u];
                                        unpack2(mul2(pack2(x[4 * u], x[4 * u + 1]), k4.x), x[4 * u], x[4 * u + 1]);
                                        unpack2(mul2(pack2(x[4 * u + 2], x[4 * u + 3]), k4.y), x[4 * u + 2], x[4 * u + 3]);
                                    }
                                    const uint32_t bits = c == 0 ? bits0 : (c == 1 ? bits1 : (c == 2 ? bits2 : bits3));
                                    if (__any_sync(0xffffffffu, bits != ~0u)) {
#pragma unroll
                                        for (int u = 0; u < 32; ++u)
                                            if (!((bits >> u) & 1u)) x[u] = -INFINITY;
                                    }
#pragma unroll
                                    for (int u = 0; u < 32; u += 8)
#pragma unroll
                                        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], x[u + 2 * k]), x[u + 2 * k + 1]);
                                }
                            } else {
#pragma unroll
                                for (int c = 0; c < 4; ++c) tc_ld32(s_col + c * 32, reinterpret_cast<uint32_t(&)[32]>(x[c * 32]));
                                tc_wait_ld();
                                if (!plain) {
#pragma unroll
                                    for (int c = 0; c < 4; ++c) {
                                        const uint32_t bits = c == 0 ? bits0 : (c == 1 ? bits1 : (c == 2 ? bits2 : bits3));
#pragma unroll
                                        for (int u = 0; u < 32; ++u)
                                            if (!((bits >> u) & 1u)) x[c * 32 + u] = -INFINITY;
                                    }
                                }
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    mx[c] = fmaxf(x[c], x[c + 4]);
#pragma unroll
                                    for (int u = 8; u < 128; u += 8) mx[c] = fmaxf(fmaxf(mx[c], x[u + c]), x[u + c + 4]);
                                }
                            }
                            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (FP8 ? 1.f : a.scale_log2);
                            // The base moves only when the maximum is more than kSlack above it; weights
                            // stay at most 2^kSlack, and sums and outputs share the base.
                            // Threads without a row hold whatever Q's memory held and have no say.
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
                            if constexpr (FP8) {
#pragma unroll 1
                                for (int c = 0; c < 4; ++c) {
                                    float x[32];
                                    uint32_t p[16];
                                    tc_ld32(s_col + c * 32, reinterpret_cast<uint32_t(&)[32]>(x));
                                    tc_wait_ld();
#pragma unroll
                                    for (int u = 0; u < 8; ++u) {
                                        const ulonglong2 k4 = ks[c * 8 + u];
                                        unpack2(fma2(pack2(x[4 * u], x[4 * u + 1]), k4.x, base2), x[4 * u], x[4 * u + 1]);
                                        unpack2(fma2(pack2(x[4 * u + 2], x[4 * u + 3]), k4.y, base2), x[4 * u + 2], x[4 * u + 3]);
                                    }
                                    const uint32_t bits = c == 0 ? bits0 : (c == 1 ? bits1 : (c == 2 ? bits2 : bits3));
                                    if (__any_sync(0xffffffffu, bits != ~0u)) {
#pragma unroll
                                        for (int u = 0; u < 32; ++u)
                                            if (!((bits >> u) & 1u)) x[u] = -INFINITY;
                                    }
#pragma unroll
                                    for (int u = 0; u < 8; ++u) {
                                        const ulonglong2 v4 = vs[c * 8 + u];
                                        const uint64_t e0 = pack2(ex2(x[4 * u]), ex2(x[4 * u + 1]));
                                        const uint64_t e1 = pack2(ex2(x[4 * u + 2]), ex2(x[4 * u + 3]));
                                        sum[0] = add2(sum[0], e0);
                                        sum[1] = add2(sum[1], e1);
                                        float w0, w1;
                                        unpack2(mul2(e0, v4.x), w0, w1);
                                        p[2 * u] = pack_bf16x2(w0, w1);
                                        unpack2(mul2(e1, v4.y), w0, w1);
                                        p[2 * u + 1] = pack_bf16x2(w0, w1);
                                    }
                                    tc_st16(s_col + c * 16, p);
                                }
                            } else {
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
                                sum[0] = add2(sum[0], sum[2]);
                                sum[1] = add2(sum[1], sum[3]);
                            }
                            {
                                float s0, s1;
                                unpack2(add2(sum[0], sum[1]), s0, s1);
                                l += s0 + s1;
                            }
                            tc_wait_st();
                        }
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&ct->p_full[w]));
                    }
                }
                if (nt == 0 && next_q) load_q(nx);
                if (next_q) q_ready();

                // ---------------- the segment's end
                float* po = nullptr;        // this row's fp32 partial
                float2* pml = nullptr;
                const int hr = r - tok * group;
                const int64_t qrow = static_cast<int64_t>(s.en.row0 + tok) * a.num_q_heads + s.h * group + hr;
                if (s.slot >= 0) {
                    const int64_t at = static_cast<int64_t>(s.slot) * a.slot_rows + r;
                    po = a.cut_o + at * kHeadDim;
                    pml = a.cut_ml + at;
                } else if (a.whole_o) {
                    po = a.whole_o + qrow * kHeadDim;
                    pml = a.whole_ml + qrow;
                }
                float f0 = 1.f, f1 = 0.f;   // factors of O0 and O1 (f0: of the own O when there are two row halves)
                float M = m, L = l;
                if (two) {
                    SVQ_WAIT(ct->o_full[w], w ? o_ph1 : o_ph0, softmax_end);
                    o_ph0 ^= 1;
                    o_ph1 ^= 1;
                    if (nt > kFoldTiles && warp_on) L = l = fold_in(o_col, folded(), valid, ct->ml[w][row], m, l);
                } else {
                    SVQ_WAIT(ct->o_full[0], o_ph0, softmax_end);
                    o_ph0 ^= 1;
                    if (n > 1) {
                        SVQ_WAIT(ct->o_full[1], o_ph1, softmax_end);
                        o_ph1 ^= 1;
                    }
                    if (nt > kFoldTiles && warp_on) l = fold_in(o_col, folded(), valid, ct->ml[w][row], m, l);
                    ct->ml[w][row] = make_float2(m, l);
                    mbar_arrive(smem_addr(&ct->join[0]));
                    SVQ_WAIT(ct->join[0], join_ph, softmax_end);
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
                    SVQ_WAIT(ct->join[1], join_ph, softmax_end);
                    join_ph ^= 1;
                }
                tile0 += n;
                seg_done(k);
            }
        softmax_end:;
        } else if (FP8) {
            // ---------------- e4m3 codes -> bf16 tiles in the MMAs' layout
            reg_dec<C::kOtherRegs>();
            const int tid = threadIdx.x - 384;
            uint32_t ld = 0, tile = 0;
            constexpr int kCodeDepth = FP8 ? C::kCodeStages : 1;
            for (uint32_t k = 0;; ++k) {
                SVQ_WAIT(ct->seg_full[k % kSegs], (k / kSegs) & 1, widen_end);
                const Seg& s = ct->seg[k % kSegs];
                const int n = s.t1 - s.t0;
                if (n == 0) break;
                const int qlo = s.en.pos0, qhi = last_pos(s.en);
                for (int i = 0; i < 2 * n; ++i) {
                    const bool is_k = load_is_k(i, n);
                    const int t = load_tile(i, n);
                    const int slot = (tile + t) % kInfoSlots;
                    const int cs = ld % kCodeDepth, st = ld % C::kStages;
                    SVQ_WAIT(ct->code_full[cs], (ld / kCodeDepth) & 1, widen_end);
                    const unsigned char* src = codes + cs * (kTileTok * kHeadDim);
                    unsigned char* dst = ring + st * kStageBytes;
                    const int i0 = (s.t0 + t) * kTilePages;
                    // Page k of the tile, every second one here: thread -> row tid / 8 % 16, 16 codes
                    // at chunk tid % 8.
                    const int r = (tid >> 3) & 15, c = tid & 7, odd = tid >> 7;
                    // Tokens no row sees may hold anything: they become zeros, scales too.  Bit k:
                    // this thread's token of page k is seen; `clean`: every token of the tile is.
                    const int base0 = logical_page(s.en, i0) * kPage, base7 = logical_page(s.en, i0 + 7) * kPage;
                    const int fault = ct->fault[slot];
                    const bool clean = !fault && i0 + kTilePages <= s.en.npages && base7 - base0 == 7 * kPage &&
                                       base7 + 15 <= qhi && (base0 > qlo - a.window || base7 + 15 < a.sink);
                    uint32_t on = 0xffu;
                    if (!clean) {
                        on = 0u;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (i0 + k < s.en.npages && !((fault >> k) & 1))
                                on |= ((union_mask(logical_page(s.en, i0 + k) * kPage, qlo, qhi, a.window, a.sink) >> r) & 1u) << k;
                    }
                    const int pages = min(kTilePages, s.en.npages - i0);   // (products with pages behind are masked or left out)
                    unsigned char* const o = dst + (r >> 3) * 2048 + (c >> 2) * 1024 + (r & 7) * 128;
                    const int at0 = ((2 * c) & 7 ^ (r & 7)) << 4, at1 = ((2 * c + 1) & 7 ^ (r & 7)) << 4;
                    // All of a thread's codes first, so that the next copy into their slot starts early.  The fence
                    // keeps that copy behind these reads: without it an arrival overtook them while other warps'
                    // stores filled the load and store unit, and rows of the tile held the next load's codes.
                    uint4 v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        v[u] = *reinterpret_cast<const uint4*>(src + (odd + 2 * u) * (kPage * kHeadDim) + r * kHeadDim + c * 16);
                        if (!((on >> (odd + 2 * u)) & 1u)) v[u] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ct->code_empty[cs]));
                    SVQ_WAIT(ct->empty[st], ((ld / C::kStages) & 1) ^ 1, widen_end);
#pragma unroll 1
                    for (int k0 = odd; k0 < pages; k0 += 4) {
                        uint4 lo[2], hi[2];
                        uint32_t nan = 0;
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            nan |= has_nan(v[u].x) | has_nan(v[u].y) | has_nan(v[u].z) | has_nan(v[u].w);
                            widen4(v[u].x, lo[u].x, lo[u].y);
                            widen4(v[u].y, lo[u].z, lo[u].w);
                            widen4(v[u].z, hi[u].x, hi[u].y);
                            widen4(v[u].w, hi[u].z, hi[u].w);
                        }
                        if (nan) {
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                keep_nan(v[u].x, lo[u].x, lo[u].y);
                                keep_nan(v[u].y, lo[u].z, lo[u].w);
                                keep_nan(v[u].z, hi[u].x, hi[u].y);
                                keep_nan(v[u].w, hi[u].z, hi[u].w);
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            *reinterpret_cast<uint4*>(o + (k0 + 2 * u) * kPageBytes + at0) = lo[u];
                            *reinterpret_cast<uint4*>(o + (k0 + 2 * u) * kPageBytes + at1) = hi[u];
                        }
                        v[0] = v[2];
                        v[1] = v[3];
                    }
                    // Scales of the tile's tokens, with its keys: 0 for tokens that no row sees.
                    if (is_k && c < 4) {
                        const int k = odd + 2 * c;
                        float* const sc = scales + slot * 2 * kTileTok + k * kPage + r;
                        const bool seen = (on >> k) & 1u;
                        *sc = seen ? *sc * a.scale_log2 : 0.f;
                        if (!seen) sc[kTileTok] = 0.f;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ct->full[st]));
                    ++ld;
                }
                tile += n;
                seg_done(k);
            }
        widen_end:;
        }
    }
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------- plan
struct PlanArgs {
    Plan plan;
    int* num_odd;
    int max_entries;
    int tok_per_entry;          // query tokens of a row tile: kRowTile / group
    const int32_t* q_start;
    int total_q;
    const int32_t* seq_lens;
    int batch;
    int max_pages;
    int window;                 // INT_MAX: none
    int sink;
    int num_q_heads;
    __nv_bfloat16* out;         // rows that see nothing get 0 / -inf here
    float* lse;
};

constexpr int kPlanThreads = 1024;

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

// Pages of request b, checked: 0 for a length the page table cannot hold.
__device__ __forceinline__ int checked_len(const PlanArgs& p, int b) {
    const int len = p.seq_lens[b];
    if (len < 0 || (static_cast<int64_t>(len) + kPage - 1) / kPage > p.max_pages) {
        svq_flag(SV_DEVERR_SEQ_LEN);
        return 0;
    }
    return len;
}

// One CTA: the list of the chunks' entries, and the running sum of their costs.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanArgs p) {
    __shared__ int64_t warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31;
    int64_t total;
    pdl_wait();   // the workspace may still be read by the call before
    pdl_launch_dependents();
    // Row tiles before each request: the entries of one are consecutive.
    int n = 0;
    for (int i0 = 0; i0 < p.batch; i0 += kPlanThreads) {
        const int i = i0 + tid;
        int count = 0;
        if (i < p.batch) {
            const int a = p.q_start[i], b = p.q_start[i + 1];
            if (a < 0 || b < a || b > p.total_q) svq_flag(SV_DEVERR_Q_START);
            else count = (b - a + p.tok_per_entry - 1) / p.tok_per_entry;
        }
        const int64_t before = n + block_scan(count, warp_sums, total);
        if (i < p.batch) p.plan.req_offset[i] = static_cast<int>(min(before, static_cast<int64_t>(INT_MAX / 2)));
        n = static_cast<int>(min(n + total, static_cast<int64_t>(INT_MAX / 2)));
    }
    // Overlapping (broken) starts could list more tiles than the workspace holds.
    if (n > p.max_entries) {
        if (tid == 0) svq_flag(SV_DEVERR_Q_START);
        n = p.max_entries;
    }
    __syncthreads();
    int64_t base = 0;
    for (int e0 = 0; e0 < n; e0 += kPlanThreads) {
        const int e = e0 + tid;
        Entry en = {0, 0, 0, 0, 0, 0, 0, 0};
        bool empty = false;   // rows that see nothing
        if (e < n) {
            const int b = find_le(p.plan.req_offset, p.batch, e);
            const int start = p.q_start[b];
            const int size = p.q_start[b + 1] - start;
            const int at = (e - p.plan.req_offset[b]) * p.tok_per_entry;
            int len = checked_len(p, b);
            if (size > len) {
                if (len > 0) svq_flag(SV_DEVERR_Q_START);
                len = 0;
            }
            en.row0 = start + at;
            en.ntok = min(p.tok_per_entry, size - at);
            en.req = b;
            if (len > 0) {
                en.pos0 = len - size + at;
                const int last = (en.pos0 + en.ntok - 1) / kPage + 1;
                const int w0 = max(0, en.pos0 - p.window + 1) / kPage;
                en.sink_pages = sink_pages_of(p.sink, w0);
                en.w0 = w0;
                en.npages = en.sink_pages + last - w0;
            } else {
                empty = true;
            }
        }
        en.tiles = tiles_of(en.npages);
        const int64_t before = base + block_scan(cost_of(en.tiles), warp_sums, total);
        base += total;
        if (e < n) {
            p.plan.entries[e] = en;
            p.plan.cum[e] = before;
        }
        for (uint32_t rest = __ballot_sync(0xffffffffu, empty); rest; rest &= rest - 1) {
            const int src = __ffs(rest) - 1;
            const int64_t r0 = static_cast<int64_t>(__shfl_sync(0xffffffffu, en.row0, src)) * p.num_q_heads;
            const int64_t r1 = r0 + static_cast<int64_t>(__shfl_sync(0xffffffffu, en.ntok, src)) * p.num_q_heads;
            uint4* o = reinterpret_cast<uint4*>(p.out + r0 * kHeadDim);
            for (int64_t i = lane; i < (r1 - r0) * (kHeadDim / 8); i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int64_t i = r0 + lane; i < r1; i += 32) p.lse[i] = -INFINITY;
        }
    }
    if (tid == 0) {
        p.plan.cum[n] = base;
        *p.plan.num_entries = n;
        *p.num_odd = 0;
    }
}

// ---------------------------------------------------------------- joining partials
// A row of an entry whose outputs may not be finite, by one warp.  The tile's
// product multiplies every value of the tile with a weight, and a weight 0 does
// not hide an infinite or NaN value from the rows that do not see its token.  So
// if the row's logits are finite, its outputs are not, and a token that other
// rows of the entry see and this one does not holds such a value, the row is
// computed again from its own tokens alone, at 10 us a page and row (loads four
// tokens at a time would be no faster and their registers cost every join 2 us
// of 212).  Finding such rows costs a call without them 1 to 1.5 us of 210.
__device__ __noinline__ void look_at_row(const AttendArgs& a, int entry, int h, int r) {
    const int lane = threadIdx.x & 31;
    const Entry en = a.plan.entries[entry];
    const int tok = r / a.group, pos = en.pos0 + tok, end = en.pos0 + en.ntok;
    const int64_t qrow = static_cast<int64_t>(en.row0 + tok) * a.num_q_heads + h * a.group + (r - tok * a.group);
    const uint2 w = *reinterpret_cast<const uint2*>(a.out + qrow * kHeadDim + 4 * lane);
    const float4 got = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
    {
        const float odd = fmaf(got.x, 0.f, fmaf(got.y, 0.f, fmaf(got.z, 0.f, got.w * 0.f)));
        if (!(fabsf(a.lse[qrow]) < INFINITY) || !__any_sync(0xffffffffu, odd != 0.f)) return;
    }
    const int32_t* const pages = a.page_table + static_cast<int64_t>(en.req) * a.max_pages;
    // Four channels of a token's row of a pool.
    auto row_of = [&](const unsigned char* pool, const float* scale, int64_t at) {
        uint2 w;
        if (!a.fp8) {
            w = *reinterpret_cast<const uint2*>(pool + at * (2 * kHeadDim) + 8 * lane);
            return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
        }
        const uint32_t c = *reinterpret_cast<const uint32_t*>(pool + at * kHeadDim + 4 * lane);
        widen4(c, w.x, w.y);
        keep_nan(c, w.x, w.y);
        const float f = scale[at];
        return make_float4(bf16lo(w.x) * f, bf16hi(w.x) * f, bf16lo(w.y) * f, bf16hi(w.y) * f);
    };
    auto place_of = [&](int page) {   // the first token's row in the pools; -1: the table gives no page
        const int ph = pages[page];
        return ph < 0 || ph >= a.num_phys_pages ? -1ll : (static_cast<int64_t>(ph) * a.num_kv_heads + h) * kPage;
    };
    if (const int64_t at = place_of(pos / kPage); at >= 0) {
        // The row's own token is NaN wherever the row is not finite (a whole cache of NaN): so is the result.
        const float4 v = row_of(a.v_pool, a.v_scale, at + pos % kPage);
        const bool known = (v.x != v.x || got.x * 0.f == 0.f) && (v.y != v.y || got.y * 0.f == 0.f) &&
                           (v.z != v.z || got.z * 0.f == 0.f) && (v.w != v.w || got.w * 0.f == 0.f);
        if (__all_sync(0xffffffffu, known)) return;
    }
    // Tokens [t0, t1) that other rows may see and this one does not.
    auto finite = [&](int t0, int t1) {
        float odd = 0.f;
        for (int t = t0; t < t1; ++t) {
            const int64_t at = place_of(t / kPage);
            if (at < 0) continue;
            const float4 v = row_of(a.v_pool, a.v_scale, at + t % kPage);
            odd = fmaf(v.x, 0.f, fmaf(v.y, 0.f, fmaf(v.z, 0.f, fmaf(v.w, 0.f, odd))));
        }
        return !__any_sync(0xffffffffu, odd != 0.f);
    };
    const bool later = finite(pos + 1, end);
    const bool passed = finite(max(a.sink, max(0, en.pos0 - a.window + 1)), max(0, pos - a.window + 1));
    if (later && passed) return;   // the row's own tokens gave it
    const uint2 qw = *reinterpret_cast<const uint2*>(a.q + qrow * kHeadDim + 4 * lane);
    const float4 q = make_float4(bf16lo(qw.x), bf16hi(qw.x), bf16lo(qw.y), bf16hi(qw.y));
    RowSum s;
    for (int i = 0; i < en.npages; ++i) {
        const int page = logical_page(en, i);
        const uint32_t seen = page_mask(page * kPage, pos, a.window, a.sink);
        const int64_t at = place_of(page);
        if (at < 0) continue;
        for (uint32_t rest = seen; rest; rest &= rest - 1) {
            const int t = __ffs(rest) - 1;
            const float4 k = row_of(a.k_pool, a.k_scale, at + t), v = row_of(a.v_pool, a.v_scale, at + t);
            float z = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
            for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
            s.join(RowSum{z * a.scale_log2, 1.f, v});
        }
    }
    (void)s.write(a.out + qrow * kHeadDim, a.lse + qrow, lane);
}

// Chunks: CTA (c, y) joins the item that attend CTA c + 1 goes on with; rows y,
// y + gridDim.y, ... (of 8 warps each, when the pieces are few).  Then the parts
// of whole items with rows that are not finite.
constexpr int kCutThreads = 256;

__global__ void __launch_bounds__(kCutThreads, 4) join_cut_kernel(const __grid_constant__ AttendArgs a) {
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
    const int rows = n ? what.y * a.group : 0;
    auto at_row = [&](int r) {
        const int tok = r / a.group;
        return static_cast<int64_t>(what.x + tok) * a.num_q_heads + what.z * a.group + (r - tok * a.group);
    };
    auto pieces = [&](int r) {
        return Pieces{a.cut_o, a.cut_ml, static_cast<int64_t>(where.x) * a.slot_rows + r,
                      static_cast<int64_t>(where.y) * a.slot_rows + r, 2ll * a.slot_rows, n};
    };
    // Rows that are not finite are looked at behind the loops (a call inside them costs 3 us of 212).
    bool odd = false;
    auto write = [&](const RowSum& s, int r) { odd |= s.write(a.out + at_row(r) * kHeadDim, a.lse + at_row(r), lane); };
    if (n <= 8) {   // few pieces: a warp a row, four rows at a time in flight when there are two
        const int step = gridDim.y * kWarps;
        for (int r0 = blockIdx.y * kWarps + warp; r0 < rows; r0 += 4 * step) {
            if (n == 2) {
                float2 ml[4][2];
                float4 x[4][2];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const Pieces p = pieces(min(r0 + u * step, rows - 1));
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        ml[u][k] = p.ml[p.row(k)];
                        x[u][k] = *reinterpret_cast<const float4*>(p.o + p.row(k) * kHeadDim + 4 * lane);
                    }
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    RowSum s;
                    s.add2(ml[u], x[u]);
                    if (r0 + u * step < rows) write(s, r0 + u * step);
                }
            } else {
                for (int u = 0; u < 4; ++u) {
                    const int r = r0 + u * step;
                    if (r >= rows) break;
                    RowSum s;
                    s.add(pieces(r), 0, 1, lane);
                    write(s, r);
                }
            }
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
        const int e = part / 8 / a.num_kv_heads, h = part / 8 % a.num_kv_heads;
        const int r = part % 8 * 32 + static_cast<int>(i % kTurns) * kWarps + warp;
        if (r < a.plan.entries[e].ntok * a.group) look_at_row(a, e, h, r);
    }
}

// Prefixes of so few requests that more than 8 splits a row read what is behind
// them: CTA (request x kv head, y) joins both for group / gridDim.y rows; a row's
// pieces go in turn to the warps it has.  With as few CTAs as fill the GPU:
// finding the pieces takes a CTA as long as adding them (a CTA a row: 50 against
// 45 us for 61 requests).
constexpr int kPrefixThreads = 512;

__global__ void __launch_bounds__(kPrefixThreads) join_prefix_kernel(const __grid_constant__ AttendArgs a,
                                                                     const __grid_constant__ PrefixParts prefix) {
    constexpr int kWarps = kPrefixThreads / 32;
    __shared__ RowSum parts[kWarps][32];
    const int b = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads;
    // Inputs: before the kernels before this one have ended.
    if (b < a.groups.start[0] || b >= a.groups.start[a.groups.n]) {   // not touched
        pdl_wait();
        return;
    }
    uint32_t fault;
    int g;
    const int page = page_behind(a.groups, b, a.seq_lens[b], fault, g);
    const int e = (b - a.groups.start[g]) / a.tok_per_entry, row = b - a.groups.start[g] - e * a.tok_per_entry;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = (a.group + gridDim.y - 1) / gridDim.y, per_row = kWarps / rows;
    const int mine = warp / per_row, part = warp - mine * per_row;   // row of this CTA, share of its pieces
    const int hr = blockIdx.y * rows + mine;                         // query head of the group
    const bool on = mine < rows && hr < a.group;
    pdl_wait();
    const GroupRec rec = a.group_rec[g];
    const int64_t total = a.group_rec[a.groups.n].before;
    if (!rec.sound) fault = SV_DEVERR_GROUP;
    if (fault && h == 0 && blockIdx.y == 0 && threadIdx.x == 0) svq_flag(fault);
    const int64_t q = static_cast<int64_t>(b) * a.num_q_heads + h * a.group + hr;
    RowSum s;
    if (on && page >= 0 && rec.sound) {
        int k0 = part;
        if (page > 0) {
            const Pieces p = prefix_pieces(prefix, rec, total, a.num_kv_heads, h, e, row * a.group + hr, q);
            s.add(p, k0, per_row, lane);
            k0 = (k0 + per_row - p.n % per_row) % per_row;
        }
        s.add(Pieces{a.split_o, a.split_ml, q * a.splits, q * a.splits + 1, 1, a.splits}, k0, per_row, lane);
    }
    parts[warp][lane] = s;
    __syncthreads();
    if (part == 0 && on) {
        for (int u = 1; u < per_row; ++u) s.join(parts[warp + u][lane]);
        s.write(a.out + q * kHeadDim, a.lse + q, lane);
    }
}

// ---------------------------------------------------------------- host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
    size_t entries, cum, num, req_offset, odd, num_odd, group_rec, cut_item, cut_o, cut_ml, whole_o, whole_ml, split_o, split_ml, total;
    int max_entries, item_rows, slot_rows;
    // rows: query tokens; num_groups: 0 for chunks
    Layout(int64_t batch, int64_t rows, int num_q_heads, int num_kv_heads, int num_groups) {
        const bool prefix = num_groups > 0;
        const int group = num_q_heads / num_kv_heads;
        const int64_t e = prefix ? 0 : rows / (kRowTile / group) + batch;
        max_entries = static_cast<int>(e);
        item_rows = static_cast<int>(rows * group < kRowTile ? rows * group : kRowTile);
        slot_rows = 2 * item_rows < kRowTile ? 2 * item_rows : kRowTile;   // (both streams of up to 128 rows fold theirs)
        size_t at = 0;
        auto take = [&](size_t bytes) { const size_t r = at; at += up(bytes); return r; };
        entries = take(e * sizeof(Entry));
        cum = take((e + 1) * sizeof(int64_t));
        num = take(sizeof(int));
        req_offset = take(prefix ? 0 : batch * sizeof(int));
        cut_item = take(prefix ? 0 : 2 * kMaxCtas * sizeof(int4));
        cut_o = take(2ull * kMaxCtas * slot_rows * kHeadDim * sizeof(float));
        cut_ml = take(2ull * kMaxCtas * slot_rows * sizeof(float2));
        const size_t b = prefix ? batch : 0, heads = b * num_q_heads;
        const size_t parts = prefix ? window_decode_rows(batch, num_q_heads, num_kv_heads) : 0;
        group_rec = take(prefix ? (num_groups + 1) * sizeof(GroupRec) : 0);
        whole_o = take(heads * kHeadDim * sizeof(float));
        whole_ml = take(heads * sizeof(float2));
        split_o = take(parts * kHeadDim * sizeof(float));
        split_ml = take(parts * sizeof(float2));
        // A warp's 32 rows of an item each.  Behind all that every call touches (in front of it: 92.8 against 90.7 us).
        odd = take(8 * e * num_kv_heads * sizeof(uint32_t));
        num_odd = take(sizeof(int));
        total = at + 256;   // the parts begin at the workspace's first multiple of 256 (rows are written 32 bytes at a time)
    }
};

unsigned char* base_of(void* workspace) {
    return reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
}

template <bool FP8>
int launch_attend(const AttendArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int ctas, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    const int st = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(attend_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Cfg<FP8>::kSmem) == cudaSuccess
                   ? SV_OK
                   : SV_ERR_CUDA;
    });
    if (st) return st;
    return launch_pdl(attend_kernel<FP8>, dim3(ctas), dim3(Cfg<FP8>::kThreads), Cfg<FP8>::kSmem, stream, a, tk, tv) ==
                   cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

// The arguments both calls share.
AttendArgs attend_args(const sv_cache* c, const void* q, int num_q_heads, const int32_t* page_table, int max_pages,
                       const Layout& lay, int window, int sink, float softmax_scale, void* out, float* lse,
                       void* workspace) {
    unsigned char* ws = base_of(workspace);
    AttendArgs a = {};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = c->num_kv_heads;
    a.group = num_q_heads / c->num_kv_heads;
    a.page_table = page_table;
    a.max_pages = max_pages;
    a.num_phys_pages = c->num_phys_pages;
    a.k_pool = static_cast<const unsigned char*>(c->k_pool);
    a.v_pool = static_cast<const unsigned char*>(c->v_pool);
    a.k_scale = static_cast<const float*>(c->k_scale);
    a.v_scale = static_cast<const float*>(c->v_scale);
    a.plan.entries = reinterpret_cast<Entry*>(ws + lay.entries);
    a.plan.cum = reinterpret_cast<int64_t*>(ws + lay.cum);
    a.plan.num_entries = reinterpret_cast<int*>(ws + lay.num);
    a.plan.req_offset = reinterpret_cast<int*>(ws + lay.req_offset);
    a.tok_per_entry = kRowTile / a.group;
    a.window = window > 0 ? window : INT_MAX;
    a.sink = sink;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.cut_o = reinterpret_cast<float*>(ws + lay.cut_o);
    a.cut_ml = reinterpret_cast<float2*>(ws + lay.cut_ml);
    a.cut_item = reinterpret_cast<int4*>(ws + lay.cut_item);
    a.odd = reinterpret_cast<uint32_t*>(ws + lay.odd);
    a.num_odd = reinterpret_cast<int*>(ws + lay.num_odd);
    a.fp8 = c->kv_format == SV_KV_FP8_E4M3;
    a.slot_rows = lay.slot_rows;
    return a;
}

int launch_tiles(const sv_cache* c, const AttendArgs& a, int ctas, cudaStream_t stream) {
    CUtensorMap tk = {}, tv = {};
    if (c->kv_format == SV_KV_FP8_E4M3) return launch_attend<true>(a, tk, tv, ctas, stream);
    // TMA coordinates are 32-bit.
    const int64_t groups = c->num_phys_pages * c->num_kv_heads * 2;
    if (groups > INT_MAX) return SV_ERR_UNSUPPORTED;
    if (!encode_pages_map(&tk, c->k_pool, groups) || !encode_pages_map(&tv, c->v_pool, groups)) return SV_ERR_CUDA;
    return launch_attend<false>(a, tk, tv, ctas, stream);
}

int cta_count(int sm_count) { return sm_count < kMaxCtas ? sm_count : kMaxCtas; }

}  // namespace

// One token a request goes to the decode kernel (partials of its splits); chunks to the tiles.
size_t window_workspace_bytes(int batch, int num_q_heads, int num_kv_heads, int total_q) {
    const size_t chunks = Layout(batch, total_q, num_q_heads, num_kv_heads, 0).total;
    const size_t rows = static_cast<size_t>(window_decode_rows(batch, num_q_heads, num_kv_heads));
    const size_t decode = total_q == batch ? up(rows * kHeadDim * sizeof(float)) + up(rows * sizeof(float2)) : 0;
    return chunks > decode ? chunks : decode;
}
size_t prefix_workspace_bytes(int batch, int num_q_heads, int num_kv_heads, int num_groups) {
    return Layout(batch, batch, num_q_heads, num_kv_heads, num_groups).total;
}

int launch_window(const sv_cache* c, const void* q, int num_q_heads, const int32_t* q_start, int total_q,
                  const int32_t* page_table, const int32_t* seq_lens, int batch, int max_pages, int window, int sink,
                  float softmax_scale, void* out, float* lse, void* workspace, int sm_count, cudaStream_t stream) {
    const int ctas = cta_count(sm_count);
    if (!q_start) {
        // Pages of a window that starts anywhere in a page, and of the sinks.
        const int64_t span = window > 0 ? (static_cast<int64_t>(window) + 14) / kPage + 1 + (sink + 15ll) / kPage : max_pages;
        const bool fp8 = c->kv_format == SV_KV_FP8_E4M3;
        const int64_t pages = span < max_pages ? span : max_pages;
        const int cluster = window_decode_cluster(fp8, batch, c->num_kv_heads, pages, ctas, false);
        if (cluster)
            return launch_window_decode(c, q, num_q_heads, page_table, seq_lens, batch, max_pages, window, sink, nullptr,
                                        nullptr, 0, softmax_scale, nullptr, cluster, out, lse, nullptr, nullptr, stream);
        const int splits = window_decode_splits(fp8, batch, c->num_kv_heads, pages, ctas);
        const int64_t heads = static_cast<int64_t>(batch) * num_q_heads;
        float* o = static_cast<float*>(workspace);
        float2* ml = reinterpret_cast<float2*>(static_cast<unsigned char*>(workspace) + up(heads * splits * kHeadDim * sizeof(float)));
        const int st = launch_window_decode(c, q, num_q_heads, page_table, seq_lens, batch, max_pages, window, sink, nullptr,
                                            nullptr, 0, softmax_scale, nullptr, splits, nullptr, nullptr, o, ml, stream);
        return st ? st : launch_join_splits(o, ml, splits, heads, out, lse, stream);
    }
    const Layout lay(batch, total_q, num_q_heads, c->num_kv_heads, 0);
    const AttendArgs a = attend_args(c, q, num_q_heads, page_table, max_pages, lay, window, sink, softmax_scale, out, lse, workspace);
    const PlanArgs p = {a.plan, a.num_odd, lay.max_entries, a.tok_per_entry, q_start, total_q, seq_lens, batch, max_pages,
                        a.window, sink, num_q_heads, a.out, lse};
    if (launch_pdl(plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p) != cudaSuccess) return SV_ERR_CUDA;
    const int st = launch_tiles(c, a, ctas, stream);
    if (st || ctas < 2) return st;
    const int y = lay.item_rows < 32 ? lay.item_rows : (lay.item_rows < 128 ? 32 : 8);
    return launch_pdl(join_cut_kernel, dim3(ctas - 1, y), dim3(kCutThreads), 0, stream, a) == cudaSuccess ? SV_OK
                                                                                                          : SV_ERR_CUDA;
}

int launch_prefix(const sv_cache* c, const void* q, int num_q_heads, const int32_t* page_table,
                  const int32_t* seq_lens, int batch, int max_pages, const int32_t* group_start,
                  const int32_t* shared_pages, int num_groups, float softmax_scale, void* out, float* lse,
                  void* workspace, int sm_count, cudaStream_t stream) {
    const Layout lay(batch, batch, num_q_heads, c->num_kv_heads, num_groups);
    const int ctas = cta_count(sm_count);
    const bool fp8 = c->kv_format == SV_KV_FP8_E4M3;
    if (prefix_alone(fp8, batch, c->num_kv_heads, max_pages))
        return launch_window_decode(c, q, num_q_heads, page_table, seq_lens, batch, max_pages, 0, 0, group_start,
                                    shared_pages, num_groups, softmax_scale, nullptr,
                                    window_decode_cluster(fp8, batch, c->num_kv_heads, max_pages, ctas, true), out, lse,
                                    nullptr, nullptr, stream);
    AttendArgs a = attend_args(c, q, num_q_heads, page_table, max_pages, lay, 0, 0, softmax_scale, out, lse, workspace);
    a.groups = Groups{group_start, shared_pages, num_groups, batch, max_pages};
    a.seq_lens = seq_lens;
    unsigned char* ws = base_of(workspace);
    a.whole_o = reinterpret_cast<float*>(ws + lay.whole_o);
    a.whole_ml = reinterpret_cast<float2*>(ws + lay.whole_ml);
    a.group_rec = reinterpret_cast<GroupRec*>(ws + lay.group_rec);
    a.split_o = reinterpret_cast<float*>(ws + lay.split_o);
    a.split_ml = reinterpret_cast<float2*>(ws + lay.split_ml);
    int st = launch_tiles(c, a, ctas, stream);
    if (st) return st;
    const PrefixParts prefix = {a.group_rec, a.cut_o, a.cut_ml, a.whole_o, a.whole_ml, a.slot_rows, a.tok_per_entry, ctas};
    const int cluster = window_decode_cluster(fp8, batch, c->num_kv_heads, max_pages, ctas, false);
    if (cluster)
        return launch_window_decode(c, q, num_q_heads, page_table, seq_lens, batch, max_pages, 0, 0, group_start,
                                    shared_pages, num_groups, softmax_scale, &prefix, cluster, out, lse, nullptr, nullptr,
                                    stream);
    a.splits = window_decode_splits(fp8, batch, c->num_kv_heads, max_pages, ctas);
    st = launch_window_decode(c, q, num_q_heads, page_table, seq_lens, batch, max_pages, 0, 0, group_start, shared_pages,
                              num_groups, softmax_scale, &prefix, a.splits, nullptr, nullptr, a.split_o, a.split_ml, stream);
    if (st) return st;
    const int rows = batch * c->num_kv_heads, fill = 2 * ctas / rows;   // two CTAs of 512 threads an SM
    const int y = fill < 1 ? 1 : (fill < a.group ? fill : a.group);
    return launch_pdl(join_prefix_kernel, dim3(rows, y), dim3(kPrefixThreads), 0, stream,
                      a, prefix) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

}  // namespace svq
