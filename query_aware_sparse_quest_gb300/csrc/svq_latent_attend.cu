// sv_latent_attention: attention in the absorbed form over the paged latents, on
// the tcgen05 tensor cores.
//
// Mathematics.  All query heads read the same token, so the query tokens of a
// request times the heads are rows of one product, and a key tile's latents C (64
// tokens x 512) are keys and values both.  With Q (rows x 576) and K = C beside the
// rotary keys,
//   S = Q K^T                 (fp32 in TMEM: 64 rows x 64 tokens, 36 MMAs of k = 16 channels)
//   P = exp2(S * scale - base)   (16 bits in shared memory; base = a running maximum a row)
//   O^T = O^T * 2^(old - new base) + C^T P^T   (fp32 in TMEM: 512 channels x rows,
//                             4 MMAs of 128 channels for each 16 tokens)
// The second product is turned round, channels on the MMA's M side and rows on its
// N side: O of 128 rows would take all of TMEM, O^T of 64 takes half of it, and 16
// rows of a single token need no padding to 64.  The other half holds most of Q,
// the first product's M side: from shared memory Q would take 72 KB and as much of
// its bandwidth as K (a tile then moves 327 KB through it, 2555 cycles; 276 KB now).
//
// P is rounded to bf16 because one MMA takes both operands in one type and C is
// bf16 (off by at most 2^-8 of each weight); over bf16 latents the average is taken
// over the sum of the rounded weights, so that rows of equal weights lose nothing.
// Sums, bases and outputs are fp32.
//
// e4m3 latents: codes are widened to fp16 tiles, exactly, by the conversion unit (77
// codes a cycle and SM; to bf16 28).  Q's latent part is fp16 as well, each row
// scaled by a power of two that puts its largest value at 2^10 .. 2^11: values down to
// 2^-27 of that stay exact, smaller ones are off by up to 2^-35 of it.  A token's scale
// acts on its logits and on its weights.  A weight times its scale is rounded to fp16
// (2^-11 of it) in a unit of the row that at most equals the largest so far, so that
// those below 2^-14 of the largest are off by up to 2^-25 of it; the unit moves with
// the base.  The average is taken over the sum of the weights themselves.  The rotary
// part of the logits is a product of its own in bf16 (64 more columns).
//
// Work.  An entry is up to kShare x N rows of a request with the pages they see;
// every group of kShare CTAs takes an equal run of the (entry, key tile) sequence.
// A run that starts or ends inside an entry leaves a partial (O, base, sum), joined
// by a second kernel.
//
// Roles of a CTA (one per SM):
//   warp 1       issues the MMAs
//   warp 2       walks the plan
//   warps 4-7    softmax and outputs: 16 rows each, or where there are fewer than 64 the
//                tokens of a tile shared out (e4m3, 64 rows: warps 4-11, half the tokens each)
//   then         four that load a page of the tile each: units of 64 tokens x 128 channels
//                (16 KB), each freed when its part of the second product is done, and
//                rotary keys (e4m3, 64 rows: warps 0 and 3, two pages each)
//   the last     (e4m3) four that widen the codes
//
// What bounds it (GB300): the MMAs and shared memory, each in the other's way.  64 bf16
// rows: a tile takes 2700 cycles, its MMAs alone 2014, its 276 KB through shared memory
// (operands 194, copies and P 82) 2160 at 128 bytes a cycle; 8 requests of 128 heads at
// 128000 tokens 324 us, 3.6 TB/s and 0.88 PFLOP/s; 512 query tokens at 8192 1.05 ms.
// e4m3: the widened tiles make it 340 KB, 2650 of 3400 cycles, or with 16 rows 290 KB,
// 2270 of 2600: 7 ragged chunks 455 us, 32 requests of 16 heads 165 us (4.3 TB/s).  So
// codes are the slower cache from 33 rows on (8 requests of 128 heads at 32768 tokens 135
// us, bf16 108).  One request: the start, the plan, three tiles and the join, one after
// the other (14.5 us).
#include <cfloat>
#include <climits>
#include <type_traits>

#include "svq_paged.cuh"
#include "svq_tcgen.cuh"

namespace svq {

SVQ_DEFINE_ERROR_WORD(read_error_latent_attend)

namespace {

constexpr int kQueryDim = kLatentDim + kRopeDim;
constexpr int kPages = 4;                           // pages of a key tile
constexpr int kTok = kPages * kPage;                // 64 tokens
constexpr int kUnit = kTok * 128 * 2;               // bytes of 128 channels of a tile
constexpr int kUnits = kLatentDim / 128;            // of a tile
constexpr int kRopeBytes = kTok * kRopeDim * 2;
constexpr int kBlockQ = 64 * 128;                   // bytes of 64 rows x 64 channels
constexpr int kInfoSlots = 8;                       // tiles whose page faults and scales are kept
constexpr int kMaxCtas = 160;                       // partial slots in the workspace
constexpr int kQueryTop = 10;                       // e4m3: the exponent that a row of Q is scaled to for fp16
constexpr float kSlack = 8.f;                       // log2 units a base may lag behind the maximum
constexpr float kBig = 256.f;                       // e4m3: weights times scales, in O's unit, that its unit moves at (fp16 ends at 65504)
// Key tiles after which O moves into fp32 sums and starts again from zero: the MMAs cut their sums off at fp32's last
// bit, four times a tile, always towards zero (values of one sign lose 2^-21.4 of their sum a tile).
constexpr int kFoldTiles = 1024;
constexpr int kMaxRows = 64;                        // rows of a CTA's tile at most

template <int N, bool FP8>
struct Cfg {
    // Units of the ring, two tiles at least, and units of codes, 8 KB each: what shared memory holds.  (e4m3, 16 rows: 8 and
    // 8 189 us for 32 requests, 9 and 6 168, 10 and 4 170, 11 and 2 248.)
    static constexpr int kRing = FP8 ? (N == 64 ? 8 : 9) : (N == 64 ? 11 : 12);
    static constexpr int kCodes = FP8 ? (N == 64 ? 3 : 6) : 0;
    static constexpr int kRope = 2;     // rotary tiles
    static constexpr int kWiden = 4;    // warps that widen, all of them a unit
    // Warps that load.  e4m3, 64 rows: the two that else idle, and eight softmax warps (490 -> 468 us for 7 requests'
    // chunks); with fewer rows a tile is over too soon for two (32 requests of 16 heads 185 us, 165 with four).
    static constexpr int kLoads = FP8 && N == 64 ? 2 : kPages;
    static constexpr int kSoft = FP8 && N == 64 ? 8 : 4;
    // Registers a thread: bf16 168 at launch, then 96 for the first four warps and the loads and 248 for the softmax
    // (128 x (96 + 248 + 96) < 384 x 168); e4m3 128, then 72, 64, 232 and 128 for widening, or with eight softmax warps 96,
    // 160 (twice) and 96.  (The compiler keeps every role's code near the count at launch: with eight warps that widen, 640
    // threads of 96, the softmax took half as long again.  At 128 it spills 32 bytes a thread with 64 e4m3 rows, 4 with 16.)
    static constexpr int kThreads = FP8 ? 512 : 384;
    static constexpr int kFirstWiden = kThreads / 32 - kWiden;
    static constexpr int kMmaRegs = FP8 && kSoft == 4 ? 72 : 96, kSoftmaxRegs = !FP8 ? 248 : (kSoft == 4 ? 232 : 160);
    static constexpr int kLoadRegs = FP8 && kSoft == 4 ? 64 : 96, kWidenRegs = kSoft == 4 ? 128 : 96;
    // Softmax warps that share 16 rows, kCols tokens each.  (Q's rows are repeated on the M side, so every warp's quarter
    // of TMEM holds its rows' logits.)
    static constexpr int kGroups = N / 16, kSplit = kSoft / kGroups, kCols = kTok / kSplit;
    static constexpr int kControl = (FP8 ? 4 : 3) * 1024;
    // TMEM columns: O^T of channels 128 m .. at m N, then S (e4m3: its latent and its rotary part), then the first
    // kQUnits units of Q's channels, two a column.  The others and the rotary ones are in shared memory.
    static constexpr int kSCols = FP8 ? 2 * kTok : kTok;
    static constexpr int kColS = 4 * N, kColQ = kColS + kSCols;
    static constexpr int kQUnits = (512 - kColQ) / 64 < kUnits ? (512 - kColQ) / 64 : kUnits;
    static constexpr int kQBlocks = 2 * (kUnits - kQUnits) + 1;            // of 64 rows x 64 channels
    static constexpr int kQ = kQBlocks * kBlockQ;
    static constexpr int kP = N * kTok * 2;
    static constexpr int kScales = FP8 ? kInfoSlots * kTok * 4 : 0;
    static constexpr int kSmem = kRing * kUnit + kRope * kRopeBytes + kCodes * (kUnit / 2) + kQ + kP + kScales + kControl;
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

struct __align__(16) Entry {
    int row0;      // first row: query token * heads + head
    int nrows;
    int posbase;   // a row's position is posbase + row / heads
    int req;
    int npages;    // pages that some row of it sees
    int tiles;
    int pad[2];
};

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
    bool fp8;
    float scale_log2;
    __nv_bfloat16* out;
    float* lse;
    int share;           // CTAs that work on the rows of an entry side by side
    int tile_rows;       // rows of each (N)
    // Plan
    Entry* entries;
    int64_t* cum;        // [E + 1] cost of the entries before each
    int64_t* total;      // of all
    bool planned;        // by a kernel before; else single tokens of few requests, which every CTA goes through itself
    int* num_entries;
    int* req_first;      // [batch]
    int max_entries;
    // Partials
    float* cut_o;        // [2 CTAs][N][512]
    float4* cut_ml;      // [2 CTAs][N] (base in log2 units, sum, sum of the rounded weights)
    int4* cut_item;      // [groups][2]: row0, nrows, pieces, entry; slots of the first piece and the second (of part 0)
    uint32_t* odd;       // CTAs' row tiles of whole entries that are not finite: entry * share + part
    int* num_odd;
};

// ---------------------------------------------------------------- tensor cores
constexpr uint32_t kF32FromBf16 = (1u << 4) | (1u << 7) | (1u << 10);
constexpr uint32_t kF32FromF16 = 1u << 4;
// (types: of the latents, which e4m3 codes are widened to, and of what is multiplied with them)
template <bool FP8>
constexpr uint32_t idesc(int m, int n) { return (FP8 ? kF32FromF16 : kF32FromBf16) | (static_cast<uint32_t>(n / 8) << 17) | (static_cast<uint32_t>(m / 16) << 24); }
constexpr uint32_t kAIsMMajor = 1u << 15;

#define LATENT_MMA_REGS "{\n\t.reg .pred acc, yes, go;\n\t.reg .b32 al, bl;\n\t.reg .b64 ad, bd;\n\t" \
    "setp.ne.u32 acc, %6, 0;\n\tsetp.ne.u32 go, %7, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\t"
// S (+)= Q K^T over a unit's 128 channels, Q in TMEM or in shared memory: 16 channels are 8 columns of the one and 32
// bytes further in the rows of the other two; the second 64 lie 1 KB on (K) and a block on (Q).  By the whole warp, as
// the others.
__device__ __forceinline__ void mma_qk8_tmem(uint32_t d, uint32_t q, uint32_t k_lo, uint32_t id, uint32_t acc, uint32_t go) {
    asm volatile(
        "{\n\t.reg .pred acc, yes, go;\n\t.reg .b32 al, bl;\n\t.reg .b64 bd;\n\t"
        "setp.ne.u32 acc, %5, 0;\n\tsetp.ne.u32 go, %6, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\t"
        SVQ_MMA_TS_IF(0, 0, acc) SVQ_MMA_TS_IF(8, 2, yes) SVQ_MMA_TS_IF(16, 4, yes) SVQ_MMA_TS_IF(24, 6, yes)
        SVQ_MMA_TS_IF(32, 64, yes) SVQ_MMA_TS_IF(40, 66, yes) SVQ_MMA_TS_IF(48, 68, yes) SVQ_MMA_TS_IF(56, 70, yes)
        "}" ::"r"(d), "r"(q), "r"(k_lo), "r"(desc_hi(2048)), "r"(id), "r"(acc), "r"(go)
        : "memory");
}
__device__ __forceinline__ void mma_qk8(uint32_t d, uint32_t q_lo, uint32_t k_lo, uint32_t id, uint32_t acc, uint32_t go) {
    asm volatile(LATENT_MMA_REGS
        SVQ_MMA_SS_IF(0, 0, acc) SVQ_MMA_SS_IF(2, 2, yes) SVQ_MMA_SS_IF(4, 4, yes) SVQ_MMA_SS_IF(6, 6, yes)
        SVQ_MMA_SS_IF(512, 64, yes) SVQ_MMA_SS_IF(514, 66, yes) SVQ_MMA_SS_IF(516, 68, yes) SVQ_MMA_SS_IF(518, 70, yes)
        "}" ::"r"(d), "r"(q_lo), "r"(k_lo), "r"(desc_hi(1024)), "r"(desc_hi(2048)), "r"(id), "r"(acc), "r"(go)
        : "memory");
}
// The rotary 64 channels.
__device__ __forceinline__ void mma_rope4(uint32_t d, uint32_t q_lo, uint32_t k_lo, uint32_t id, uint32_t acc, uint32_t go) {
    asm volatile(LATENT_MMA_REGS
        SVQ_MMA_SS_IF(0, 0, acc) SVQ_MMA_SS_IF(2, 2, yes) SVQ_MMA_SS_IF(4, 4, yes) SVQ_MMA_SS_IF(6, 6, yes)
        "}" ::"r"(d), "r"(q_lo), "r"(k_lo), "r"(desc_hi(1024)), "r"(desc_hi(1024)), "r"(id), "r"(acc), "r"(go)
        : "memory");
}
// O^T (+)= C^T P^T of 128 channels: a page (16 tokens) is 4 KB of the unit and 32 bytes of P's rows.
__device__ __forceinline__ void mma_pv4(uint32_t d, uint32_t c_lo, uint32_t p_lo, uint32_t id, uint32_t acc, uint32_t go) {
    asm volatile(LATENT_MMA_REGS
        SVQ_MMA_SS_IF(0, 0, acc) SVQ_MMA_SS_IF(256, 2, yes) SVQ_MMA_SS_IF(512, 4, yes) SVQ_MMA_SS_IF(768, 6, yes)
        "}" ::"r"(d), "r"(c_lo), "r"(p_lo), "r"(desc_hi(2048)), "r"(desc_hi(1024)), "r"(id), "r"(acc), "r"(go)
        : "memory");
}
__device__ __forceinline__ void mma_pv1(uint32_t d, uint32_t c_lo, uint32_t p_lo, uint32_t id, uint32_t acc, uint32_t go) {
    asm volatile(LATENT_MMA_REGS
        SVQ_MMA_SS_IF(0, 0, acc)
        "}" ::"r"(d), "r"(c_lo), "r"(p_lo), "r"(desc_hi(2048)), "r"(desc_hi(1024)), "r"(id), "r"(acc), "r"(go)
        : "memory");
}
// 16 rows x 2 K columns: lane l gets rows l / 4 and + 8 of columns 8 c + 2 (l % 4), + 1, at x[4 c ..] and x[4 c + 2 ..].
template <int K>
__device__ __forceinline__ void tc_ld_rows(uint32_t addr, float (&x)[K]) {
    uint32_t(&r)[K] = reinterpret_cast<uint32_t(&)[K]>(x);
    static_assert(K == 8 || K == 16 || K == 32);
    if constexpr (K == 8)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr));
    else if constexpr (K == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(addr));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
            "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
            "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
              "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
              "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(addr));
}
// 16 rows of 32 columns: lanes 0 .. 15 have the rows' first 16, lanes 16 .. 31 the others.
__device__ __forceinline__ void tc_st_halves(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], 16, {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// Four 8 x 8 blocks of 16-bit values: lane l gives the address of row l % 8 of block l / 8.
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// Copies by a whole warp in step, of which the elected lane issues (go): from four lanes at once each takes 130 cycles.
__device__ __forceinline__ void tma_page_if(uint32_t go, uint32_t dst, const void* map, int half, int group, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred go;\n\tsetp.ne.u32 go, %6, 0;\n\t"
        "@go cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3, %4}], [%5];\n\t}"
        ::"r"(dst), "l"(map), "r"(0), "r"(half), "r"(group), "r"(bar), "r"(go)
        : "memory");
}
__device__ __forceinline__ void tma_2d_if(uint32_t go, uint32_t dst, const void* map, int x, int y, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred go;\n\tsetp.ne.u32 go, %5, 0;\n\t"
        "@go cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar), "r"(go)
        : "memory");
}
// The softmax warps' barrier.
template <int WARPS>
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(32 * WARPS) : "memory"); }
template <int WARPS>
__device__ __forceinline__ bool softmax_any(bool mine) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, r;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred r, 1, %2, p;\n\tselp.u32 %0, 1, 0, r;\n\t}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(mine)), "n"(32 * WARPS)
        : "memory");
    return any != 0;
}

// The softmax warps meet at barriers, so they leave together: a warp whose wait ran out says so at the next one.
#define LATENT_WAIT(bar, parity)                                                    \
    do {                                                                            \
        if (__any_sync(0xffffffffu, !bar_ready(smem_addr(&(bar)), (parity)))) {      \
            if (lane == 0) gave_up(ct);                                             \
            dead = true;                                                            \
        }                                                                           \
    } while (0)

// A run of key tiles of one entry; none: the CTA's work is over.
struct __align__(16) Seg {
    Entry en;
    int t0, t1;
    int slot;         // where a partial goes; -1 - entry: the segment is the whole entry
    int pad;
};
constexpr int kSegs = 4;
// Single tokens of at most so many requests: an entry is a request, and every CTA sums up their costs by itself (a plan
// kernel before takes 3 us; one request of 4096 tokens 25.5 -> 22 us).
constexpr int kOwnPlan = 256;

template <int SOFT, bool FP8>   // softmax warps
struct Control {
    uint64_t full[12], empty[12];          // units
    uint64_t rope_full[2], rope_empty[2];
    uint64_t code_full[8], code_empty[8];
    uint64_t scale_full[kInfoSlots];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t s_full, s_read, p_full, pv_done, q_full, vote, drain;
    uint32_t tmem;
    int gave_up;
    uint8_t fault[kInfoSlots][kPages];     // pages of a tile that the table does not give
    int over[4];                           // a logit of the tile is too far above its row's base
    int lens[kOwnPlan];                       // of the requests, where the CTA plans by itself
    Seg seg[kSegs];
    // Rows' maxima of the warps that share them, and at a segment's end their sums.
    union {
        struct {
            float top[16 * SOFT], big[16 * SOFT];
        };
        float2 sum[16 * SOFT];
    };
    float unit[FP8 ? kMaxRows : 1];        // e4m3: of the rows of Q
    alignas(16) float alpha[kMaxRows], factor[kMaxRows];   // of a row's O: where its base moves, and at a segment's end
};

template <int SOFT, bool FP8>
__device__ __forceinline__ void gave_up(Control<SOFT, FP8>* ct) {
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

// What an entry costs beside its tiles, in tiles (Q, the first tile's bases, the outputs: 64 rows take 25000 cycles, and
// with 3 for them 7 requests' e4m3 chunks take 603 us, with 9 490, with 14 520; seven others with 5 / 9 / 13: e4m3 1099 / 956
// / 976, bf16 732 / 662 / 680; 300 tokens of 128 heads 102 / 94 / 88 and 75 / 69 / 68; 40 single tokens of 64 heads at 3000 60 /
// 61 / 65 and 57 / 58 / 60; 16 rows 1: 32 requests 169 us, 3: 165, 5: 164), and the least share that is worth a CTA (one request
// of 64 tiles and 16 heads: 1 20.1 us, 2 19.5, 3 17.4, 4 18.0; later 2 / 3 / 5, bf16: 16 heads at 1000 tokens 12.9 / 13.9 /
// 15.5, 4096 14.9 / 15.4 / 16.1, 16000 24.2 / 21.0 / 20.5; 128 heads 20.3 / 18.9 / 21.7, 29.1 / 24.9 / 24.2, 45.9 / 46.6 / 37.8).
constexpr int kMinShare = 3;
__host__ __device__ constexpr int entry_cost(int rows) { return rows == 64 ? 9 : 3; }
__device__ __forceinline__ int cost_of_entry(int tiles, int rows) { return tiles ? tiles + entry_cost(rows) : 0; }
// Groups of CTAs that share the work.
__device__ __forceinline__ int groups_of(int64_t total, int most) {
    const int64_t n = (total + kMinShare - 1) / kMinShare;
    return n < 1 ? 1 : (n < most ? static_cast<int>(n) : most);
}
struct PlacedEntry {
    int64_t begin;
    int c0, c1;
    __device__ __forceinline__ PlacedEntry(const Share& share, int64_t at, int n, int rows)
        : begin(at), c0(share.cta_of(at + entry_cost(rows))), c1(share.cta_of(at + entry_cost(rows) + n - 1)) {}
};

template <int N, bool FP8>
__global__ void __launch_bounds__(Cfg<N, FP8>::kThreads, 1)
    latent_kernel(const __grid_constant__ LatentArgs a, const __grid_constant__ CUtensorMap tmap_c,
                  const __grid_constant__ CUtensorMap tmap_r) {
    using C = Cfg<N, FP8>;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* const ring = smem;
    unsigned char* const ropes = ring + C::kRing * kUnit;
    unsigned char* const codes = ropes + C::kRope * kRopeBytes;
    unsigned char* const qs = codes + C::kCodes * (kUnit / 2);
    unsigned char* const ps = qs + C::kQ;
    float* const scales = reinterpret_cast<float*>(ps + C::kP);
    using Ctrl = Control<C::kSoft, FP8>;
    static_assert(sizeof(Ctrl) <= C::kControl, "control block");
    Ctrl* const ct = reinterpret_cast<Ctrl*>(ps + C::kP + C::kScales);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = blockIdx.x % a.share, group = blockIdx.x / a.share;

    if (threadIdx.x == 0) {
        ct->gave_up = 0;
        for (int i = 0; i < C::kRing; ++i) {
            mbar_init(smem_addr(&ct->full[i]), FP8 ? C::kWiden : kPages);
            mbar_init(smem_addr(&ct->empty[i]), 1);
        }
        for (int i = 0; i < C::kRope; ++i) {
            mbar_init(smem_addr(&ct->rope_full[i]), kPages);
            mbar_init(smem_addr(&ct->rope_empty[i]), 1);
        }
        for (int i = 0; i < C::kCodes; ++i) {
            mbar_init(smem_addr(&ct->code_full[i]), kPages);
            mbar_init(smem_addr(&ct->code_empty[i]), C::kWiden);
        }
        for (int i = 0; i < kInfoSlots; ++i) mbar_init(smem_addr(&ct->scale_full[i]), kPages);
        for (int i = 0; i < kSegs; ++i) {
            mbar_init(smem_addr(&ct->seg_full[i]), 1);
            mbar_init(smem_addr(&ct->seg_empty[i]), C::kLoads + 1 + C::kSoft + (FP8 ? C::kWiden : 0));   // loads, MMAs, softmax, widening
        }
        mbar_init(smem_addr(&ct->s_full), 1);
        mbar_init(smem_addr(&ct->s_read), C::kSoft);
        mbar_init(smem_addr(&ct->p_full), C::kSoft);
        mbar_init(smem_addr(&ct->pv_done), 1);
        mbar_init(smem_addr(&ct->q_full), 4);
        mbar_init(smem_addr(&ct->vote), C::kSoft);
        for (int i = 0; i < 4; ++i) ct->over[i] = 0;
        mbar_init(smem_addr(&ct->drain), 1);
        mbar_init_fence();
        prefetch_tmap(&tmap_c);
        prefetch_tmap(&tmap_r);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&ct->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_wait();
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
        if (warp == 1) {
            // ---------------- MMAs: the whole warp, in step.  The tensor pipe queues next to nothing, so whatever the warp
            // does between two MMAs is lost: a tile is waited for once, its MMAs follow one another, and there is one
            // copy of each product in the code (the roles share the instruction caches).
            reg_dec<C::kMmaRegs>();
            const uint32_t go = elected();
            uint32_t tile = 0, segs = 0;   // tiles before the segment; segments with tiles
            const uint32_t ring_s = smem_addr(ring), q_s = smem_addr(qs), p_lo = desc_lo(smem_addr(ps), 16);
            auto wait = [&](uint64_t& bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_ready(smem_addr(&bar), parity)) != 0; };
            auto test = [&](uint64_t& bar, uint32_t parity) { return __all_sync(0xffffffffu, bar_test(smem_addr(&bar), parity)) != 0; };
            auto commit = [&](uint64_t& bar) {
                if (go) mma_commit(smem_addr(&bar));
            };
            uint32_t qk_slot = 0, qk_ph = 0, pv_slot = 0, rope = 0, rope_ph = 0;   // places in the rings, and their phases
            auto next = [](uint32_t slot, uint32_t by) { return slot + by >= C::kRing ? slot + by - C::kRing : slot + by; };
            bool ok = true;
            for (uint32_t k = 0; ok; ++k) {
                ok = wait(ct->seg_full[k % kSegs], (k / kSegs) & 1);
                const Seg& s = ct->seg[k % kSegs];
                const int n = uniform(s.t1 - s.t0);
                if (!ok || n == 0) break;
                int pages = uniform(s.en.npages - s.t0 * kPages);   // from the tile of the second product on
                ok = wait(ct->q_full, segs & 1);
                ++segs;
                // S of tile t, then the product with P of the tile before: while the softmax works on one tile the tensor
                // cores work on the next.  What the start of the one needs is asked for between the MMAs of the other, which
                // the queue covers (`seen`: the first unit, the rotary keys, S of the tile before read; and P).
                uint32_t seen = 0;
                bool p_seen = false;
#pragma unroll 1
                for (int i = 0; i <= n && ok; ++i) {
                    const uint32_t t = tile + i;
                    if (i < n) {
                        const uint32_t d = tmem + C::kColS;
                        if (t > 0 && !((seen >> (kUnits + 1)) & 1u)) ok = wait(ct->s_read, (t - 1) & 1);
#pragma unroll
                        for (int u = 0; u < kUnits; ++u) {
                            const uint32_t slot = next(qk_slot, u);
                            if (!((seen >> u) & 1u)) ok = ok && wait(ct->full[slot], qk_ph ^ (slot < qk_slot));
                            if (!ok) break;
                            if (u == 0 || !((seen >> u) & 1u)) tc_fence_after();
                            const uint32_t k_lo = desc_lo(ring_s + slot * kUnit, 16);
                            if (u < C::kQUnits) mma_qk8_tmem(d, tmem + C::kColQ + u * 64, k_lo, idesc<FP8>(64, kTok), u != 0, go);
                            else mma_qk8(d, desc_lo(q_s + 2 * (u - C::kQUnits) * kBlockQ, 16), k_lo, idesc<FP8>(64, kTok), u != 0, go);
                        }
                        if (ok && !((seen >> kUnits) & 1u)) ok = wait(ct->rope_full[rope], rope_ph);
                        if (!ok) break;
                        tc_fence_after();
                        mma_rope4(FP8 ? d + kTok : d, desc_lo(q_s + (C::kQBlocks - 1) * kBlockQ, 16),
                                  desc_lo(smem_addr(ropes) + rope * kRopeBytes, 16), idesc<false>(64, kTok), !FP8, go);
                        p_seen = i > 0 && test(ct->p_full, (t - 1) & 1);
                        commit(ct->s_full);
                        commit(ct->rope_empty[rope]);
                        qk_ph ^= qk_slot + kUnits >= C::kRing;
                        qk_slot = next(qk_slot, kUnits);
                        rope_ph ^= rope + 1 == C::kRope;
                        rope = rope + 1 == C::kRope ? 0 : rope + 1;
                    }
                    seen = 0;
                    if (i > 0) {
                        if (!p_seen || i == n) ok = wait(ct->p_full, (t - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const bool acc = ((i - 1) & (kFoldTiles - 1)) != 0;
                        if (pages >= kPages) {
#pragma unroll
                            for (int u = 0; u < kUnits; ++u) {
                                const uint32_t slot = next(pv_slot, u);
                                mma_pv4(tmem + u * N, desc_lo(ring_s + slot * kUnit, 1024), p_lo, idesc<FP8>(128, N) | kAIsMMajor, acc, go);
                                if (u == kUnits - 1) {
                                    seen |= test(ct->rope_full[rope], rope_ph) ? 1u << kUnits : 0u;
                                    seen |= test(ct->s_read, t & 1) ? 2u << kUnits : 0u;
                                } else if (u == 0) {
                                    seen |= test(ct->full[qk_slot], qk_ph) ? 1u : 0u;
                                }
                                commit(ct->empty[slot]);
                            }
                        } else {
#pragma unroll 1
                            for (int u = 0; u < kUnits; ++u) {
                                const uint32_t slot = next(pv_slot, u), c_lo = desc_lo(ring_s + slot * kUnit, 1024);
                                for (int p = 0; p < pages; ++p)
                                    mma_pv1(tmem + u * N, c_lo + p * 256, p_lo + p * 2, idesc<FP8>(128, N) | kAIsMMajor, acc || p != 0, go);
                                commit(ct->empty[slot]);
                            }
                        }
                        commit(ct->pv_done);
                        pv_slot = next(pv_slot, kUnits);
                        pages -= kPages;
                    }
                }
                tile += n;
                if (ok && go) mbar_arrive(smem_addr(&ct->seg_empty[k % kSegs]));
            }
            if (!ok && go) gave_up(ct);
            commit(ct->drain);   // nothing of this CTA's is in flight when TMEM is freed
            (void)wait(ct->drain, 0);
            __syncwarp();
        } else if (warp == 2) {
            // ---------------- the group's share of the plan, segment by segment
            reg_dec<C::kMmaRegs>();
            int num_entries;
            int64_t total = 0;
            auto own_cost = [&](int b) { return cost_of_entry((ct->lens[b] + kTok - 1) / kTok, N); };
            if (a.planned) {
                num_entries = *a.num_entries;
                total = *a.total;
            } else {
                num_entries = a.batch;
                for (int b0 = 0; b0 < a.batch; b0 += 32) {
                    const int b = b0 + lane;
                    int64_t cost = 0;
                    if (b < a.batch) {
                        int len = a.seq_lens[b];
                        if (len < 0 || (static_cast<int64_t>(len) + kPage - 1) / kPage > a.max_pages) {
                            if (blockIdx.x == 0) svq_flag(SV_DEVERR_SEQ_LEN);
                            len = 0;
                        }
                        ct->lens[b] = len;
                        cost = own_cost(b);
                    }
#pragma unroll
                    for (int d = 16; d; d >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, d);
                    total += cost;
                }
                if (blockIdx.x == 0 && lane == 0) *a.total = total;   // for the join
                __syncwarp();
            }
            const int groups = groups_of(total, gridDim.x / a.share);
            const Share share(total, groups);
            const int64_t first = group < groups ? share.start(group) : total;
            int64_t left = group < groups ? share.start(group + 1) - first : 0;
            int e = 0;
            int64_t off = 0;                 // into the entry's cost
            if (left > 0) {
                if (a.planned) {
                    e = warp_find_le(a.cum, num_entries, first);
                    off = first - a.cum[e];
                } else {
                    int64_t before = 0;
                    for (int b0 = 0;; b0 += 32) {
                        const int b = b0 + lane;
                        const int64_t cost = b < a.batch ? own_cost(b) : 0;
                        int64_t x = cost;
#pragma unroll
                        for (int d = 1; d < 32; d <<= 1) {
                            const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
                            if (lane >= d) x += y;
                        }
                        const uint32_t here = __ballot_sync(0xffffffffu, before + x > first);
                        if (here) {
                            const int src = __ffs(here) - 1;
                            e = b0 + src;
                            off = first - __shfl_sync(0xffffffffu, before + x - cost, src);
                            break;
                        }
                        before += __shfl_sync(0xffffffffu, x, 31);
                    }
                }
            }
            auto entry = [&](int e) {
                if (a.planned) {
                    const int4* p = reinterpret_cast<const int4*>(a.entries + e);
                    const int4 x = p[0], y = p[1];
                    return Entry{x.x, x.y, x.z, x.w, y.x, y.y, {0, 0}};
                }
                const int pages = (ct->lens[e] + kPage - 1) / kPage;
                return Entry{e * a.heads, a.heads, ct->lens[e] - e - 1, e, pages, (pages + kPages - 1) / kPages, {0, 0}};
            };
            const int64_t into = off;        // (where the share begins inside its first entry)
            if (left <= 0 && lane == 0 && part == 0) a.cut_item[2 * group] = make_int4(0, 0, 0, 0);
            bool first_item = true, name = left > 0;
            Entry en = {};
            for (uint32_t k = 0;;) {
                int t0 = 0, t1 = 0;
                if (left > 0) {
                    if (off == 0 || first_item) {
                        do en = entry(e);   // (entries without tiles: rows that see nothing)
                        while (en.tiles == 0 && ++e < num_entries);
                    }
                    const int64_t take = min(left, cost_of_entry(en.tiles, N) - off);
                    t0 = static_cast<int>(max(static_cast<int64_t>(0), off - entry_cost(N)));
                    t1 = static_cast<int>(max(static_cast<int64_t>(0), off + take - entry_cost(N)));
                    left -= take;
                    off += take;
                }
                const int rows = min(N, en.nrows - part * N);
                bool over = false;   // the last one
                if ((t1 > t0 && rows > 0) || left <= 0) {
                    for (int round = 0;; ++round) {
                        if (!__any_sync(0xffffffffu, !bar_wait(smem_addr(&ct->seg_empty[k % kSegs]), ((k / kSegs) & 1) ^ 1))) break;
                        if (__any_sync(0xffffffffu, *static_cast<volatile int*>(&ct->gave_up)) || round == kSegRounds) {
                            if (lane == 0) gave_up(ct);
                            goto plan_end;
                        }
                    }
                    over = t1 == t0 || rows <= 0;
                    if (lane == 0) {
                        Seg& s = ct->seg[k % kSegs];
                        s.en = en;
                        s.en.row0 += part * N;
                        s.en.nrows = rows;
                        s.t0 = over ? 0 : t0;
                        s.t1 = over ? 0 : t1;
                        s.slot = t0 == 0 && t1 == en.tiles ? -1 - e : 2 * static_cast<int>(blockIdx.x) + (first_item ? 0 : 1);
                        mbar_arrive(smem_addr(&ct->seg_full[k % kSegs]));
                    }
                    ++k;
                }
                if (name && lane == 0 && part == 0) {
                    // The group after the one with an entry's first tile names the entry for the join.
                    int4 what = make_int4(0, 0, 0, 0), where = make_int4(0, 0, 0, 0);
                    if (into > 0) {
                        const PlacedEntry it(share, first - into, en.tiles, N);
                        if (group == it.c0 + 1) {
                            what = make_int4(en.row0, en.nrows, it.c1 - it.c0 + 1, e);
                            where.x = 2 * it.c0 + (share.start(it.c0) >= it.begin ? 0 : 1);
                            where.y = 2 * (it.c0 + 1);
                        }
                    }
                    a.cut_item[2 * group] = what;
                    a.cut_item[2 * group + 1] = where;
                }
                if (over) break;
                first_item = name = false;
                if (off == cost_of_entry(en.tiles, N)) {
                    off = 0;
                    ++e;
                }
            }
        plan_end:
            // Requests without tokens: a group takes those at its distance.
            for (int b = group; !a.planned && part == 0 && b < a.batch; b += gridDim.x / a.share) {
                if (ct->lens[b]) continue;
                const int64_t r0 = static_cast<int64_t>(b) * a.heads;
                uint4* const o = reinterpret_cast<uint4*>(a.out + r0 * kLatentDim);
                for (int i = lane; i < a.heads * (kLatentDim / 8); i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
                for (int i = lane; i < a.heads; i += 32) a.lse[r0 + i] = -INFINITY;
            }
        } else if (warp >= 4 && warp < 4 + C::kSoft) {
            // ---------------- softmax: warp w rows 16 (w % kGroups) .. and kCols tokens from tok0 on, lane l rows l / 4 and
            // + 8 of those and tokens 8 c + 2 (l % 4), + 1
            constexpr int kC = C::kCols / 8;
            reg_inc<C::kSoftmaxRegs>();
            const int w = warp - 4, tid = threadIdx.x - 128;
            const int rg = w % C::kGroups, tp = w / C::kGroups, tok0 = tp * C::kCols;
            const int quad = lane & 3;
            const uint32_t lanes = static_cast<uint32_t>((w & 3) * 32) << 16;
            // O^T's columns from first_col on are this warp's to scale and to write, its channels 128 u + chan.
            constexpr int kOCols = 4 * N / (C::kSoft / 4);
            const int first_col = (w >> 2) * kOCols, chan = tid & 127;
            uint32_t tile = 0;
            bool dead = false;   // a wait of this warp's ran out
            // Q of a segment's rows: the first units to TMEM, where row r is lane 32 (r / 16) + r % 16, the rest to shared
            // memory.  Eight lanes read a row, rows 4 i + lane / 8 and chunks of 8 channels (a row a lane would touch 32
            // lines a load), and the way to TMEM leads through the warp's rows of the last block.
            auto load_q = [&](int row0, int nrows) {
                if (w >= 4) return;   // (the first four)
                if (16 * rg < nrows) {
                    constexpr int kBlocks = kQueryDim / 64;
                    const uint4* from[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        from[i] = reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(row0 + min(16 * rg + 4 * i + (lane >> 3), nrows - 1)) * kQueryDim) + (lane & 7);
                    float shrink[4];
                    if (FP8) {
                        // The rows' largest exponents (of their finite values).
                        uint32_t top[4] = {0, 0, 0, 0};
#pragma unroll
                        for (int c = 0; c < kBlocks - 1; ++c)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint4 v = from[i][8 * c];
                                top[i] = __vmaxu2(top[i], __vmaxu2(__vmaxu2(v.x & 0x7f807f80u, v.y & 0x7f807f80u), __vmaxu2(v.z & 0x7f807f80u, v.w & 0x7f807f80u)));
                            }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t t = max(top[i] >> 16, top[i] & 0xffffu);
#pragma unroll
                            for (int d = 1; d < 8; d <<= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, d));
                            const int up = max(static_cast<int>(min(t >> 7, 254u)) - 127 - kQueryTop, -126);
                            shrink[i] = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
                            if ((lane & 7) == 0) ct->unit[16 * w + 4 * i + (lane >> 3)] = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
                        }
                    }
                    constexpr int kBatch = 5;   // blocks on their way at a time
                    unsigned char* const to = qs + w * 2048, * const way = to + (C::kQBlocks - 1) * kBlockQ;
                    auto put = [](unsigned char* at, int r, int chunk) { return reinterpret_cast<uint4*>(at + r * 128 + ((chunk ^ (r & 7)) << 4)); };
#pragma unroll
                    for (int c0 = 0; c0 < kBlocks; c0 += kBatch) {
                        uint4 x[kBatch][4];
#pragma unroll
                        for (int c = c0; c < c0 + kBatch && c < kBlocks; ++c)
#pragma unroll
                            for (int i = 0; i < 4; ++i) x[c - c0][i] = from[i][8 * c];
#pragma unroll
                        for (int c = c0; c < c0 + kBatch && c < kBlocks; ++c) {
                            const bool to_tmem = c < 2 * C::kQUnits;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint4 v = x[c - c0][i];
                                if (FP8 && c < kBlocks - 1) {
                                    auto half2 = [&](uint32_t e) {
                                        float y, z;
                                        unpack2(mul2(pack2(bf16lo(e), bf16hi(e)), pack2(shrink[i], shrink[i])), y, z);
                                        return pack_f16x2(y, z);
                                    };
                                    v = make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
                                }
                                *put(to_tmem ? way : to + (c - 2 * C::kQUnits) * kBlockQ, 4 * i + (lane >> 3), lane & 7) = v;
                            }
                            if (to_tmem) {
                                __syncwarp();
                                uint32_t y[16];   // half of row l % 16
#pragma unroll
                                for (int u = 0; u < 4; ++u) *reinterpret_cast<uint4*>(&y[4 * u]) = *put(way, lane & 15, (lane >> 4) * 4 + u);
                                tc_st_halves(tmem + lanes + C::kColQ + c * 32, y);
                                __syncwarp();
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ct->q_full));
            };
            for (uint32_t k = 0;; ++k) {
                const Seg& s = ct->seg[k % kSegs];
                if (k == 0) {
                    // The rows of a single request are known before the plan (one request of 4096 tokens 15.3 -> 14.5 us).
                    const bool known = !a.planned && a.batch == 1;
                    if (!known) {
                        LATENT_WAIT(ct->seg_full[0], 0);
                        if (softmax_any<C::kSoft>(dead)) goto softmax_end;
                    }
                    const int rows = known ? min(N, a.heads - part * N) : s.en.nrows;
                    if (known || s.t1 > s.t0) load_q(known ? part * N : s.en.row0, rows);
                    if (known) {
                        LATENT_WAIT(ct->seg_full[0], 0);
                        if (softmax_any<C::kSoft>(dead)) goto softmax_end;
                    }
                }
                const int n = s.t1 - s.t0;
                if (n == 0) break;
                LATENT_WAIT(ct->seg_full[(k + 1) % kSegs], ((k + 1) / kSegs) & 1);
                if (softmax_any<C::kSoft>(dead)) goto softmax_end;
                const Seg& nx = ct->seg[(k + 1) % kSegs];
                // e4m3: what the lane's rows of Q are in units of (the barrier has passed since they were written).
                const float qs0 = FP8 ? ct->unit[16 * (w & 3) + (lane >> 2)] : 1.f, qs1 = FP8 ? ct->unit[16 * (w & 3) + 8 + (lane >> 2)] : 1.f;
                const int rows = s.en.nrows;
                // Tokens that a row sees.
                auto see = [&](int r) { return s.en.posbase + (s.en.row0 + min(r, rows - 1)) / a.heads + 1; };
                const int see_all = see(0), see_any = see(rows - 1);
                const int r0 = 16 * rg + (lane >> 2), r1 = r0 + 8;
                const int lim0 = see(r0), lim1 = see(r1);
                const bool on = 16 * rg < rows;         // (warps without rows have no logits, but their share of O)
                float m0 = -INFINITY, m1 = -INFINITY;   // the rows' bases
                // e4m3: O is in units of 2^up, so that the largest weight times its token's scale is about 1 in fp16.
                float up0 = -126.f, up1 = -126.f;
                float l0 = 0.f, l1 = 0.f, lr0 = 0.f, lr1 = 0.f;
                float folded0 = -INFINITY, folded1 = -INFINITY;   // the bases of what was folded
                float* const fold_to = a.cut_o + static_cast<int64_t>(s.slot >= 0 ? s.slot : 2 * static_cast<int>(blockIdx.x) + 1) * N * kLatentDim;
                // The rows' factors, by the lane that has them first; all read them behind a barrier.
                auto publish = [&](float* to, float f0, float f1) {
                    if (quad == 0 && tp == 0) {
                        to[r0] = f0;
                        to[r1] = f1;
                    }
                };
                // Maxima over the warps that share the rows, in `at`, a warp's 16 rows each.
                auto across = [&](float* at, float& v0, float& v1) {
                    if (quad == 0) {
                        at[16 * w + (lane >> 2)] = v0;
                        at[16 * w + 8 + (lane >> 2)] = v1;
                    }
                    softmax_sync<C::kSoft>();
#pragma unroll
                    for (int i = 0; i < C::kSplit; ++i) {
                        v0 = fmaxf(v0, at[i * N + r0]);
                        v1 = fmaxf(v1, at[i * N + r1]);
                    }
                };
                for (int j = 0; j < n; ++j, ++tile) {
                    const int first = (s.t0 + j) * kTok;
                    const int slot = tile % kInfoSlots;
                    LATENT_WAIT(ct->s_full, tile & 1);
                    tc_fence_after();
                    const uint32_t fault = *reinterpret_cast<const uint32_t*>(ct->fault[slot]);
                    float x[4 * kC];
                    if (on) {
                        tc_ld_rows(tmem + lanes + C::kColS + tok0, x);
                        tc_wait_ld();
                        if (FP8) {
                            float y[4 * kC];
                            tc_ld_rows(tmem + lanes + C::kColS + kTok + tok0, y);
                            tc_wait_ld();
                            LATENT_WAIT(ct->scale_full[slot], (tile / kInfoSlots) & 1);
#pragma unroll
                            for (int c = 0; c < kC; ++c) {
                                const float2 sc = *reinterpret_cast<const float2*>(&scales[slot * kTok + tok0 + 8 * c + 2 * quad]);
                                const uint64_t s2 = pack2(sc.x, sc.y);
                                unpack2(fma2(mul2(pack2(x[4 * c], x[4 * c + 1]), pack2(qs0, qs0)), s2, pack2(y[4 * c], y[4 * c + 1])),
                                        x[4 * c], x[4 * c + 1]);
                                unpack2(fma2(mul2(pack2(x[4 * c + 2], x[4 * c + 3]), pack2(qs1, qs1)), s2, pack2(y[4 * c + 2], y[4 * c + 3])),
                                        x[4 * c + 2], x[4 * c + 3]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ct->s_read));
                    const bool plain = first + kTok <= see_all && !fault;
                    if (on && !plain) {
#pragma unroll
                        for (int c = 0; c < kC; ++c) {
                            const bool gone = (fault >> ((tok0 / 16 + c / 2) * 8)) & 1u;
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int tok = first + tok0 + 8 * c + 2 * quad + u;
                                if (gone || tok >= lim0) x[4 * c + u] = -INFINITY;
                                if (gone || tok >= lim1) x[4 * c + 2 + u] = -INFINITY;
                            }
                        }
                    }
                    // Weights go by the rows' bases as they are, unless a logit is more than kSlack above its row's: then
                    // (at a run's first tile, and seldom behind it) the tile's maxima move the bases.  The warps say so to
                    // one another while they work out the weights, as each holds channels of all rows' O.  A row without
                    // a base has seen nothing in the run's tiles so far (pages that are not there): there any finite logit
                    // is far above -FLT_MAX, and -inf, all that such a row has in a tile if its base does not move, has the
                    // weight 0.
                    uint32_t p[kC][2];
                    float add0, add1, add_r0, add_r1, over = -INFINITY;
                    float big0, big1;   // e4m3: the largest weight times scale, in O's unit
                    auto weights = [&](float g0, float g1) {
                        big0 = big1 = 0.f;
                        const float b0 = m0 == -INFINITY ? -FLT_MAX : m0, b1 = m1 == -INFINITY ? -FLT_MAX : m1;
                        const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), base0 = pack2(-b0, -b0), base1 = pack2(-b1, -b1);
                        uint64_t sum0 = 0ull, sum1 = 0ull, sumr0 = 0ull, sumr1 = 0ull;
#pragma unroll
                        for (int c = 0; c < kC; ++c) {
                            float y[4];
                            unpack2(fma2(pack2(x[4 * c], x[4 * c + 1]), scale2, base0), y[0], y[1]);
                            unpack2(fma2(pack2(x[4 * c + 2], x[4 * c + 3]), scale2, base1), y[2], y[3]);
                            over = fmaxf(over, fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])));
                            uint64_t e0 = pack2(ex2(y[0]), ex2(y[1])), e1 = pack2(ex2(y[2]), ex2(y[3]));
                            sum0 = add2(sum0, e0);
                            sum1 = add2(sum1, e1);
                            if (FP8) {
                                // (Scales of tokens that no row sees may hold anything.)
                                const float2 sc = *reinterpret_cast<const float2*>(&scales[slot * kTok + tok0 + 8 * c + 2 * quad]);
                                const int tok = first + tok0 + 8 * c + 2 * quad;
                                const bool gone = (fault >> ((tok0 / 16 + c / 2) * 8)) & 1u;
                                const uint64_t s2 = plain ? pack2(sc.x, sc.y)
                                                          : pack2(gone || tok >= see_any ? 0.f : sc.x, gone || tok + 1 >= see_any ? 0.f : sc.y);
                                e0 = mul2(mul2(e0, s2), pack2(g0, g0));
                                e1 = mul2(mul2(e1, s2), pack2(g1, g1));
                            }
                            unpack2(e0, y[0], y[1]);
                            unpack2(e1, y[2], y[3]);
                            if (FP8) {
                                big0 = fmaxf(big0, fmaxf(fabsf(y[0]), fabsf(y[1])));
                                big1 = fmaxf(big1, fmaxf(fabsf(y[2]), fabsf(y[3])));
                            }
                            p[c][0] = FP8 ? pack_f16x2(y[0], y[1]) : pack_bf16x2(y[0], y[1]);
                            p[c][1] = FP8 ? pack_f16x2(y[2], y[3]) : pack_bf16x2(y[2], y[3]);
                            if (!FP8) {
                                sumr0 = add2(sumr0, pack2(bf16lo(p[c][0]), bf16hi(p[c][0])));
                                sumr1 = add2(sumr1, pack2(bf16lo(p[c][1]), bf16hi(p[c][1])));
                            }
                        }
                        float u, v;
                        unpack2(sum0, u, v);
                        add0 = u + v;
                        unpack2(sum1, u, v);
                        add1 = u + v;
                        unpack2(sumr0, u, v);
                        add_r0 = u + v;
                        unpack2(sumr1, u, v);
                        add_r1 = u + v;
                    };
                    if (j > 0) {
                        if (on) weights(FP8 ? ex2(-up0) : 1.f, FP8 ? ex2(-up1) : 1.f);
                        if (dead || over > kSlack || (FP8 && on && fmaxf(big0, big1) > kBig)) *static_cast<volatile int*>(&ct->over[tile & 3]) = 1;
                    } else if (lane == 0) {
                        *static_cast<volatile int*>(&ct->over[tile & 3]) = 1;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ct->vote));
                    // (P's memory and O are free when the product before is done: the same look asks for that.)
                    {
                        const bool vote = lane == 0 || j == 0;
                        const uint32_t bar = vote ? smem_addr(&ct->vote) : smem_addr(&ct->pv_done), parity = (vote ? tile : tile - 1) & 1;
                        if (!__all_sync(0xffffffffu, bar_test(bar, parity)) && __any_sync(0xffffffffu, !bar_wait(bar, parity))) {
                            if (lane == 0) gave_up(ct);
                            dead = true;
                        }
                    }
                    const bool any = *static_cast<volatile int*>(&ct->over[tile & 3]) != 0;
                    // (The slot of the tile after the next: all have read it, and none is there yet.)
                    if (tid == 0) *static_cast<volatile int*>(&ct->over[(tile + 2) & 3]) = 0;
                    if (any) {
                        if (softmax_any<C::kSoft>(dead)) goto softmax_end;
                        float top0 = -INFINITY, top1 = -INFINITY;
                        if (on) {
#pragma unroll
                            for (int c = 0; c < kC; ++c) {
                                top0 = fmaxf(top0, fmaxf(x[4 * c], x[4 * c + 1]));
                                top1 = fmaxf(top1, fmaxf(x[4 * c + 2], x[4 * c + 3]));
                            }
                        }
#pragma unroll
                        for (int d = 1; d < 4; d <<= 1) {
                            top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, d));
                            top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, d));
                        }
                        if (C::kSplit > 1) across(ct->top, top0, top1);
                        const float n0 = fmaxf(m0, top0 * a.scale_log2), n1 = fmaxf(m1, top1 * a.scale_log2);
                        // (A row that has seen nothing yet has added nothing.)
                        float alpha0 = m0 == -INFINITY ? 0.f : ex2(m0 - n0), alpha1 = m1 == -INFINITY ? 0.f : ex2(m1 - n1);
                        l0 *= alpha0;
                        lr0 *= alpha0;
                        l1 *= alpha1;
                        lr1 *= alpha1;
                        if (FP8) {
                            // (The unit of what has been added moves with the base, unless the tile has more.)
                            const float by0 = m0 - n0, by1 = m1 - n1, was0 = m0 == -INFINITY ? -126.f : up0 + by0,
                                        was1 = m1 == -INFINITY ? -126.f : up1 + by1;
                            const bool none0 = m0 == -INFINITY, none1 = m1 == -INFINITY;
                            m0 = n0;
                            m1 = n1;
                            if (on) weights(1.f, 1.f);
                            else big0 = big1 = 0.f;
#pragma unroll
                            for (int d = 1; d < 4; d <<= 1) {
                                big0 = fmaxf(big0, __shfl_xor_sync(0xffffffffu, big0, d));
                                big1 = fmaxf(big1, __shfl_xor_sync(0xffffffffu, big1, d));
                            }
                            if (C::kSplit > 1) across(ct->big, big0, big1);
                            auto unit = [](float big, float before) {
                                const float e = static_cast<float>(static_cast<int>(__float_as_uint(big) >> 23) - 127);
                                return fminf(fmaxf(fmaxf(e, before), -126.f), 126.f);
                            };
                            const float to0 = unit(big0, was0), to1 = unit(big1, was1);
                            alpha0 = none0 ? 0.f : ex2(by0 + (up0 - to0));
                            alpha1 = none1 ? 0.f : ex2(by1 + (up1 - to1));
                            up0 = to0;
                            up1 = to1;
                        } else {
                            m0 = n0;
                            m1 = n1;
                        }
                        if (j > 0) {
                            publish(ct->alpha, alpha0, alpha1);
                            tc_fence_after();
                            softmax_sync<C::kSoft>();
#pragma unroll 1
                            for (int c = first_col; c < first_col + kOCols; c += 16) {
                                uint32_t y[16];
                                tc_ld16(tmem + lanes + c, y);
                                tc_wait_ld();
#pragma unroll
                                for (int u = 0; u < 16; ++u) y[u] = __float_as_uint(__uint_as_float(y[u]) * ct->alpha[(c + u) % N]);
                                tc_st16(tmem + lanes + c, y);
                            }
                            tc_wait_st();
                        }
                        if (on) weights(FP8 ? ex2(-up0) : 1.f, FP8 ? ex2(-up1) : 1.f);
                    }
                    if (j > 0 && (j & (kFoldTiles - 1)) == 0) {
                        // O moves to the fp32 sums: thread's channel 128 u + chan, row after row.
                        tc_fence_after();
                        const float o0 = FP8 ? m0 + up0 : m0, o1 = FP8 ? m1 + up1 : m1;
                        publish(ct->factor, folded0 == -INFINITY ? 0.f : ex2(folded0 - o0), folded1 == -INFINITY ? 0.f : ex2(folded1 - o1));
                        folded0 = o0;
                        folded1 = o1;
                        softmax_sync<C::kSoft>();
#pragma unroll 1
                        for (int c = first_col; c < first_col + kOCols; c += 16) {
                            uint32_t y[16];
                            tc_ld16(tmem + lanes + c, y);
                            tc_wait_ld();
#pragma unroll
                            for (int u = 0; u < 16; ++u) {
                                const int r = (c + u) % N;
                                if (r < rows) {
                                    float* const at = fold_to + r * kLatentDim + (c + u) / N * 128 + chan;
                                    *at = j > kFoldTiles ? fmaf(*at, ct->factor[r], __uint_as_float(y[u])) : __uint_as_float(y[u]);
                                }
                            }
                        }
                        softmax_sync<C::kSoft>();   // (the factors are written again)
                    }
                    // P, a row of 64 tokens each: blocks of 8 rows x 8 tokens.
                    if (on) {
#pragma unroll
                        for (int c = 0; c < kC; c += 2) {
                            const int r = 16 * rg + (lane & 15), chunk = tok0 / 8 + c + (lane >> 4);
                            stmatrix_x4(smem_addr(ps) + r * 128 + ((chunk ^ (r & 7)) << 4), p[c][0], p[c][1], p[c + 1][0], p[c + 1][1]);
                        }
                    }
                    // Tokens that no row sees may hold anything: their channels become zeros (P = 0 must not meet a
                    // NaN) in the pages that the product reads.
                    const int pages = min(kPages, s.en.npages - (s.t0 + j) * kPages);
                    if (fault || first + pages * kPage > see_any) {
                        for (int i = tid; i < pages * kPage * kUnits * 16; i += 32 * C::kSoft) {
                            const int r = i >> 6, u = (i >> 4) & 3, c = i & 15;
                            if (first + r >= see_any || ((fault >> (r / kPage * 8)) & 1u))
                                *reinterpret_cast<uint4*>(ring + (tile * kUnits + u) % C::kRing * kUnit + (r >> 3) * 2048 + (c >> 3) * 1024 +
                                                          (r & 7) * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ct->p_full));
                    if (on) {
                        l0 += add0;
                        l1 += add1;
                        lr0 += add_r0;
                        lr1 += add_r1;
                    }
                }
                if (nx.t1 > nx.t0) load_q(nx.en.row0, nx.en.nrows);   // the segment's last use of Q is over

                // ---------------- the segment's end
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
                    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
                    lr0 += __shfl_xor_sync(0xffffffffu, lr0, d);
                    lr1 += __shfl_xor_sync(0xffffffffu, lr1, d);
                }
                if (FP8) {
                    lr0 = l0;
                    lr1 = l1;
                }
                const bool whole = s.slot < 0;
                LATENT_WAIT(ct->pv_done, (tile - 1) & 1);   // (all warps have read the factors and maxima of their last tile, too)
                tc_fence_after();
                if (C::kSplit > 1) {
                    if (quad == 0) {
                        ct->sum[16 * w + (lane >> 2)] = make_float2(l0, lr0);
                        ct->sum[16 * w + 8 + (lane >> 2)] = make_float2(l1, lr1);
                    }
                    softmax_sync<C::kSoft>();
                    l0 = l1 = lr0 = lr1 = 0.f;
#pragma unroll
                    for (int i = 0; i < C::kSplit; ++i) {
                        const float2 a0 = ct->sum[i * N + r0], a1 = ct->sum[i * N + r1];
                        l0 += a0.x;
                        lr0 += a0.y;
                        l1 += a1.x;
                        lr1 += a1.y;
                    }
                }
                // A row that sees nothing is 0, whatever the others see.
                if (on) {
                    const float g0 = FP8 ? ex2(up0) : 1.f, g1 = FP8 ? ex2(up1) : 1.f;
                    publish(ct->factor, whole ? (lr0 > 0.f ? 1.f / lr0 * g0 : lr0) : g0, whole ? (lr1 > 0.f ? 1.f / lr1 * g1 : lr1) : g1);
                    publish(ct->alpha, folded0 == -INFINITY ? 0.f : ex2(folded0 - (FP8 ? m0 + up0 : m0)),
                            folded1 == -INFINITY ? 0.f : ex2(folded1 - (FP8 ? m1 + up1 : m1)));
                    if (quad == 0 && tp == 0) {
                        auto result = [&](int r, float m, float l, float lr) {
                            if (r >= rows) return;
                            if (whole) a.lse[s.en.row0 + r] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
                            else a.cut_ml[static_cast<int64_t>(s.slot) * N + r] = make_float4(m, l, lr, 0.f);
                        };
                        result(r0, m0, l0, lr0);
                        result(r1, m1, l1, lr1);
                    }
                }
                softmax_sync<C::kSoft>();
                float odd = 0.f;   // NaN once a channel of a row that sees something is not finite
                const bool fold = n > kFoldTiles;
#pragma unroll 1
                for (int c = first_col; c < first_col + kOCols; c += 16) {   // channel 128 (c / N) + chan of 16 rows
                    uint32_t y[16];
                    tc_ld16(tmem + lanes + c, y);
                    const int first_row = c % N, channel = c / N * 128 + chan, left = rows - first_row;
                    float f[16];
#pragma unroll
                    for (int u = 0; u < 16; u += 4) *reinterpret_cast<float4*>(&f[u]) = *reinterpret_cast<const float4*>(&ct->factor[first_row + u]);
                    tc_wait_ld();
                    if (fold) {
                        const float* const from = fold_to + first_row * kLatentDim + channel;
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            if (u < left) y[u] = __float_as_uint(fmaf(from[u * kLatentDim], ct->alpha[first_row + u], __uint_as_float(y[u])));
                    }
                    // (The rows mostly are all there: without the tests a partial's 16 take 340 cycles instead of 1070.)
                    auto write = [&](auto all) {
                        if (!whole) {
                            float* const to = a.cut_o + (static_cast<int64_t>(s.slot) * N + first_row) * kLatentDim + channel;
#pragma unroll
                            for (int u = 0; u < 16; ++u)
                                if (all || u < left) to[u * kLatentDim] = FP8 ? __uint_as_float(y[u]) * f[u] : __uint_as_float(y[u]);
                            return;
                        }
                        // Pairs of lanes change values, so that each has two channels of one of two rows.
                        const bool high = tid & 1;
                        __nv_bfloat16* const to = a.out + static_cast<int64_t>(s.en.row0 + first_row + high) * kLatentDim + (channel & ~1);
#pragma unroll
                        for (int u = 0; u < 16; u += 2) {
                            const float v0 = f[u] == 0.f || !(all || u < left) ? 0.f : __uint_as_float(y[u]) * f[u];
                            const float v1 = f[u + 1] == 0.f || !(all || u + 1 < left) ? 0.f : __uint_as_float(y[u + 1]) * f[u + 1];
                            odd = fmaf(v0, 0.f, fmaf(v1, 0.f, odd));
                            const float other = __shfl_xor_sync(0xffffffffu, high ? v0 : v1, 1);
                            if (all || u + high < left)
                                *reinterpret_cast<uint32_t*>(to + u * kLatentDim) = high ? pack_bf16x2(other, v1) : pack_bf16x2(v0, other);
                        }
                    };
                    if (left >= 16) write(std::true_type{});
                    else write(std::false_type{});
                }
                // (Rows of one token see the same.)
                if (whole && softmax_any<C::kSoft>(odd != 0.f) && tid == 0 && see_all != see_any)
                    a.odd[atomicAdd(a.num_odd, 1)] = static_cast<uint32_t>(~s.slot) * a.share + part;
                tc_fence_before();
                softmax_sync<C::kSoft>();   // all have read O before the next segment's first product writes it
                seg_done(k);
            }
        softmax_end:;
        } else if (C::kLoads == 2 ? warp == 0 || warp == 3 : warp >= 8 && warp < 12) {
            // ---------------- loads: warp 8 + p page p of every tile, in step; e4m3: of 64 rows: warps 0 and 3, two pages each
            reg_dec<C::kLoads == 2 ? C::kMmaRegs : C::kLoadRegs>();
            const uint32_t go = elected();
            constexpr int kMine = kPages / C::kLoads;
            const int p0 = C::kLoads == 2 ? (warp == 0 ? 0 : 2) : warp - 8;
            uint32_t tile = 0, loaded = 0;
            constexpr uint32_t kDepth = FP8 ? (C::kCodes ? C::kCodes : 1) : C::kRing;
            constexpr uint32_t kPageBytes = kPage * (FP8 ? 128 : 256);   // of a unit
            uint64_t* const empty = FP8 ? ct->code_empty : ct->empty;
            const uint32_t to = smem_addr(FP8 ? codes : ring) + p0 * kPageBytes;
            const uint32_t rope_to = smem_addr(ropes) + p0 * (kPage * kRopeDim * 2);
            for (uint32_t k = 0;; ++k) {
                TEST_WAIT(ct->seg_full[k % kSegs], (k / kSegs) & 1, loads_end);
                const Seg& s = ct->seg[k % kSegs];
                const int t0 = uniform(s.t0), n = uniform(s.t1) - t0;
                if (n == 0) break;
                const int end = min(s.en.npages, s.t1 * kPages);
                const int32_t* const pages = a.page_table + static_cast<int64_t>(s.en.req) * a.max_pages;
                // Lane l resolves the pages of tile i + l, well before the loads that need them: -2 behind the last page, -1
                // what the table does not give.
                auto fetch = [&](int i0, int p) {
                    const int i = (t0 + i0 + lane) * kPages + p0 + p;
                    if (i0 + lane >= n || i >= end) return -2;
                    const int ph = pages[i];
                    return ph < 0 || ph >= a.num_pages ? -1 : ph;
                };
                int cur[kMine], nxt[kMine];
#pragma unroll
                for (int p = 0; p < kMine; ++p) nxt[p] = fetch(0, p);
                for (int i = 0; i < n; ++i, ++tile) {
                    if (i % 32 == 0) {
#pragma unroll
                        for (int p = 0; p < kMine; ++p) {
                            cur[p] = nxt[p];
                            if (i + 32 < n) nxt[p] = fetch(i + 32, p);
                        }
                    }
                    const uint32_t slot = tile % kInfoSlots;
                    int ph[kMine];
#pragma unroll
                    for (int p = 0; p < kMine; ++p) {
                        ph[p] = uniform(__shfl_sync(0xffffffffu, cur[p], i % 32));
                        if (go) {
                            if (ph[p] == -1) svq_flag(SV_DEVERR_PAGE_TABLE);
                            ct->fault[slot][p0 + p] = ph[p] == -1;
                        }
                        if (FP8) {
                            const uint32_t bar = smem_addr(&ct->scale_full[slot]);
                            if (go) {
                                if (ph[p] >= 0) {
                                    mbar_arrive_expect_tx(bar, kPage * 4);
                                    bulk_copy_g2s(smem_addr(scales + slot * kTok + (p0 + p) * kPage), a.scale + static_cast<int64_t>(ph[p]) * kPage, kPage * 4, bar);
                                } else {
                                    mbar_arrive(bar);
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) {
                        const uint32_t at = tile * kUnits + u, st = at % kDepth;
                        TEST_WAIT(empty[st], ((at / kDepth) & 1) ^ 1, loads_end);
                        const uint32_t bar = smem_addr(FP8 ? &ct->code_full[st] : &ct->full[st]);
#pragma unroll
                        for (int p = 0; p < kMine; ++p) {
                            const uint32_t on = ph[p] >= 0 ? go : 0u, dst = to + st * (kPageBytes * kPages) + p * kPageBytes;
                            if (go) {
                                if (ph[p] >= 0) mbar_arrive_expect_tx(bar, kPageBytes);
                                else mbar_arrive(bar);
                            }
                            __syncwarp();
                            if (FP8) tma_2d_if(on, dst, &tmap_c, u * 128, ph[p] * kPage, bar);
                            else tma_page_if(on, dst, &tmap_c, 2 * u, 2 * ph[p], bar);
                        }
                        loaded = at + 1;
                    }
                    const uint32_t st = tile % C::kRope;
                    TEST_WAIT(ct->rope_empty[st], ((tile / C::kRope) & 1) ^ 1, loads_end);
                    const uint32_t bar = smem_addr(&ct->rope_full[st]);
#pragma unroll
                    for (int p = 0; p < kMine; ++p) {
                        if (go) {
                            if (ph[p] >= 0) mbar_arrive_expect_tx(bar, kPage * kRopeDim * 2);
                            else mbar_arrive(bar);
                        }
                        __syncwarp();
                        tma_2d_if(ph[p] >= 0 ? go : 0u, rope_to + st * kRopeBytes + p * (kPage * kRopeDim * 2), &tmap_r, 0, ph[p] * kPage, bar);
                    }
                }
                seg_done(k);
            }
            goto loads_done;   // every load has been waited for by the MMAs or the widening warps
        loads_end:
            // Gave up: the copies still in flight land before the CTA (and its shared memory) retires.
            for (uint32_t x = loaded > kDepth ? loaded - kDepth : 0; x < loaded; ++x)
                (void)bar_wait(smem_addr(FP8 ? &ct->code_full[x % kDepth] : &ct->full[x % kDepth]), (x / kDepth) & 1);
            for (uint32_t x = tile > C::kRope ? tile - C::kRope : 0; x < tile; ++x)
                (void)bar_wait(smem_addr(&ct->rope_full[x % C::kRope]), (x / C::kRope) & 1);
            if (FP8) (void)bar_wait(smem_addr(&ct->scale_full[tile % kInfoSlots]), (tile / kInfoSlots) & 1);
        loads_done:;
        } else if (FP8 && warp >= C::kFirstWiden) {
            // ---------------- e4m3 codes -> fp16 units in the MMAs' layout, four warps a unit
            reg_dec<C::kWidenRegs>();
            const int tid = threadIdx.x & 127;
            uint32_t at = 0, until = 0;
            constexpr uint32_t kDepth = FP8 ? C::kCodes : 1;
            for (uint32_t k = 0;; ++k) {
                TEST_WAIT(ct->seg_full[k % kSegs], (k / kSegs) & 1, widen_end);
                const Seg& s = ct->seg[k % kSegs];
                const int n = s.t1 - s.t0;
                if (n == 0) break;
                until += n * kUnits;
                for (; at < until; ++at) {
                    const uint32_t cs = at % kDepth, st = at % C::kRing;
                    TEST_WAIT(ct->code_full[cs], (at / kDepth) & 1, widen_end);
                    // 16 codes at chunk tid / 8 % 8 of every eighth row: eight lanes read, and write, eight rows' bytes in
                    // different banks.  The fence keeps the next copy into the slot behind these reads.
                    const int r = tid & 7, c = (tid >> 3) & 7, u0 = (tid >> 6) * 4;
                    uint4 v[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        v[u] = *reinterpret_cast<const uint4*>(codes + cs * (kUnit / 2) + (r + 8 * (u0 + u)) * 128 + ((c ^ r) << 4));
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ct->code_empty[cs]));
                    TEST_WAIT(ct->empty[st], ((at / C::kRing) & 1) ^ 1, widen_end);
                    unsigned char* const o = ring + st * kUnit + u0 * 2048 + (c >> 2) * 1024 + r * 128;
                    const int at0 = ((2 * c) & 7 ^ r) << 4, at1 = ((2 * c + 1) & 7 ^ r) << 4;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint4 lo, hi;
                        widen4_f16(v[u].x, lo.x, lo.y);
                        widen4_f16(v[u].y, lo.z, lo.w);
                        widen4_f16(v[u].z, hi.x, hi.y);
                        widen4_f16(v[u].w, hi.z, hi.w);
                        *reinterpret_cast<uint4*>(o + u * 2048 + at0) = lo;
                        *reinterpret_cast<uint4*>(o + u * 2048 + at1) = hi;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&ct->full[st]));
                }
                seg_done(k);
            }
        widen_end:;
        } else {
            reg_dec<C::kMmaRegs>();   // (warps 0 and 3)
        }
    }
    __threadfence();
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024, kFewPlanThreads = 256;   // (few where a thread each is enough: 0.7 us less)

// One CTA: the list of entries, and the running sum of their costs.
__global__ void __launch_bounds__(kPlanThreads) latent_plan_kernel(const __grid_constant__ LatentArgs a) {
    __shared__ int64_t warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
    int64_t total;
    pdl_wait();   // the workspace may still be read by the call before
    pdl_launch_dependents();
    const int rows_per = a.share * a.tile_rows;
    auto range = [&](int b, int& q0, int& q1) {
        q0 = a.q_start ? a.q_start[b] : b;
        q1 = a.q_start ? a.q_start[b + 1] : b + 1;
        return q0 >= 0 && q1 >= q0 && q1 <= a.total_q;
    };
    int n = 0;
    for (int i0 = 0; i0 < a.batch; i0 += threads) {
        const int i = i0 + tid;
        int count = 0;
        if (i < a.batch) {
            int q0, q1;
            if (!range(i, q0, q1)) svq_flag(SV_DEVERR_Q_START);
            else count = static_cast<int>((static_cast<int64_t>(q1 - q0) * a.heads + rows_per - 1) / rows_per);
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
    __syncthreads();
    int64_t base = 0;
    for (int e0 = 0; e0 < n; e0 += threads) {
        const int e = e0 + tid;
        Entry en = {0, 0, 0, 0, 0, 0, {0, 0}};
        bool empty = false;   // rows that see nothing
        if (e < n) {
            const int b = find_le(a.req_first, a.batch, e);
            int q0, q1;
            (void)range(b, q0, q1);
            int len = a.seq_lens[b];
            if (len < 0 || (static_cast<int64_t>(len) + kPage - 1) / kPage > a.max_pages) {
                svq_flag(SV_DEVERR_SEQ_LEN);
                len = 0;
            } else if (len > 0 && q1 - q0 > len) {
                svq_flag(SV_DEVERR_Q_START);
                len = 0;
            }
            const int64_t row0 = static_cast<int64_t>(q0) * a.heads + static_cast<int64_t>(e - a.req_first[b]) * rows_per;
            en.row0 = static_cast<int>(row0);
            en.nrows = static_cast<int>(min(static_cast<int64_t>(rows_per), static_cast<int64_t>(q1) * a.heads - row0));
            en.posbase = len - q1;
            en.req = b;
            if (len > 0) en.npages = (en.posbase + (en.row0 + en.nrows - 1) / a.heads) / kPage + 1;
            empty = len == 0;
        }
        en.tiles = (en.npages + kPages - 1) / kPages;
        const int64_t before = base + block_scan(cost_of_entry(en.tiles, a.tile_rows), warp_sums, total);
        base += total;
        if (e < n) {
            a.entries[e] = en;
            a.cum[e] = before;
        }
        for (uint32_t rest = __ballot_sync(0xffffffffu, empty); rest; rest &= rest - 1) {
            const int src = __ffs(rest) - 1;
            const int64_t r0 = __shfl_sync(0xffffffffu, en.row0, src);
            const int64_t r1 = r0 + __shfl_sync(0xffffffffu, en.nrows, src);
            uint4* o = reinterpret_cast<uint4*>(a.out + r0 * kLatentDim);
            for (int64_t i = lane; i < (r1 - r0) * (kLatentDim / 8); i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
            for (int64_t i = r0 + lane; i < r1; i += 32) a.lse[i] = -INFINITY;
        }
    }
    if (tid == 0) {
        a.cum[n] = base;
        *a.total = base;
        *a.num_entries = n;
        *a.num_odd = 0;
    }
}

// ---------------------------------------------------------------- joining partials
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = bf16lo(w[e]);
        f[2 * e + 1] = bf16hi(w[e]);
    }
}

// A row whose outputs may not be finite, by one warp (lane l: channels 16 l .. and
// rotary channels 2 l, 2 l + 1).  The tile's product multiplies every latent of
// the tile with a weight, and a weight 0 does not hide an infinite or NaN latent
// from the rows that do not see its token.  So if the row's logits are finite, its
// outputs are not, and a token that other rows of the entry see and this one does
// not holds such a value, the row is computed again from its own tokens alone.
__device__ __noinline__ void look_at_row(const LatentArgs& a, int entry, int row) {
    const int lane = threadIdx.x & 31;
    const Entry en = a.entries[entry];
    const int end = en.posbase + row / a.heads + 1;
    const int last = en.posbase + (en.row0 + en.nrows - 1) / a.heads + 1;
    float got[16];
    uint4* const to = reinterpret_cast<uint4*>(a.out + static_cast<int64_t>(row) * kLatentDim + 16 * lane);
    unpack8(to[0], got);
    unpack8(to[1], got + 8);
    {
        float odd = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) odd = fmaf(got[e], 0.f, odd);
        if (!(fabsf(a.lse[row]) < INFINITY) || !__any_sync(0xffffffffu, odd != 0.f)) return;
    }
    const int32_t* const pages = a.page_table + static_cast<int64_t>(en.req) * a.max_pages;
    auto place_of = [&](int t) {
        const int64_t ph = pages[t / kPage];
        return ph < 0 || ph >= a.num_pages ? -1ll : ph * kPage + t % kPage;
    };
    auto latent = [&](int64_t s, float (&c)[16]) {
        if (a.fp8) {
            const uint4 v = *reinterpret_cast<const uint4*>(a.pool + s * kLatentDim + 16 * lane);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const float sc = a.scale[s];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t lo, hi;
                widen4(w[e], lo, hi);
                keep_nan(w[e], lo, hi);
                c[4 * e] = bf16lo(lo) * sc;
                c[4 * e + 1] = bf16hi(lo) * sc;
                c[4 * e + 2] = bf16lo(hi) * sc;
                c[4 * e + 3] = bf16hi(hi) * sc;
            }
        } else {
            const uint4* const from = reinterpret_cast<const uint4*>(a.pool + s * (2 * kLatentDim) + 32 * lane);
            unpack8(from[0], c);
            unpack8(from[1], c + 8);
        }
    };
    float c[16];
    if (const int64_t s = place_of(end - 1); s >= 0) {
        // The row's own token is NaN wherever the row is not finite (a whole cache of NaN): so is the result.
        latent(s, c);
        bool known = true;
#pragma unroll
        for (int e = 0; e < 16; ++e) known &= c[e] != c[e] || got[e] * 0.f == 0.f;
        if (__all_sync(0xffffffffu, known)) return;
    }
    float odd = 0.f;   // of the tokens that other rows see and this one does not
    for (int t = end; t < last; ++t) {
        const int64_t s = place_of(t);
        if (s < 0) continue;
        latent(s, c);
#pragma unroll
        for (int e = 0; e < 16; ++e) odd = fmaf(c[e], 0.f, odd);
    }
    if (!__any_sync(0xffffffffu, odd != 0.f)) return;   // the row's own tokens gave it
    float q[16], o[16], m = -INFINITY, l = 0.f;
    const __nv_bfloat16* const qr = a.q + static_cast<int64_t>(row) * kQueryDim;
    unpack8(*reinterpret_cast<const uint4*>(qr + 16 * lane), q);
    unpack8(*reinterpret_cast<const uint4*>(qr + 16 * lane + 8), q + 8);
    const uint32_t qw = *reinterpret_cast<const uint32_t*>(qr + kLatentDim + 2 * lane);
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = 0.f;
    for (int t = 0; t < end; ++t) {
        const int64_t s = place_of(t);
        if (s < 0) continue;
        latent(s, c);
        const uint32_t rw = *reinterpret_cast<const uint32_t*>(a.rope + s * kRopeDim + 2 * lane);
        float z = bf16lo(qw) * bf16lo(rw) + bf16hi(qw) * bf16hi(rw);
#pragma unroll
        for (int e = 0; e < 16; ++e) z = fmaf(q[e], c[e], z);
#pragma unroll
        for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
        z *= a.scale_log2;
        const float mn = fmaxf(m, z), base = mn == -INFINITY ? 0.f : mn;
        const float f = ex2(m - base), p = ex2(z - base);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = fmaf(p, c[e], o[e] * f);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = l != 0.f ? pack_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
}

// CTA (c, y) joins the entry that group c + 1 goes on with, a row at a time (rows
// y, y + gridDim.y, ...): thread i channels 4 i .. 4 i + 3.  Then the row tiles of
// whole entries with values that are not finite.
constexpr int kJoinThreads = 128;

__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const __grid_constant__ LatentArgs a) {
    const int tid = threadIdx.x, warp = tid >> 5;
    pdl_wait();
    const int N = a.tile_rows;
    const int groups = groups_of(*a.total, gridDim.x + 1);
    const int c = blockIdx.x + 1;
    const int4 what = c < groups ? a.cut_item[2 * c] : make_int4(0, 0, 0, 0);
    const int num_odd = a.planned ? *a.num_odd : 0;   // (rows of one token see the same)
    const int pieces = what.z;
    const int4 where = pieces ? a.cut_item[2 * c + 1] : what;
    for (int r = blockIdx.y; pieces && r < what.y; r += gridDim.y) {
        const int part = r / N, tr = r - part * N;
        // Slots count CTAs: group g's part p is CTA g * share + p.
        auto row_of = [&](int k) {
            const int slot = k == 0 ? where.x : where.y + 2 * (k - 1);
            return (static_cast<int64_t>(2 * ((slot >> 1) * a.share + part) + (slot & 1))) * N + tr;
        };
        float m = -INFINITY, l = 0.f, lr = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAhead = 8;   // pieces on their way at a time
        for (int k0 = 0; k0 < pieces; k0 += kAhead) {
            float4 ml[kAhead], x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const bool on = k0 + u < pieces;
                ml[u] = on ? a.cut_ml[row_of(k0 + u)] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
                x[u] = on ? *reinterpret_cast<const float4*>(a.cut_o + row_of(k0 + u) * kLatentDim + 4 * tid) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mn = m;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) mn = fmaxf(mn, ml[u].x);
            const float base = mn == -INFINITY ? 0.f : mn;   // pieces without a visible token: weights 0
            const float e = ex2(m - base);
            m = mn;
            l *= e;
            lr *= e;
            o.x *= e, o.y *= e, o.z *= e, o.w *= e;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const float f = ex2(ml[u].x - base);
                l = fmaf(ml[u].y, f, l);
                lr = fmaf(ml[u].z, f, lr);
                o.x = fmaf(x[u].x, f, o.x);
                o.y = fmaf(x[u].y, f, o.y);
                o.z = fmaf(x[u].z, f, o.z);
                o.w = fmaf(x[u].w, f, o.w);
            }
        }
        const float inv = lr > 0.f ? 1.f / lr : lr;
        uint2 v = make_uint2(0u, 0u);
        if (lr != 0.f) {
            v.x = pack_bf16x2(o.x * inv, o.y * inv);
            v.y = pack_bf16x2(o.z * inv, o.w * inv);
        }
        const int row = what.x + r;
        *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(row) * kLatentDim + 4 * tid) = v;
        if (tid == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : (l == 0.f ? -INFINITY : l);
        const float odd = fmaf(o.x, 0.f, fmaf(o.y, 0.f, fmaf(o.z, 0.f, o.w * 0.f)));
        if (a.planned && __syncthreads_or(odd != 0.f && l > 0.f && l < INFINITY) && warp == 0) look_at_row(a, what.w, row);
    }
    for (int64_t i = blockIdx.y * gridDim.x + blockIdx.x; i < static_cast<int64_t>(num_odd) * (N / 4); i += gridDim.x * gridDim.y) {
        const uint32_t id = a.odd[i / (N / 4)];
        const int e = id / a.share, r = static_cast<int>(id % a.share) * N + static_cast<int>(i % (N / 4)) * 4 + warp;
        if (r < a.entries[e].nrows) look_at_row(a, e, a.entries[e].row0 + r);
    }
    __threadfence();
}

// ---------------------------------------------------------------- host side
size_t up(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
    size_t entries, cum, num, all, req_first, cut_item, cut_o, cut_ml, odd, num_odd, total;
    int tile_rows, share, max_entries;
    Layout(int64_t batch, int64_t total_q, int heads) {
        // Rows of a CTA: as many as a request has at the most if each has one query token, else 64; two CTAs side by
        // side take the rows of a token or a chunk that has more.
        const int64_t rows = total_q <= batch ? heads : static_cast<int64_t>(total_q) * heads;
        tile_rows = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
        share = rows <= 64 ? 1 : 2;
        const int64_t e = total_q * heads / (share * tile_rows) + batch;
        max_entries = static_cast<int>(e);
        size_t at = 0;
        auto take = [&](size_t bytes) { const size_t r = at; at += up(bytes); return r; };
        entries = take(e * sizeof(Entry));
        cum = take((e + 1) * sizeof(int64_t));
        num = take(sizeof(int));
        all = take(sizeof(int64_t));
        req_first = take(batch * sizeof(int));
        cut_item = take(2 * kMaxCtas * sizeof(int4));
        cut_o = take(2ull * kMaxCtas * tile_rows * kLatentDim * sizeof(float));
        cut_ml = take(2ull * kMaxCtas * tile_rows * sizeof(float4));
        odd = take(e * share * sizeof(uint32_t));
        num_odd = take(sizeof(int));
        total = at + 256;   // the parts begin at the workspace's first multiple of 256
    }
};

bool encode(CUtensorMap* map, CUtensorMapDataType type, const void* p, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encode_entry());
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    return enc && enc(map, type, rank, const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of 64 bf16 channels blocks, `rows` of them a box.
bool encode_rows(CUtensorMap* map, const void* p, int channels, int64_t n, int rows) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(channels), static_cast<cuuint64_t>(n)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(channels) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(rows)};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// A page's latents: bf16 in boxes of 128 channels that land as [8-row group][64-channel half][8 rows of 128 bytes], each
// 1 KB swizzled; codes in boxes of 128.
bool encode_latents(CUtensorMap* map, const void* p, int64_t pages, bool fp8) {
    if (fp8) {
        const cuuint64_t dims[2] = {kLatentDim, static_cast<cuuint64_t>(pages) * kPage};
        const cuuint64_t strides[1] = {kLatentDim};
        const cuuint32_t box[2] = {128, kPage};
        return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    const cuuint64_t dims[4] = {64, 8, kLatentDim / 64, static_cast<cuuint64_t>(pages) * 2};
    const cuuint64_t strides[3] = {2 * kLatentDim, 128, 16 * kLatentDim};
    const cuuint32_t box[4] = {64, 8, 2, 2};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int N, bool FP8>
int launch_tiles(const LatentArgs& a, const CUtensorMap& tc, const CUtensorMap& tr, int ctas, cudaStream_t stream) {
    static std::atomic<bool> attr_set[64];
    const int st = once_per_device(attr_set, [] {
        return cudaFuncSetAttribute(latent_kernel<N, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<N, FP8>::kSmem) ==
                       cudaSuccess
                   ? SV_OK
                   : SV_ERR_CUDA;
    });
    if (st) return st;
    return launch_pdl(latent_kernel<N, FP8>, dim3(ctas), dim3(Cfg<N, FP8>::kThreads), Cfg<N, FP8>::kSmem, stream, a, tc, tr) ==
                   cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

}  // namespace

size_t latent_workspace_bytes(int batch, int num_q_heads, int total_q) { return Layout(batch, total_q, num_q_heads).total; }

int launch_latent_attention(const sv_cache* c, const void* q, int num_q_heads, const int32_t* q_start, int total_q,
                            const int32_t* page_table, const int32_t* seq_lens, int batch, int max_pages,
                            float softmax_scale, void* out, float* lse, void* workspace, int sm_count,
                            cudaStream_t stream) {
    const Layout lay(batch, total_q, num_q_heads);
    unsigned char* const ws =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
    LatentArgs a = {};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.heads = num_q_heads;
    a.q_start = q_start;
    a.total_q = total_q;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.batch = batch;
    a.max_pages = max_pages;
    a.num_pages = c->num_phys_pages;
    a.pool = static_cast<const unsigned char*>(c->k_pool);
    a.rope = static_cast<const __nv_bfloat16*>(c->v_pool);
    a.scale = static_cast<const float*>(c->k_scale);
    a.fp8 = c->kv_format == SV_KV_LATENT_E4M3;
    a.scale_log2 = softmax_scale * 1.4426950408889634f;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.share = lay.share;
    a.tile_rows = lay.tile_rows;
    a.entries = reinterpret_cast<Entry*>(ws + lay.entries);
    a.cum = reinterpret_cast<int64_t*>(ws + lay.cum);
    a.num_entries = reinterpret_cast<int*>(ws + lay.num);
    a.total = reinterpret_cast<int64_t*>(ws + lay.all);
    a.planned = q_start || batch > kOwnPlan;
    a.req_first = reinterpret_cast<int*>(ws + lay.req_first);
    a.max_entries = lay.max_entries;
    a.cut_o = reinterpret_cast<float*>(ws + lay.cut_o);
    a.cut_ml = reinterpret_cast<float4*>(ws + lay.cut_ml);
    a.cut_item = reinterpret_cast<int4*>(ws + lay.cut_item);
    a.odd = reinterpret_cast<uint32_t*>(ws + lay.odd);
    a.num_odd = reinterpret_cast<int*>(ws + lay.num_odd);
    CUtensorMap tc, tr;
    if (!encode_latents(&tc, c->k_pool, c->num_phys_pages, a.fp8) ||
        !encode_rows(&tr, c->v_pool, kRopeDim, c->num_phys_pages * kPage, kPage))
        return SV_ERR_CUDA;
    const int plan_threads = lay.max_entries <= kFewPlanThreads ? kFewPlanThreads : kPlanThreads;
    if (a.planned && launch_pdl(latent_plan_kernel, dim3(1), dim3(plan_threads), 0, stream, a) != cudaSuccess) return SV_ERR_CUDA;
    // No more groups than the longest requests that the table can name could use.
    const int64_t cost = (max_pages + kPages - 1) / kPages + static_cast<int64_t>(entry_cost(lay.tile_rows));
    const int64_t most = (cost * (a.planned ? lay.max_entries : batch) + kMinShare - 1) / kMinShare;
    const int fit = (sm_count < kMaxCtas ? sm_count : kMaxCtas) / lay.share;
    const int groups = most < fit ? static_cast<int>(most) : fit;
    const int ctas = groups * lay.share;
    int st;
    if (a.fp8)
        st = lay.tile_rows == 16   ? launch_tiles<16, true>(a, tc, tr, ctas, stream)
             : lay.tile_rows == 32 ? launch_tiles<32, true>(a, tc, tr, ctas, stream)
                                   : launch_tiles<64, true>(a, tc, tr, ctas, stream);
    else
        st = lay.tile_rows == 16   ? launch_tiles<16, false>(a, tc, tr, ctas, stream)
             : lay.tile_rows == 32 ? launch_tiles<32, false>(a, tc, tr, ctas, stream)
                                   : launch_tiles<64, false>(a, tc, tr, ctas, stream);
    if (st || groups < 2) return st;
    // (CTAs for the rows of an entry: 16 329 us for 8 requests of 128 heads, 32 323, 64 324, 128 328.)
    const int rows = lay.share * lay.tile_rows;
    return launch_pdl(latent_join_kernel, dim3(groups - 1, rows < 32 ? rows : 32), dim3(kJoinThreads), 0, stream, a) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

}  // namespace svq
