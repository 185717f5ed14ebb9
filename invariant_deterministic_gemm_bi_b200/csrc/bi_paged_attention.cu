// bi_paged_attention.cu -- decode attention over the paged 8-bit cache
// (include/bi_paged_attention.h).
//
// Memory bound: a key and a value of one head are 2 D bytes for at most 16 query heads, so the
// kernel streams the cache once and everything else has to hide behind that.
//
// Work.  A sequence's positions are cut into steps of 256 at multiples of 256, and runs of steps
// into chunks whose length follows from the number of steps alone.  An item is one chunk of one
// key/value head; persistent CTAs take items round robin, those of most steps first so that short
// ones fill the gaps at the end.  Consumer warp w of a CTA owns positions
// 32 w .. 32 w + 31 of every step and keeps a softmax state of its own over the chunk; the eight
// states are added in warp order at the chunk's end, and the chunks in ascending order by a second
// kernel.  Every sum's order is thus fixed by the sequence's length and window.
//
// Roles (12 warps, one CTA per SM).  One producer warp streams half-steps of 128 positions into a
// ring of stages with TMA (boxes of 16 or 32 positions of one page and head).  Eight consumer warps
// do nothing but the matrix products and the softmax.  Three helper warps prepare the next items'
// queries, add the states of the chunks that are done and keep the table of items filled.  (With
// all jobs in every warp, a tile took 964 warp instructions, 149 us for 64 sequences of 4096
// positions, 32/8 heads; with four producer warps and cp.async 865, 108 us.)
//
// Matrix products.  The cache is the first operand of mma.m16n8k16 (16 positions, or 16 dimensions,
// a time) and the query heads are the 8 columns, so grouped queries fill the tile instead of
// padding it to 16 rows.  e4m3 codes become fp16 exactly; queries become fp16 exactly after a power
// of two per head has been taken out of them (bf16 has fewer significant bits; entries below 2^-28 of the
// head's largest are off by up to 2^-39 of it, which an fp32 sum loses anyway unless the keys are zero
// where the query is large).  The order of dimensions
// inside a 16-byte group is permuted alike on both sides, so codes go from ldmatrix to the
// conversion without shuffles; values are read transposed, two dimensions to a 16-bit element.
// tcgen05 would need the weights and queries split into several e4m3 parts, or the codes written
// back to shared memory as fp16.  For 64 sequences of 4096 positions the call takes 97 us (5.5 TB/s), 3 of
// them the merge; without loads 79, without products and softmax 89: the loads bound it.  Where sequences are short or ragged the products do: conversions and byte permutations
// issue every second cycle, an m16n8k16 every eighth, and they do not overlap.
//
// Weights.  With sv the value scale of a position's page, the state's maximum M is that of
// t_j = s_j log2 e + log2 sv, and the weight of a value's code is a_j = 2^(t_j - M + 15) <= 2^15,
// rounded to fp16 (2^-11 of itself, an eighth of what bf16 would cost; the output is rounded to bf16
// anyway).  The value scale so costs nothing per element and weights down to 2^-29 of the largest keep
// all of fp16's bits.  The softmax sum adds 2^(s_j log2 e - M) in fp32.  With scales from 2^-64 to 2^64
// a position may count in it although t_j is far below M: by 128 for the scales and 54 for the score
// (2^30 positions of 2^-54 are what an fp32 sum rounds away).  So a_j is held as 2^(t_j - M + 60), an
// fp32 number down to t_j = M - 186, before it is rounded, and a change of M is applied in two halves.
// The sum itself lies between 2^-64 and 2^94.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "bi_kv_common.cuh"
#include "bi_paged_attention.h"
#include "ptx_sm100.cuh"

namespace {

using bi_kv::kFull;

constexpr int kConsumers = 8;               // warps, as for the next two
constexpr int kHelpers = 3;
constexpr int kProducers = 1;
constexpr int kThreads = 32 * (kConsumers + kHelpers + kProducers);
constexpr int kTile = 32;                   // positions of a warp's tile
constexpr int kTiles = 4;                   // tiles of a stage
constexpr int kHalf = kTiles * kTile;       // positions of a stage: half a step
constexpr int kStep = kConsumers * kTile;   // positions of a CTA's step
constexpr int kMaxChunks = 128;             // chunks of a sequence
constexpr int kMaxGroup = 16;               // query heads of a key/value head
constexpr int kEntries = 256;               // entries of the scanned chunk counts
constexpr int kClasses = 4;                 // of chunks, by steps: 4 and more, 3, 2, 1
constexpr int kItemBlock = 32;              // items whose table entries one warp makes at once
constexpr int kItemRing = 4 * kItemBlock;   // entries of the items' table
// Sequences.  With more of them than entries an entry stands for several, up to 64, whose lengths are read
// one after the other to find a chunk's.  The reads hide behind the items: 256 sequences of 200 tokens,
// 8 heads of 128, take 33.2 us and 257 33.7; 2048 of 40 tokens, 2 heads of 64, 39 us, and 16384 339 us,
// 1.4 and 1.5 us for each item of a block.
constexpr int kMaxBatch = 16384;
constexpr int64_t kMaxLen = INT64_C(1) << 30;   // positions of a sequence
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A head's factor up to which products with every valid key scale stay in fp32's range.
constexpr float kPlainFactor = 0x1p62f;
constexpr float kWeightExp = 60.0f;         // weights are held times 2^60,
constexpr float kToHalf = 0x1p-45f;         // times 2^15 in fp16,
constexpr float kToSum = 0x1p-60f;          // and as they are, over their value scale, in the sum
constexpr float kOutput = 0x1p-15f;         // takes the 2^15 out of the outputs
constexpr uint64_t kWaitNs = UINT64_C(2000000000);   // limit of a wait, unless the program sets another
static_assert(kStep == 2 * kHalf, "a step is two stages");

// Steps per chunk of a sequence of `steps` steps.  Opening and closing a chunk costs about as much as
// one step, so chunks grow with the sequence; short sequences keep one-step chunks, which spread a
// single request over more CTAs, and no sequence has more than kMaxChunks.
__host__ __device__ __forceinline__ int chunk_steps(int steps)
{
    int s = steps <= 4 ? 1 : steps <= 16 ? 2 : 4;
    while (s * kMaxChunks < steps)
        s *= 2;
    return s;
}

struct AttnArgs {
    const __nv_bfloat16 *q;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    __nv_bfloat16 *out;
    float *lse;
    float *part;        // [b][hq][chunks][D] unnormalised outputs
    float2 *part_ml;    // [b][hq][chunks] (M, sum)
    int64_t ldq, ldo, ld_table, window;
    int num_pages, max_len, b, hq, heads, group, page_shift, chunks;
    float scale_m;      // scale * log2 e = scale_m * 2^scale_e
    int scale_e;
    uint32_t skip_load;   // test only: the stage, counted from 1, that producers leave out
    uint64_t wait_cycles;
};

// What of a sequence is attended: positions [lo, hi), in steps from `first`.  A sequence without any,
// or of a length out of range, has no chunks.
struct Span {
    int lo, hi, first, steps, per_chunk, chunks;
    bool bad;
};

__host__ __device__ __forceinline__ int class_of(int steps) { return steps >= 4 ? 0 : 4 - steps; }

__device__ __forceinline__ Span span_of(int len, const AttnArgs &a)
{
    Span s;
    s.bad = len < 0 || len > a.max_len;
    s.hi = s.bad ? 0 : len;
    s.lo = a.window > 0 && s.hi > a.window ? s.hi - static_cast<int>(a.window) : 0;
    s.first = s.lo / kStep;
    s.steps = (s.hi + kStep - 1) / kStep - s.first;
    s.per_chunk = chunk_steps(s.steps);
    s.chunks = (s.steps + s.per_chunk - 1) / s.per_chunk;
    return s;
}

// How many chunks of class c a span has: its whole chunks, and a shorter last one.
__device__ __forceinline__ int chunks_of_class(const Span &s, int c)
{
    const int whole = s.steps / s.per_chunk, rest = s.steps - whole * s.per_chunk;   // 0 of both without steps
    return (class_of(s.per_chunk) == c ? whole : 0) + (rest > 0 && class_of(rest) == c ? 1 : 0);
}

// ---------------------------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// one box of codes: positions [pos, pos + rows) of a page's head, all dimensions
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int pos, int head, int page, uint64_t policy)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;"
                 ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(pos), "r"(head), "r"(page),
                   "l"(policy) : "memory");
}
__device__ __forceinline__ void expect_bytes(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// two e4m3 codes as fp16, the low byte in the low half (exact; NaN stays NaN)
__device__ __forceinline__ uint32_t codes_f16(uint32_t two)
{
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(static_cast<uint16_t>(two)));
    return y;
}
// d += a b: 16 x 16 times 16 x 8, fp32 sums
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log2_approx(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// The square root of the factor that takes sums relative to the maximum `from` to the maximum `to`:
// 2^(from - to) may be below fp32's range where a sum times it is not.
__device__ __forceinline__ float half_factor(float from, float to) { return exp2_approx((from - to) * 0.5f); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// s, or NaN unless 2^-64 <= s <= 2^64
__device__ __forceinline__ float checked_scale(float s) { return s >= 0x1p-64f && s <= 0x1p64f ? s : NAN; }

// ---------------------------------------------------------------------------------------------
// shared memory
// ---------------------------------------------------------------------------------------------

enum : int { kFirst = 1, kLast = 2, kEnd = 4 };

// What a stage holds: positions key0 .. key0 + 127, of which [lo, hi) count.
struct Stage {
    int key0, lo, hi, flags;
};

// One chunk of one key/value head.
struct Item {
    int b, kvh;          // b < 0: no more items
    int lo, hi;          // the sequence's attended positions
    int key0, steps;     // the chunk's first position and length
    int chunk, chunks;
};
static_assert(sizeof(Item) == 32, "two 16-byte words");

// MG: the most query heads of a key/value head, 4, 8 or 16 (columns come in eights).
template <int D, int MG>
struct Shared {
    static constexpr int NT = MG > 8 ? 2 : 1;
    static constexpr int kCols = NT * 8;
    // 32 KB stages of D = 128 (16 KB of D = 64) beside the chunk states, 192 KB together.  A stage always
    // serves the same half of the steps: a consumer then waits for every use of its stages in turn,
    // which waiting by parity needs.
    static constexpr int kStages = D == 128 ? 4 : MG > 8 ? 8 : 10;
    // States of two chunks, so that one is added while the next is written (16 heads of 128: one).
    static constexpr int kStates = D * MG > 1024 ? 1 : 2;
    static_assert(kStages % 2 == 0, "two halves");
    static constexpr int kMatrix = kTile * D;               // bytes of a tile's keys (or values)
    uint8_t ring[kStages][kTiles][2][kMatrix];              // keys, values
    float state[kStates][kConsumers][MG][D];                // a chunk's outputs, not normalised
    uint4 q[2][NT][D / 32][32];                             // two items' queries, as the consumers' lanes hold them
    float4 scale[kStages][kHalf / 16];                      // of 16 positions: key scale, log2 and kToSum / of the value scale
    Item items[kItemRing];
    Stage stage[kStages];
    float2 ml[kStates][kConsumers][kCols];                  // a chunk's maxima and sums
    float qc[2][kCols];                                     // scale * log2 e * the power of two taken out,
    int qe[2][kCols];                                       // and the exponent e of it as scale_m * 2^e
    uint64_t full[kStages], empty[kStages];                 // a stage is filled, is consumed
    // An item's states are written; the helpers are done with the item two before: its states are read,
    // and the queries that take the place of its own are there.  Even and odd items apart, since
    // consumers and helpers may be one ahead.
    uint64_t states[2], helped[2];
    int32_t first_chunk[kClasses][kEntries];                // chunks of the class before each entry
    int32_t class_chunks[kClasses];
    int32_t len[kEntries];                                  // lengths, when an entry is one sequence
    int32_t warp_sum[kClasses][kThreads / 32];
    int dead;                                               // a wait gave up
};

// Byte of the 16-byte group `grp` of row `row` inside a tile: groups are spread over the banks so
// that eight rows of one group (a matrix of ldmatrix) touch all of them once.
template <int D>
__device__ __forceinline__ int tile_offset(int row, int grp)
{
    return row * D + ((D == 128 ? grp ^ (row & 7) : grp ^ ((row >> 1) & 3)) << 4);
}

// Float of dimension d (even) of column `head` inside a state: the columns 2t of a quad fall on
// different banks.
template <int D>
__device__ __forceinline__ int state_offset(int head, int d)
{
    return head * D + (d ^ (((head >> 1) & 3) << 3));
}

// Whether the phase completed, one answer for the whole warp.  After a wait that gave up no warp goes on
// as if it had not: it neither reads, writes, copies nor arrives, so every other warp that needs it
// gives up at once, and what is running keeps its order.
template <typename S>
__device__ __forceinline__ bool wait_for(S &sm, const AttnArgs &a, uint64_t *bar, uint32_t parity)
{
    if (__all_sync(kFull, bi::ptx::mbar_wait(bar, parity, a.wait_cycles, &sm.dead)))
        return true;
    *static_cast<volatile int *>(&sm.dead) = 1;
    return false;
}

// One arrival of this warp, which releases what all of it has written.
__device__ __forceinline__ void warp_arrive(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        bi::ptx::mbar_arrive(bar);
}

// Item number i of this CTA, one lane an item: chunk ordinal u of the classes in order, and a
// key/value head.
template <typename S>
__device__ __forceinline__ Item make_item(const AttnArgs &a, const S &sm, int i)
{
    Item it = {};
    const int64_t n = blockIdx.x + static_cast<int64_t>(i) * gridDim.x;
    it.b = -1;
    int most = 0;
#pragma unroll
    for (int c = 0; c < kClasses; ++c)
        most += sm.class_chunks[c];
    if (n >= static_cast<int64_t>(most) * a.heads)
        return it;
    int chunk = static_cast<int>(n) / a.heads;
    it.kvh = static_cast<int>(n) - chunk * a.heads;
    int cls = 0;
    while (chunk >= sm.class_chunks[cls])
        chunk -= sm.class_chunks[cls++];
    const int32_t *first_chunk = sm.first_chunk[cls];
    int e = 0;   // the last entry with first_chunk <= chunk
#pragma unroll
    for (int step = kEntries / 2; step > 0; step >>= 1)
        if (first_chunk[e + step] <= chunk)
            e += step;
    chunk -= first_chunk[e];
    int b = e;
    Span s;
    if (a.b <= kEntries) {
        s = span_of(sm.len[b], a);
    } else {   // an entry is several consecutive sequences
        b = e * ((a.b + kEntries - 1) / kEntries);
        s = span_of(a.lens[b], a);
        for (int n_here; chunk >= (n_here = chunks_of_class(s, cls)); s = span_of(a.lens[++b], a))
            chunk -= n_here;
    }
    // of a sequence's chunks of the class: the whole ones from the first on, or its last
    if (class_of(s.per_chunk) != cls)
        chunk = s.chunks - 1;
    it.b = b;
    it.lo = s.lo;
    it.hi = s.hi;
    it.key0 = (s.first + chunk * s.per_chunk) * kStep;
    it.steps = min(s.per_chunk, s.steps - chunk * s.per_chunk);
    it.chunk = chunk;
    it.chunks = s.chunks;
    return it;
}

// ---------------------------------------------------------------------------------------------
// the roles
// ---------------------------------------------------------------------------------------------

// The producer warp.  Lane 8 s + j stands for the j-th 16 positions of stage s of a block of four
// stages; it holds their page number, asked for one block ahead, and scales, asked for half a block
// ahead.
template <int D, int MG>
__device__ __forceinline__ void produce(Shared<D, MG> &sm, const AttnArgs &a, const CUtensorMap *k_map, const CUtensorMap *v_map)
{
    using S = Shared<D, MG>;
    constexpr int kBlock = 4;              // stages
    const int lane = threadIdx.x & 31, group = lane & 7, quarter = lane >> 3;
    const int box = a.page_shift == 4 ? 16 : kTile;   // positions of a TMA box
    const int page_mask = (1 << a.page_shift) - 1;
    // codes are read once a call: marked first to leave L2 they do not push one another out before they
    // arrive (64 x 4096, 32/8 heads: 92 us against 102 us without the mark)
    const uint64_t policy = bi::ptx::policy_evict_first();

    // this lane's box of a block: whether any of it is attended, and its page
    struct Pages {
        int key, id;
        bool in, ok;
    };
    auto pages_of = [&](const Item &it, int block) {
        Pages x;
        x.key = it.key0 + (block * kBlock + quarter) * kHalf + (group * 16 & ~(box - 1));
        x.in = it.b >= 0 && block * kBlock + quarter < 2 * it.steps && x.key < it.hi && x.key + box > it.lo;
        x.id = x.in ? a.table[it.b * a.ld_table + (x.key >> a.page_shift)] : -1;
        x.ok = false;
        return x;
    };
    struct Scales {
        float k, v;
    };
    auto scales_of = [&](const Item &it, Pages &x) {
        x.ok = x.in && x.id >= 0 && x.id < a.num_pages;
        const int64_t at = static_cast<int64_t>(x.id) * a.heads + it.kvh;
        Scales s = {x.in ? NAN : 1.0f, 1.0f};   // a page number out of range gives NaN
        if (x.ok)
            s = {a.k_scale[at], a.v_scale[at]};
        return s;
    };

    int slot = 0;
    uint32_t parity = 1;     // of a stage not used yet
    bool used_all = false;   // every stage has been used
    bool ok = true;          // no wait has given up
    uint32_t skip = a.skip_load;   // 1: the next stage is left out
    auto take_slot = [&]() { return ok = wait_for(sm, a, &sm.empty[slot], parity); };
    auto give_slot = [&]() {
        if (skip != 1)
            warp_arrive(&sm.full[slot]);   // releases the words stored for it
        skip -= skip != 0;
        if (++slot == S::kStages) {
            slot = 0;
            parity ^= 1;
            used_all = true;
        }
    };

    int item = 0, block = 0;
    Item it = sm.items[0];
    Pages px = pages_of(it, 0);
    Scales sc = scales_of(it, px);
    while (ok && it.b >= 0) {
        const int stages = min(kBlock, 2 * it.steps - block * kBlock);
        // the next block, of this item or of the next one
        int next_block = block + 1;
        Item next = it;
        if (next_block * kBlock >= 2 * it.steps) {
            next_block = 0;
            next = sm.items[++item % kItemRing];
        }
        Pages px_next = pages_of(next, next_block);
        Scales sc_next = {1.0f, 1.0f};
        for (int s = 0; s < stages && take_slot(); ++s) {
            const bool mine = quarter == s;
            const bool issue = mine && px.ok && (group * 16 & (box - 1)) == 0 && skip != 1;
            const uint32_t boxes = __popc(__ballot_sync(kFull, issue));
            if (lane == 0) {
                const int at = block * kBlock + s;
                sm.stage[slot] = {it.key0 + at * kHalf, it.lo, it.hi,
                                  (at < 2 ? kFirst : 0) | (at >= 2 * it.steps - 2 ? kLast : 0)};
                expect_bytes(&sm.full[slot], boxes * 2u * box * D);
            }
            __syncwarp();
            if (issue) {
                const uint32_t dst = smem_u32(&sm.ring[slot][group >> 1][0][0]) + (group & 1) * 16 * D;
                tma_box(dst, k_map, &sm.full[slot], px.key & page_mask, it.kvh, px.id, policy);
                tma_box(dst + S::kMatrix, v_map, &sm.full[slot], px.key & page_mask, it.kvh, px.id, policy);
            }
            if (mine) {
                // approximate to 2^-22: a page's weights are all off by one factor below 2^-21
                const float v = checked_scale(sc.v);
                sm.scale[slot][group] = make_float4(checked_scale(sc.k), log2_approx(v), kToSum * rcp_approx(v), 0.0f);
            }
            if (s == min(1, stages - 1))
                sc_next = scales_of(next, px_next);
            give_slot();
        }
        it = next;
        block = next_block;
        px = px_next;
        sc = sc_next;
    }
    for (int half = 0; ok && half < 2; ++half)   // both halves of the consumers are told
        if (take_slot()) {
            if (lane == 0)
                sm.stage[slot] = {0, 0, 0, kEnd};
            give_slot();
        }
    // No copy is in flight when the block ends, whoever has given up: consumers that go on have waited for
    // every stage themselves.  The last use of a stage before `slot` was in this round of the ring, of the
    // others in the round before.
    for (int i = 0; i < S::kStages; ++i)
        if (i < slot || used_all)
            bi::ptx::mbar_wait(&sm.full[i], i < slot ? parity ^ 1 : parity, a.wait_cycles, nullptr);
}

template <int D, int MG>
__device__ __forceinline__ void consume(Shared<D, MG> &sm, const AttnArgs &a, int warp)
{
    using S = Shared<D, MG>;
    constexpr int NT = S::NT;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tile = warp % kTiles;
    const int mrow = (lane & 7) + ((lane >> 3) & 1) * 8, mgrp = lane >> 4;   // ldmatrix: this lane's row
    uint32_t qf[NT][D / 16][2];       // queries as the second operand
    float qc[NT][2];                  // factors of heads 2t, 2t + 1
    float o[NT][D / 16][4];           // [dimension 16 j + 2 g, + 1][head 2t, 2t + 1]
    float m[NT][2], l[NT][2];
    bool plain = true;                // every head's factor is below kPlainFactor
    int slot = warp / kTiles;         // stages of this warp's half of the steps
    uint32_t parity = 0;
    int item = 0;
    while (true) {
        if (!wait_for(sm, a, &sm.full[slot], parity))
            break;
        const Stage st = sm.stage[slot];
        if (st.flags & kEnd)
            break;
        if (st.flags & kFirst) {
            if (!wait_for(sm, a, &sm.helped[item & 1], (item >> 1) & 1))
                break;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int kp = 0; kp < D / 32; ++kp) {
                    const uint4 x = sm.q[item & 1][n][kp][lane];
                    qf[n][2 * kp][0] = x.x;
                    qf[n][2 * kp][1] = x.y;
                    qf[n][2 * kp + 1][0] = x.z;
                    qf[n][2 * kp + 1][1] = x.w;
                }
                qc[n][0] = sm.qc[item & 1][n * 8 + 2 * t];
                qc[n][1] = sm.qc[item & 1][n * 8 + 2 * t + 1];
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        o[n][j][x] = 0.0f;
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
            }
            plain = true;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                plain = plain && fabsf(qc[n][0]) < kPlainFactor && fabsf(qc[n][1]) < kPlainFactor;
            plain = __all_sync(kFull, plain);
        }
        const int key0 = st.key0 + tile * kTile;
        if (key0 < st.hi && key0 + kTile > st.lo) {
            const uint32_t ks_base = smem_u32(&sm.ring[slot][tile][0][0]);
            const uint32_t vs_base = ks_base + S::kMatrix;
            const bool whole = key0 >= st.lo && key0 + kTile <= st.hi;
            if (!whole) {
                // rows outside the sequence may hold anything: a NaN value would pass through a zero weight
                const int key = key0 + lane;
                if (key < st.lo || key >= st.hi) {
#pragma unroll
                    for (int x = 0; x < D / 16; ++x)
                        *reinterpret_cast<uint4 *>(&sm.ring[slot][tile][1][lane * D + x * 16]) = make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the stage's next load comes after
                }
                __syncwarp();
            }
            // scores of 32 positions: rows g and g + 8 of two tiles of 16
            float s[NT][2][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        s[n][mt][x] = 0.0f;
#pragma unroll
            for (int jp = 0; jp < D / 32; ++jp)
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    uint32_t r[4];
                    ldmatrix4(r, ks_base + tile_offset<D>(mt * 16 + mrow, 2 * jp + mgrp));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t a0 = codes_f16(r[2 * x]), a2 = codes_f16(r[2 * x] >> 16);
                        const uint32_t a1 = codes_f16(r[2 * x + 1]), a3 = codes_f16(r[2 * x + 1] >> 16);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma(s[n][mt], a0, a1, a2, a3, qf[n][2 * jp + x][0], qf[n][2 * jp + x][1]);
                    }
                }
            // base-2 exponents t_j, and their maximum
            const float4 sc[2] = {sm.scale[slot][2 * tile], sm.scale[slot][2 * tile + 1]};
            const float sk[2] = {sc[0].x, sc[1].x}, lsv[2] = {sc[0].y, sc[1].y}, rsv[2] = {sc[0].z, sc[1].z};
            uint32_t pf[NT][2][2];    // weights as the second operand: [tile of 16][keys 0-7, 8-15]
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float mx[2] = {m[n][0], m[n][1]};
                if (plain) {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt) {
                        const float c[2] = {qc[n][0] * sk[mt], qc[n][1] * sk[mt]};
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            s[n][mt][x] = fmaf(s[n][mt][x], c[x & 1], lsv[mt]);
                    }
                } else {   // rare: the factor may be beyond fp32 where a score is not, so its power of two comes in two halves
                    const int *e = &sm.qe[item & 1][n * 8 + 2 * t];
                    const float p[2][2] = {{pow2(max(e[0] >> 1, -126)), pow2(max(e[0] - (e[0] >> 1), -126))},
                                           {pow2(max(e[1] >> 1, -126)), pow2(max(e[1] - (e[1] >> 1), -126))}};
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            s[n][mt][x] = s[n][mt][x] * (a.scale_m * sk[mt]) * p[x & 1][0] * p[x & 1][1] + lsv[mt];
                }
                if (!whole) {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int key = key0 + mt * 16 + g + (x >> 1) * 8;
                            if (key < st.lo || key >= st.hi)
                                s[n][mt][x] = -INFINITY;
                        }
                }
#pragma unroll
                for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mx[x & 1] = fmaxf(mx[x & 1], s[n][mt][x]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 4));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 8));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 16));
                }
                const float half[2] = {half_factor(m[n][0], mx[0]), half_factor(m[n][1], mx[1])};
                const float corr[2] = {half[0] * half[0], half[1] * half[1]};
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        // the maximum first: it may be so large that kWeightExp beside it rounds away
                        s[n][mt][x] = exp2_approx((s[n][mt][x] - mx[x & 1]) + kWeightExp);
                        sum[x & 1] = fmaf(s[n][mt][x], rsv[mt], sum[x & 1]);
                    }
                    pf[n][mt][0] = transpose8x8(pack_half(s[n][mt][0] * kToHalf, s[n][mt][1] * kToHalf));
                    pf[n][mt][1] = transpose8x8(pack_half(s[n][mt][2] * kToHalf, s[n][mt][3] * kToHalf));
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    l[n][h] = fmaf(l[n][h] * half[h], half[h], sum[h]);
                    m[n][h] = mx[h];
                }
                // outputs so far to the new maximum
                if (!(st.flags & kFirst)) {
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        o[n][j][0] *= corr[0];
                        o[n][j][1] *= corr[1];
                        o[n][j][2] *= corr[0];
                        o[n][j][3] *= corr[1];
                    }
                }
            }
            // values: 16 dimensions by 16 positions a time
#pragma unroll
            for (int jp = 0; jp < D / 32; ++jp)
#pragma unroll
                for (int kt = 0; kt < 2; ++kt) {
                    uint32_t r[4];
                    ldmatrix4_trans(r, vs_base + tile_offset<D>(kt * 16 + mrow, 2 * jp + mgrp));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // bytes (key 2t: d, d + 1)(key 2t + 1: d, d + 1) -> both keys of d, both of d + 1
                        const uint32_t lo = __byte_perm(r[2 * x], 0, 0x3120), hi = __byte_perm(r[2 * x + 1], 0, 0x3120);
                        const uint32_t a0 = codes_f16(lo), a1 = codes_f16(lo >> 16);
                        const uint32_t a2 = codes_f16(hi), a3 = codes_f16(hi >> 16);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma(o[n][2 * jp + x], a0, a1, a2, a3, pf[n][kt][0], pf[n][kt][1]);
                    }
                }
        }
        warp_arrive(&sm.empty[slot]);
        slot += 2;
        if (slot >= S::kStages) {
            slot -= S::kStages;
            parity ^= 1;
        }
        if (st.flags & kLast) {
            const int buf = S::kStates == 1 ? 0 : item & 1;
            ++item;
            if constexpr (S::kStates == 1)
                if (!wait_for(sm, a, &sm.helped[item & 1], (item >> 1) & 1))   // the states of the item before have been read
                    break;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = l[n][h];
                    x += __shfl_xor_sync(kFull, x, 4);
                    x += __shfl_xor_sync(kFull, x, 8);
                    x += __shfl_xor_sync(kFull, x, 16);
                    const int head = n * 8 + 2 * t + h;
                    if (g == 0)
                        sm.ml[buf][warp][head] = make_float2(m[n][h], x);
                    if (head < a.group) {
#pragma unroll
                        for (int j = 0; j < D / 16; ++j)
                            *reinterpret_cast<float2 *>(&sm.state[buf][warp][0][0] + state_offset<D>(head, 16 * j + 2 * g)) =
                                make_float2(o[n][j][h], o[n][j][2 + h]);
                    }
                }
            warp_arrive(&sm.states[(item - 1) & 1]);
        }
    }
}

// Queries of an item as fp16 with a power of two taken out: helper warp w converts heads w, w +
// kHelpers, ..., four dimensions a lane.
template <int D, int MG>
struct Queries {
    static constexpr int kHeads = (MG + kHelpers - 1) / kHelpers;
    uint2 x[kHeads];
    int e[kHeads];       // the query's factor is scale_m * 2^e

    __device__ __forceinline__ void load(const AttnArgs &a, const Item &it, int w)
    {
        const int lane = threadIdx.x & 31;
        const __nv_bfloat16 *from = a.q + it.b * a.ldq + static_cast<int64_t>(it.kvh) * a.group * D + lane * 4;
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int head = w + i * kHelpers;
            x[i] = make_uint2(0, 0);
            if (it.b >= 0 && head < a.group && lane < D / 4)
                x[i] = __ldg(reinterpret_cast<const uint2 *>(from + head * D));
        }
    }
    __device__ __forceinline__ void convert(const AttnArgs &a)
    {
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            uint32_t top = max(max(x[i].x & 0x7fffu, (x[i].x >> 16) & 0x7fffu), max(x[i].y & 0x7fffu, (x[i].y >> 16) & 0x7fffu));
            top = __reduce_max_sync(kFull, top);
            // the largest magnitude goes to [2^14, 2^15)
            const int out = top == 0 ? 0 : max(-120, static_cast<int>(top >> 7) - 127 - 14);
            const float down = pow2(-out);
            x[i] = make_uint2(pack_half(__uint_as_float(x[i].x << 16) * down, __uint_as_float(x[i].x & 0xffff0000u) * down),
                              pack_half(__uint_as_float(x[i].y << 16) * down, __uint_as_float(x[i].y & 0xffff0000u) * down));
            e[i] = a.scale_e + out;
        }
    }
    __device__ __forceinline__ void store(Shared<D, MG> &sm, const AttnArgs &a, int buf, int w) const
    {
        const int lane = threadIdx.x & 31, ks = lane >> 2;
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            const int head = w + i * kHelpers;
            if (head < a.group) {
                if (lane < D / 4)   // as the consumers' lanes hold them
                    reinterpret_cast<uint2 *>(&sm.q[buf][head >> 3][ks >> 1][(head & 7) * 4 + (lane & 3)])[ks & 1] = x[i];
                if (lane == 0) {   // below 2^-126 it makes scores of at most 2^-31 either way
                    sm.qc[buf][head] = a.scale_m * pow2(max(-126, min(127, e[i])));
                    sm.qe[buf][head] = e[i];
                }
            }
        }
    }
};

// Four dimensions of a query head of an item: its result, or its chunk's part, from the maximum, the sum
// and the outputs that belong to them.
template <int D>
__device__ __forceinline__ void put(const AttnArgs &a, const Item &it, int head, int dd, float mx, float sum, const float4 &acc)
{
    const int h = it.kvh * a.group + head;
    const int64_t row = static_cast<int64_t>(it.b) * a.hq + h;
    if (it.chunks == 1) {
        const float r = kOutput / sum;
        uint2 y;
        *reinterpret_cast<__nv_bfloat162 *>(&y.x) = __floats2bfloat162_rn(acc.x * r, acc.y * r);
        *reinterpret_cast<__nv_bfloat162 *>(&y.y) = __floats2bfloat162_rn(acc.z * r, acc.w * r);
        *reinterpret_cast<uint2 *>(a.out + it.b * a.ldo + static_cast<int64_t>(h) * D + dd) = y;
        if (a.lse && dd == 0)
            a.lse[row] = (mx + log2f(sum)) * kLn2;
    } else {
        const int64_t at = row * a.chunks + it.chunk;
        *reinterpret_cast<float4 *>(a.part + at * D + dd) = acc;
        if (dd == 0)
            a.part_ml[at] = make_float2(mx, sum);
    }
}

// The eight states of an item added in warp order.
template <int D, int MG>
__device__ __forceinline__ void add_states(Shared<D, MG> &sm, const AttnArgs &a, const Item &it, int buf, int tid)
{
    constexpr int kQuads = D / 4;
#pragma unroll 2
    for (int x = tid; x < a.group * kQuads; x += 32 * kHelpers) {
        const int head = x / kQuads, dd = (x % kQuads) * 4;
        float2 ml[kConsumers];
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
            ml[w] = sm.ml[buf][w][head];
            mx = fmaxf(mx, ml[w].x);
        }
        float sum = 0.0f;
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kConsumers; ++w) {
            const float4 v = *reinterpret_cast<const float4 *>(&sm.state[buf][w][0][0] + state_offset<D>(head, dd));
            const float half = half_factor(ml[w].x, mx), f = half * half;
            sum = fmaf(ml[w].y * half, half, sum);
            acc.x = fmaf(v.x, f, acc.x);
            acc.y = fmaf(v.y, f, acc.y);
            acc.z = fmaf(v.z, f, acc.z);
            acc.w = fmaf(v.w, f, acc.w);
        }
        put<D>(a, it, head, dd, mx, sum, acc);
    }
}

// NaN in this warp's share of the block's items from number `from` on.  The table of items is not used:
// warps that have given up no longer keep one another's pace, on which refilling it depends.
template <int D, int MG>
__device__ __noinline__ void give_up(const Shared<D, MG> &sm, const AttnArgs &a, int from, int tid)
{
    const int lane = tid & 31;
    for (int first = from;; first += 32) {
        const Item mine = make_item(a, sm, first + lane);
        for (int l = 0; l < 32; ++l) {
            Item it = {};
            it.b = __shfl_sync(kFull, mine.b, l);
            it.kvh = __shfl_sync(kFull, mine.kvh, l);
            it.chunk = __shfl_sync(kFull, mine.chunk, l);
            it.chunks = __shfl_sync(kFull, mine.chunks, l);
            if (it.b < 0)
                return;
            for (int x = tid; x < a.group * (D / 4); x += 32 * kHelpers)
                put<D>(a, it, x / (D / 4), x % (D / 4) * 4, NAN, NAN, make_float4(NAN, NAN, NAN, NAN));
        }
    }
}

// The outputs of sequences that have no chunks: 0 and -inf, or NaN.  CTA c looks at sequences c, c +
// gridDim, ..., 32 a warp at a time.  (In a padded batch they would cost an item for each head.)
template <int D>
__device__ __forceinline__ void fill_empty(const AttnArgs &a, int w)
{
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kHelpers;
    for (int64_t b0 = blockIdx.x + static_cast<int64_t>(gridDim.x) * w; b0 < a.b; b0 += 32 * step) {
        const int64_t mine = b0 + lane * step;
        const int len = mine < a.b ? a.lens[mine] : 1;
        const bool bad = mine < a.b && (len < 0 || len > a.max_len);
        const uint32_t bads = __ballot_sync(kFull, bad);
        for (uint32_t todo = __ballot_sync(kFull, bad || len == 0); todo != 0; todo &= todo - 1) {
            const int l = __ffs(todo) - 1;
            const int64_t b = b0 + l * step;
            const bool nan = (bads >> l) & 1u;
            const uint32_t y = nan ? 0x7fff7fffu : 0u;   // two bf16
            for (int x = lane; x < a.hq * D / 8; x += 32)
                reinterpret_cast<uint4 *>(a.out + b * a.ldo)[x] = make_uint4(y, y, y, y);
            if (a.lse)
                for (int x = lane; x < a.hq; x += 32)
                    a.lse[b * a.hq + x] = nan ? NAN : -INFINITY;
        }
    }
}

template <int D, int MG>
__device__ __forceinline__ void help(Shared<D, MG> &sm, const AttnArgs &a, int w)
{
    Queries<D, MG> q;
    for (int i = 0; i < 2; ++i) {
        q.load(a, sm.items[i], w);
        q.convert(a);
        q.store(sm, a, i, w);
        warp_arrive(&sm.helped[i]);
    }
    fill_empty<D>(a, w);
    for (int i = 0;; ++i) {
        const Item now = sm.items[i % kItemRing];
        if (now.b < 0)
            break;
        // the queries of the item after next come while this one's states do (both in turn took 1.3 us
        // an item, more than a chunk of one step)
        const Item then = sm.items[(i + 2) % kItemRing];
        q.load(a, then, w);
        q.convert(a);
        if (!wait_for(sm, a, &sm.states[i & 1], (i >> 1) & 1)) {
            give_up(sm, a, i, threadIdx.x - 32 * kConsumers);
            break;
        }
        if (then.b >= 0)
            q.store(sm, a, i & 1, w);   // every consumer has read item i's
        add_states(sm, a, now, Shared<D, MG>::kStates == 1 ? 0 : i & 1, threadIdx.x - 32 * kConsumers);
        // A block of the table whose items are behind item i - 1 makes room for the one four further on.
        // No helper warp is behind item i - 1 (item i's states were written after all of them had arrived
        // for item i - 2), and the other warps read the new entries behind the barriers of the items between.
        if (w == 0 && i > 1 && (i - 1) % kItemBlock == 0) {
            const int lane = threadIdx.x & 31, first = i - 1 - kItemBlock;
            sm.items[(first + lane) % kItemRing] = make_item(a, sm, first + kItemRing + lane);
        }
        warp_arrive(&sm.helped[i & 1]);
    }
}

template <int D, int MG>
__global__ void __launch_bounds__(kThreads, 1)
paged_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const __grid_constant__ AttnArgs a)
{
    using S = Shared<D, MG>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            bi::ptx::mbar_init(&sm.full[i], 1);
            bi::ptx::mbar_init(&sm.empty[i], kTiles);
        }
        bi::ptx::mbar_init(&sm.states[0], kConsumers);
        bi::ptx::mbar_init(&sm.states[1], kConsumers);
        bi::ptx::mbar_init(&sm.helped[0], kHelpers);
        bi::ptx::mbar_init(&sm.helped[1], kHelpers);
        bi::ptx::fence_mbarrier_init();
        bi::ptx::prefetch_tmap(&k_map);
        bi::ptx::prefetch_tmap(&v_map);
        sm.dead = 0;
    }
    // query columns that no head fills stay zero
    for (int x = tid; x < 2 * S::NT * (D / 32) * 32; x += kThreads)
        (&sm.q[0][0][0][0])[x] = make_uint4(0, 0, 0, 0);
    if (tid < 2 * S::kCols) {
        (&sm.qc[0][0])[tid] = 0.0f;
        (&sm.qe[0][0])[tid] = 0;
    }
    bi_kv::dependency_wait();

    // chunks before each entry, class by class, one entry a thread
    const int per = (a.b + kEntries - 1) / kEntries;
    static_assert(kThreads >= kEntries, "one entry a thread");
    int n[kClasses] = {}, incl[kClasses];
    if (tid < kEntries)
        for (int b = tid * per; b < (tid + 1) * per && b < a.b; ++b) {
            const int len = a.lens[b];
            if (per == 1)
                sm.len[tid] = len;
            const Span s = span_of(len, a);
#pragma unroll
            for (int c = 0; c < kClasses; ++c)
                n[c] += chunks_of_class(s, c);
        }
#pragma unroll
    for (int c = 0; c < kClasses; ++c) {
        incl[c] = n[c];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(kFull, incl[c], off);
            if (lane >= off)
                incl[c] += y;
        }
        if (lane == 31)
            sm.warp_sum[c][warp] = incl[c];
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kClasses; ++c) {
        int before = incl[c] - n[c], total = 0;
#pragma unroll
        for (int w = 0; w < kEntries / 32; ++w) {
            before += w < warp ? sm.warp_sum[c][w] : 0;
            total += sm.warp_sum[c][w];
        }
        // entries behind the last sequence hold INT_MAX
        if (tid < kEntries)
            sm.first_chunk[c][tid] = tid * per < a.b ? before : INT_MAX;
        if (tid == 0)
            sm.class_chunks[c] = total;
    }
    __syncthreads();
    if (tid < kItemRing)
        sm.items[tid] = make_item(a, sm, tid);
    __syncthreads();
    bi_kv::launch_dependents();   // the merge kernel's CTAs take the places that CTAs of this one leave
    if (warp < kConsumers)
        consume(sm, a, warp);
    else if (warp < kConsumers + kHelpers)
        help(sm, a, warp - kConsumers);
    else
        produce(sm, a, &k_map, &v_map);
}

// The chunks of one query head added; sequences of one chunk are done already.  Chunks are added
// eight at a time in ascending order, and the eights in ascending order, so how many warps share
// the eights of a head changes no bit: kWide warps, and kRows heads in a block.  Latency bound: a
// warp has its eight parts in flight at once.
constexpr int kEight = 8;

template <int D, int kWide>
__global__ void __launch_bounds__(kWide < 8 ? 256 : 32 * kWide) paged_merge_kernel(const __grid_constant__ AttnArgs a)
{
    constexpr int kRows = kWide < 8 ? 8 / kWide : 1;
    constexpr int kVec = D / 32;   // dimensions a lane
    constexpr int kEights = kWide == 1 ? 1 : kMaxChunks / kEight;
    __shared__ float acc_s[kRows][kEights][D];
    __shared__ float2 ml_s[kRows][kEights];
    const int lane = threadIdx.x & 31, r = (threadIdx.x >> 5) / kWide, w = (threadIdx.x >> 5) % kWide;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + r;
    bi_kv::dependency_wait();
    const bool real = row < static_cast<int64_t>(a.b) * a.hq;
    const int b = real ? static_cast<int>(row / a.hq) : 0;
    float v[kEight][kVec];
    float2 x[kEight];
    auto load_eight = [&](int e, int limit) {   // parts below the limit; the others stay what they are
        const float2 *ml = a.part_ml + row * a.chunks + e * kEight;
        const float *part = a.part + (row * a.chunks + e * kEight) * D + lane * kVec;
#pragma unroll
        for (int j = 0; j < kEight; ++j)
            if (e * kEight + j < limit) {
                x[j] = ml[j];
                if constexpr (kVec == 4)
                    *reinterpret_cast<float4 *>(v[j]) = *reinterpret_cast<const float4 *>(part + j * D);
                else
                    *reinterpret_cast<float2 *>(v[j]) = *reinterpret_cast<const float2 *>(part + j * D);
            }
    };
    // With at most eight chunks the parts are asked for before the length is known; those of chunks
    // that the sequence does not have (never written, or by an earlier call) are not used.
    if constexpr (kWide == 1)
        if (real)
            load_eight(0, a.chunks);
    const int chunks = real ? span_of(a.lens[b], a).chunks : 0;
    const int eights = chunks <= 1 ? 0 : (chunks + kEight - 1) / kEight;
    for (int e = w; e < eights; e += kWide) {
        if constexpr (kWide > 1)
            load_eight(e, chunks);
#pragma unroll
        for (int j = 0; j < kEight; ++j)
            if (e * kEight + j >= chunks) {
                x[j] = make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    v[j][i] = 0.0f;
            }
        float mx = -INFINITY, sum = 0.0f, acc[kVec] = {};
#pragma unroll
        for (int j = 0; j < kEight; ++j)
            mx = fmaxf(mx, x[j].x);
#pragma unroll
        for (int j = 0; j < kEight; ++j) {
            // a chunk of NaN scores has no maximum: its sum is NaN and stays so
            const float half = half_factor(x[j].x, mx == -INFINITY ? 0.0f : mx), f = half * half;
            sum = fmaf(x[j].y * half, half, sum);
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                acc[i] = fmaf(v[j][i], f, acc[i]);
        }
        if (lane == 0)
            ml_s[r][e] = make_float2(mx, sum);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            acc_s[r][e][lane * kVec + i] = acc[i];
    }
    if constexpr (kWide > 1)
        __syncthreads();
    else
        __syncwarp();
    if (w != 0 || eights == 0)
        return;
    float mx = -INFINITY, sum = 0.0f, acc[kVec] = {};
    for (int e = 0; e < eights; ++e)
        mx = fmaxf(mx, ml_s[r][e].x);
    for (int e = 0; e < eights; ++e) {
        const float half = half_factor(ml_s[r][e].x, mx == -INFINITY ? 0.0f : mx), f = half * half;
        sum = fmaf(ml_s[r][e].y * half, half, sum);
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            acc[i] = fmaf(acc_s[r][e][lane * kVec + i], f, acc[i]);
    }
    const float inv = kOutput / sum;
    __nv_bfloat16 *out = a.out + b * a.ldo + (row - static_cast<int64_t>(b) * a.hq) * D + lane * kVec;
#pragma unroll
    for (int i = 0; i < kVec; i += 2)
        *reinterpret_cast<__nv_bfloat162 *>(out + i) = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
    if (a.lse && lane == 0)
        a.lse[row] = (mx + log2f(sum)) * kLn2;
}

template <int D, int kWide>
bi_status_t run_merge(const AttnArgs &a, cudaStream_t stream)
{
    constexpr int kRows = kWide < 8 ? 8 / kWide : 1;
    const int64_t rows = static_cast<int64_t>(a.b) * a.hq;
    return bi_kv::launch(paged_merge_kernel<D, kWide>, dim3(static_cast<unsigned>((rows + kRows - 1) / kRows)),
                         dim3(32 * kWide * kRows), 0, stream, 1, a);
}

// The most chunks a sequence of up to max_len positions can have: chunk_steps() jumps at 4, 16 and
// 512 steps, where the number of chunks falls.
int64_t most_chunks(int64_t max_len)
{
    const int64_t steps = (max_len + kStep - 1) / kStep;
    int64_t most = 1;
    for (int64_t s : {INT64_C(4), INT64_C(16), INT64_C(4) * kMaxChunks, steps}) {
        const int64_t n = s < steps ? s : steps;
        if (n > 0) {
            const int64_t per = chunk_steps(static_cast<int>(n)), chunks = (n + per - 1) / per;
            most = chunks > most ? chunks : most;
        }
    }
    return most;
}

template <int D, int MG>
bi_status_t run_attention(const AttnArgs &a, const CUtensorMap &k_map, const CUtensorMap &v_map, int dev, int sms, cudaStream_t stream)
{
    static std::mutex mu;
    static bool set[bi_kv::kMaxDevices] = {};
    static_assert(sizeof(Shared<D, MG>) <= 232448, "shared memory of an SM");
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
            if (cudaFuncSetAttribute(paged_attention_kernel<D, MG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(sizeof(Shared<D, MG>))) != cudaSuccess) {
                cudaGetLastError();
                return BI_ERR_CUDA;
            }
            set[dev] = true;
        }
    }
    // no more CTAs than there can be items
    const int64_t items = static_cast<int64_t>(a.b) * a.heads * a.chunks;
    const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
    bi_status_t st = bi_kv::launch(paged_attention_kernel<D, MG>, dim3(grid), dim3(kThreads), sizeof(Shared<D, MG>), stream, 1,
                                  k_map, v_map, a);
    if (st != BI_OK || a.chunks == 1)
        return st;
    // Warps for a head: one or two where no sequence can have more eights of chunks; else four, or sixteen
    // (all eights at once) while there is at most one head for an SM.  The call with four and with
    // sixteen, 16/1 heads: 131000 positions, 32 heads in all 28.7 and 25.1 us, 128 heads 66.1 and 62.4,
    // 256 heads 117.4 and 116.3; 40000 positions, 128 heads 32.5 and 31.4, 256 heads 48.0 and 48.8, 512
    // heads 77.4 and 82.0; 20 ragged sequences of up to 30000, 640 heads 44.4 and 48.3.
    const int eights = (a.chunks + kEight - 1) / kEight;
    return eights <= 1   ? run_merge<D, 1>(a, stream)
           : eights <= 2 ? run_merge<D, 2>(a, stream)
           : eights <= 4 || static_cast<int64_t>(a.b) * a.hq > sms ? run_merge<D, 4>(a, stream)
                                                                   : run_merge<D, 16>(a, stream);
}

std::atomic<uint64_t> wait_ns{kWaitNs};
std::atomic<uint32_t> debug_skip_load{0};

} // namespace

extern "C" {

bi_status_t bi_paged_decode_attention_set_wait_timeout(uint64_t timeout_ns)
{
    wait_ns = timeout_ns ? timeout_ns : kWaitNs;
    return BI_OK;
}

bi_status_t bi_paged_decode_attention_debug_skip_load(uint32_t n)
{
    debug_skip_load = n;
    return BI_OK;
}

size_t bi_paged_decode_attention_workspace_bytes(int64_t B, int Hq, int D, int64_t max_len)
{
    if (B < 1 || Hq < 1 || max_len < 1 || B > kMaxBatch || B * Hq > INT32_MAX || (D != 64 && D != 128) || max_len > kMaxLen)
        return 0;   // the call refuses these, and the sizes below would not fit their types
    const int64_t chunks = most_chunks(max_len);
    return chunks == 1 ? 0 : static_cast<size_t>(B) * Hq * chunks * (D + 2) * sizeof(float);
}

bi_status_t bi_paged_decode_attention(const bi_kv_cache_t *cache, const void *Q, int64_t ldq,
                                      const int32_t *block_table, int64_t ld_table,
                                      int64_t max_pages, const int32_t *seq_lens, int64_t B, int Hq,
                                      float scale, int64_t window, void *workspace,
                                      size_t workspace_bytes, void *O, int64_t ldo, float *lse,
                                      cudaStream_t stream)
{
    bi_status_t st = bi_kv::check_cache(cache);
    if (st != BI_OK)
        return st;
    const int64_t row = static_cast<int64_t>(Hq) * cache->head_dim;
    if (B < 0 || Hq < 1 || max_pages < 0 || ld_table < max_pages || window < 0 || ldq < row || ldo < row ||
        !std::isfinite(scale))
        return BI_ERR_INVALID_ARG;
    if (Hq % cache->num_heads != 0 || Hq / cache->num_heads > kMaxGroup || max_pages > INT32_MAX / cache->page_size ||
        B > kMaxBatch || B * Hq > INT32_MAX || ldq > (INT64_C(1) << 40) || ldo > (INT64_C(1) << 40) || ld_table > (INT64_C(1) << 40))
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (B == 0)
        return BI_OK;
    if (!Q || !O || !seq_lens || (max_pages > 0 && !block_table))
        return BI_ERR_INVALID_ARG;
    if (!bi_kv::aligned(Q, 16) || !bi_kv::aligned(O, 16) || ldq % 8 || ldo % 8 || !bi_kv::aligned(block_table, 4) ||
        !bi_kv::aligned(seq_lens, 4) || !bi_kv::aligned(lse, 4))
        return BI_ERR_ALIGNMENT;
    const int64_t max_len = max_pages * cache->page_size;
    if (max_len > kMaxLen || B * cache->num_heads > (INT64_C(1) << 30) / most_chunks(max_len))
        return BI_ERR_UNSUPPORTED_SHAPE;
    const size_t need = bi_paged_decode_attention_workspace_bytes(B, Hq, cache->head_dim, max_len);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return BI_ERR_INVALID_ARG;
        if (!bi_kv::aligned(workspace, 16))
            return BI_ERR_ALIGNMENT;
    }
    int dev = 0, sms = 0;
    if ((st = bi_kv::current_device(&dev, &sms)) != BI_OK)
        return st;
    AttnArgs a = {};
    a.q = static_cast<const __nv_bfloat16 *>(Q);
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.table = block_table;
    a.lens = seq_lens;
    a.out = static_cast<__nv_bfloat16 *>(O);
    a.lse = lse;
    a.ldq = ldq;
    a.ldo = ldo;
    a.ld_table = ld_table;
    a.window = window;
    a.num_pages = static_cast<int>(cache->num_pages);
    a.max_len = static_cast<int>(max_len);
    a.b = static_cast<int>(B);
    a.hq = Hq;
    a.heads = cache->num_heads;
    a.group = Hq / cache->num_heads;
    a.page_shift = bi_kv::log2_of(cache->page_size);
    a.chunks = static_cast<int>(most_chunks(max_len));
    a.scale_m = std::frexp(scale, &a.scale_e) * kLog2e;
    a.skip_load = debug_skip_load;
    // two cycles a nanosecond, at or above the highest SM clock; a limit of centuries stays one
    const uint64_t ns = wait_ns;
    a.wait_cycles = ns > UINT64_MAX / 4 ? UINT64_MAX / 2 : 2 * ns;
    a.part = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(a.part + B * Hq * a.chunks * cache->head_dim);
    CUtensorMap k_map, v_map;
    if ((st = bi_kv::page_map(&k_map, cache, cache->k)) != BI_OK || (st = bi_kv::page_map(&v_map, cache, cache->v)) != BI_OK)
        return st;
    // Groups of up to four heads of 128 have a kernel of their own: 16 x 4096 of 4 heads takes 30.8 us, in
    // the kernel for eight 31.2, of 2 heads 31.3 and 31.5 (less work for the helper warps; elsewhere equal).
    if (cache->head_dim == 128)
        return a.group <= 4   ? run_attention<128, 4>(a, k_map, v_map, dev, sms, stream)
               : a.group <= 8 ? run_attention<128, 8>(a, k_map, v_map, dev, sms, stream)
                              : run_attention<128, 16>(a, k_map, v_map, dev, sms, stream);
    return a.group <= 8 ? run_attention<64, 8>(a, k_map, v_map, dev, sms, stream)
                        : run_attention<64, 16>(a, k_map, v_map, dev, sms, stream);
}

} // extern "C"
