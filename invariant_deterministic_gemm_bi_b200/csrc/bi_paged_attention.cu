// bi_paged_attention.cu -- decode attention over the paged 8-bit cache
// (include/bi_paged_attention.h).
//
// Memory bound: a key and a value of one head are 2 D bytes for at most 16 query heads, so the
// kernel streams the cache once and everything else has to hide behind that.
//
// Work.  A sequence's positions are cut into steps of 256 at multiples of 256, and runs of steps
// into chunks whose length follows from the number of steps alone.  An item is one chunk of one
// key/value head; persistent CTAs take items round robin.  Warp w of a CTA owns positions
// 32 w .. 32 w + 31 of every step and keeps a softmax state of its own over the chunk; the eight
// states are added in warp order at the chunk's end, and the chunks in ascending order by a second
// kernel.  Every sum's order is thus fixed by the sequence's length and window.
//
// Loads.  Each warp streams its own tiles through a private ring of stages with cp.async: rows
// outside the sequence are filled with zeros (so a stale NaN code cannot reach a sum through a
// zero weight); page numbers come twice as many tiles ahead as codes.  No CTA-wide hand-off.
//
// Matrix products.  The cache is the first operand of mma.m16n8k16 (16 positions, or 16 dimensions,
// a time) and the query heads are the 8 columns, so grouped queries fill the tile instead of
// padding it to 16 rows.  e4m3 codes become fp16 exactly; queries become fp16 exactly after a power
// of two per head has been taken out of them (bf16 has fewer significant bits; entries below 2^-29
// of the head's largest lose bits that are below the fp32 sum's own).  The order of dimensions
// inside a 16-byte group is permuted alike on both sides, so codes go from ldmatrix to the
// conversion without shuffles; values are read transposed, two dimensions to a 16-bit element.
// tcgen05 would need the weights and queries split into several e4m3 parts, or the codes written
// back to shared memory as fp16, to save instructions that are not the bound.
//
// Weights.  With sv the value scale of a position's page, the state's maximum M is that of
// t_j = s_j log2 e + log2 sv, and the weight of a value's code is a_j = 2^(t_j - M + 15) <= 2^15,
// rounded to fp16 (2^-11 of itself, a quarter of what bf16 would cost; the output is rounded to bf16
// anyway); the softmax sum adds a_j / sv in fp32.  The value scale so costs nothing per element and
// weights down to 2^-29 of the largest keep all of fp16's bits, whatever the scales.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "bi_kv_common.cuh"
#include "bi_paged_attention.h"

namespace {

using bi_kv::kFull;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;                   // positions of a warp's tile
constexpr int kStep = kWarps * kTile;       // positions of a CTA's step
constexpr int kMaxChunks = 128;             // chunks of a sequence
constexpr int kMaxGroup = 16;               // query heads of a key/value head
constexpr int kEntries = 512;               // entries of the scanned chunk counts
constexpr int kMaxBatch = kEntries * 32;    // an entry stands for up to 32 sequences
constexpr int kDescs = 16;                  // ring of tile descriptors
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kWeightExp = 15.0f;         // weights are held times 2^15

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
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    __nv_bfloat16 *out;
    float *lse;
    float *part;        // [b][hq][chunks][D] unnormalised outputs
    float2 *part_ml;    // [b][hq][chunks] (M, sum)
    int64_t ldq, ldo, ld_table, page_stride, token_stride, head_stride;
    int64_t window;
    int num_pages, max_len, b, hq, heads, group, page_shift, chunks;
    float scale;
};

// What of a sequence is attended: positions [lo, hi), in steps from `first`.
struct Span {
    int lo, hi, first, steps, per_chunk, chunks;
    bool bad;
};

__device__ __forceinline__ Span span_of(int len, const AttnArgs &a)
{
    Span s;
    s.bad = len < 0 || len > a.max_len;
    s.hi = s.bad ? 0 : len;
    s.lo = a.window > 0 && s.hi > a.window ? s.hi - static_cast<int>(a.window) : 0;
    s.first = s.lo / kStep;
    s.steps = (s.hi + kStep - 1) / kStep - s.first;
    s.steps = s.steps < 1 ? 1 : s.steps;   // an empty sequence is one empty step
    s.per_chunk = chunk_steps(s.steps);
    s.chunks = (s.steps + s.per_chunk - 1) / s.per_chunk;
    return s;
}

// One warp's tile.
enum : int { kFirst = 1, kLast = 2, kEnd = 4, kBad = 8, kHalf0 = 16, kHalf1 = 32, kWhole = 64 };
struct Desc {
    int b, kvh, key0, lo, hi, flags, chunk, chunks;
};
static_assert(sizeof(Desc) == 32, "two 16-byte words");

// ---------------------------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// 16 bytes, or 16 zero bytes when `valid` is false (nothing is read then)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// s, or NaN unless 2^-64 <= s <= 2^64
__device__ __forceinline__ float checked_scale(float s) { return s >= 0x1p-64f && s <= 0x1p64f ? s : NAN; }

// ---------------------------------------------------------------------------------------------
// shared memory
// ---------------------------------------------------------------------------------------------

template <int D, int NT>
struct Shared {
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kAhead = kStages - 1;              // tiles of codes in flight
    static constexpr int kQueries = kAhead + 2;             // items whose queries are held
    static constexpr int kMatrix = kTile * D;               // bytes of a tile's keys (or values)
    uint8_t ring[kWarps][kStages][2][kMatrix];              // codes; at a chunk's end a warp's outputs
    alignas(16) __nv_bfloat16 q[kQueries][NT * 8][D];
    float4 scale[kWarps][kStages];                          // key scales of the halves, value scales
    Desc desc[kWarps][kDescs];
    int32_t page[kWarps][kDescs][2];                    // page numbers of a tile's halves
    float2 ml[kWarps][NT * 8];
    int32_t first_chunk[kEntries + 32];                     // chunks before each entry
    int32_t len[kEntries];                                  // lengths, when an entry is one sequence
    int32_t warp_sum[kWarps];
};

// Byte of the 16-byte group `grp` of row `row` inside a tile: groups are spread over the banks so
// that eight rows of one group (a matrix of ldmatrix) touch all of them once.
template <int D>
__device__ __forceinline__ int tile_offset(int row, int grp)
{
    return row * D + ((D == 128 ? grp ^ (row & 7) : grp ^ ((row >> 1) & 3)) << 4);
}

// Float of dimension d (even) of column `head` inside a warp's outputs: the columns 2t of a quad
// fall on different banks.
template <int D>
__device__ __forceinline__ int out_offset(int head, int d)
{
    return head * D + (d ^ (((head >> 1) & 3) << 3));
}

// Walks the items of this CTA and the steps of each, giving one warp's tiles in order.
struct Cursor {
    int item, items, stride;   // item = chunk ordinal * heads + key/value head
    int u, du, dh;             // chunk ordinal; the stride's quotient and remainder by the heads
    const int32_t *pages;      // the sequence's row of the block table
    int step, steps;           // of the current chunk
    Desc d;
    int chunk_key;             // the chunk's first position
};

__device__ __forceinline__ int len_of(const AttnArgs &a, const int32_t *len_s, int b)
{
    return a.b <= kEntries ? len_s[b] : a.lens[b];
}

// The sequence and chunk of chunk ordinal u (all lanes alike).
__device__ __forceinline__ void open_item(Cursor &c, const AttnArgs &a, const int32_t *first_chunk, const int32_t *len_s)
{
    const int lane = threadIdx.x & 31;
    const int u = c.u;
    // the last entry with first_chunk <= u: 16 entries a lane, then one
    const int blk = __popc(__ballot_sync(kFull, first_chunk[lane * 16] <= u)) - 1;
    const int e = blk * 16 + __popc(__ballot_sync(kFull, lane < 16 && first_chunk[blk * 16 + lane] <= u)) - 1;
    int chunk = u - first_chunk[e], b = e;
    Span s;
    if (a.b <= kEntries) {
        s = span_of(len_s[b], a);
    } else {
        // an entry is `per` consecutive sequences
        const int per = (a.b + kEntries - 1) / kEntries;
        const int mine = e * per + lane;
        const bool own = lane < per && mine < a.b;
        const Span x = span_of(own ? a.lens[mine] : 0, a);
        int incl = own ? x.chunks : 0;
        const int n = incl;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, off);
            if (lane >= off)
                incl += y;
        }
        const int at = __ffs(__ballot_sync(kFull, incl > chunk)) - 1;
        chunk -= __shfl_sync(kFull, incl - n, at);
        b = e * per + at;
        s = span_of(a.lens[b], a);
    }
    c.d.b = b;
    c.d.lo = s.lo;
    c.d.hi = s.hi;
    c.d.chunk = chunk;
    c.d.chunks = s.chunks;
    c.d.flags = s.bad ? kBad : 0;
    c.pages = a.table + b * a.ld_table;
    c.step = 0;
    c.steps = min(s.per_chunk, s.steps - chunk * s.per_chunk);
    c.chunk_key = (s.first + chunk * s.per_chunk) * kStep;
}

// The cursor's tile, then one tile on.
__device__ __forceinline__ Desc next_tile(Cursor &c, const AttnArgs &a, const int32_t *first_chunk, const int32_t *len_s)
{
    Desc d = c.d;
    if (c.item >= c.items) {
        d.flags = kEnd;
        return d;
    }
    d.key0 = c.chunk_key + c.step * kStep + static_cast<int>(threadIdx.x >> 5) * kTile;
    d.flags |= d.key0 >= d.lo && d.key0 + kTile <= d.hi ? kWhole : 0;
    d.flags |= (c.step == 0 ? kFirst : 0) | (c.step == c.steps - 1 ? kLast : 0);
    d.flags |= (d.key0 < d.hi && d.key0 + kTile / 2 > d.lo ? kHalf0 : 0) |
               (d.key0 + kTile / 2 < d.hi && d.key0 + kTile > d.lo ? kHalf1 : 0);
    if (++c.step == c.steps) {
        c.item += c.stride;
        c.u += c.du;
        c.d.kvh += c.dh;
        if (c.d.kvh >= a.heads) {
            c.d.kvh -= a.heads;
            ++c.u;
        }
        if (c.item < c.items)
            open_item(c, a, first_chunk, len_s);
    }
    return d;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_kernel(const __grid_constant__ AttnArgs a)
{
    using S = Shared<D, NT>;
    constexpr int kCols = NT * 8;
    constexpr int kGroups = D / 16;                 // 16-byte groups of a row
    constexpr int kRows = 32 / kGroups;             // rows one load instruction of a warp covers
    constexpr int kQueries = S::kQueries;
    // page numbers are asked for kIds tiles ahead: the copies of that many less kAhead tiles ago, whose
    // group they are in, have been waited for when the codes are
    constexpr int kIds = 2 * S::kAhead;
    static_assert(kIds + 1 <= kDescs && (kDescs & (kDescs - 1)) == 0, "live descriptors");
    static_assert(kCols * D * 4 <= 2 * S::kMatrix, "a warp's outputs fit in a stage");
    extern __shared__ __align__(128) uint8_t smem_raw[];
    S &sm = *reinterpret_cast<S *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    bi_kv::dependency_wait();

    // chunks before each entry: thread i scans entries 2i and 2i + 1
    {
        const int per = (a.b + kEntries - 1) / kEntries;
        int n[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = 2 * tid + j;
            n[j] = 0;
            for (int b = e * per; b < (e + 1) * per && b < a.b; ++b) {
                const int len = a.lens[b];
                if (per == 1)
                    sm.len[e] = len;
                n[j] += span_of(len, a).chunks;
            }
        }
        int incl = n[0] + n[1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, off);
            if (lane >= off)
                incl += y;
        }
        if (lane == 31)
            sm.warp_sum[warp] = incl;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w)
            before += sm.warp_sum[w];
        // entries behind the last sequence hold INT_MAX but the first of them, which ends the scan
        const int base = before + incl - n[0] - n[1];
        const int last = (a.b + per - 1) / per;
        sm.first_chunk[2 * tid] = 2 * tid <= last ? base : INT_MAX;
        sm.first_chunk[2 * tid + 1] = 2 * tid + 1 <= last ? base + n[0] : INT_MAX;
        if (tid < 32)
            sm.first_chunk[kEntries + tid] = INT_MAX;
        __syncthreads();
    }
    int total = 0;
    for (int w = 0; w < kWarps; ++w)
        total += sm.warp_sum[w];
    Cursor cur;
    cur.item = blockIdx.x;
    cur.items = total * a.heads;
    cur.stride = gridDim.x;
    cur.u = cur.item / a.heads;
    cur.d.kvh = cur.item - cur.u * a.heads;
    cur.du = cur.stride / a.heads;
    cur.dh = cur.stride - cur.du * a.heads;
    if (cur.item >= cur.items)
        return;
    open_item(cur, a, sm.first_chunk, sm.len);

    // tile i: descriptor and page numbers
    auto ask_pages = [&](int i) {
        const int32_t *pages = cur.pages;
        const Desc d = next_tile(cur, a, sm.first_chunk, sm.len);
        if (lane < 2) {
            reinterpret_cast<int4 *>(&sm.desc[warp][i % kDescs])[lane] =
                lane == 0 ? make_int4(d.b, d.kvh, d.key0, d.lo) : make_int4(d.hi, d.flags, d.chunk, d.chunks);
            if (d.flags & (lane == 0 ? kHalf0 : kHalf1))
                copy4(smem_u32(&sm.page[warp][i % kDescs][lane]),
                      pages + ((d.key0 + lane * (kTile / 2)) >> a.page_shift));
        }
    };
    // this lane's 16-byte group and first row of a tile, in the cache and in shared memory
    const int grp = lane % kGroups, row0 = lane / kGroups;
    const int64_t lane_at = row0 * a.token_stride + grp * 16, row_step = kRows * a.token_stride;
    const uint32_t lane_dst = tile_offset<D>(row0, grp);
    // tile i: codes and scales, its page numbers having come
    auto ask_codes = [&](int i) {
        const Desc d = sm.desc[warp][i % kDescs];
        if (!(d.flags & (kHalf0 | kHalf1)))
            return;
        const int stage = i % S::kStages;
        const int page_mask = (1 << a.page_shift) - 1;
        int64_t base[2];
        bool ok[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int id = sm.page[warp][i % kDescs][h];
            const bool in = (d.flags & (h == 0 ? kHalf0 : kHalf1)) != 0;
            ok[h] = in && id >= 0 && id < a.num_pages;
            base[h] = ok[h] ? id * a.page_stride + ((d.key0 + h * (kTile / 2)) & page_mask) * a.token_stride +
                                  d.kvh * a.head_stride
                            : 0;
            if (lane == h || lane == h + 2) {   // lanes 0, 1: key scales, 2, 3: value scales
                float *dst = reinterpret_cast<float *>(&sm.scale[warp][stage]) + lane;
                if (ok[h])
                    copy4(smem_u32(dst), (lane < 2 ? a.k_scale : a.v_scale) + static_cast<int64_t>(id) * a.heads + d.kvh);
                else
                    *dst = in ? NAN : 1.0f;     // a page number out of range
            }
        }
        const uint32_t dst = smem_u32(&sm.ring[warp][stage][0][0]);
        if ((d.flags & kWhole) && ok[0] && ok[1]) {
            // 16 rows of each half; the swizzle of rows kRows apart repeats after one or two of them
            const int64_t from[2] = {base[0] + lane_at, base[1] + lane_at};
#pragma unroll
            for (int r = 0; r < kTile; r += kRows) {
                const int64_t at = from[r / (kTile / 2)] + (r % (kTile / 2)) / kRows * row_step;
                const uint32_t off = dst + r * D + (D == 128 && (r & 4) ? lane_dst ^ 64 : lane_dst);
                copy16(off, a.k + at, true);
                copy16(off + S::kMatrix, a.v + at, true);
            }
            return;
        }
#pragma unroll
        for (int r = 0; r < kTile; r += kRows) {
            const int row = r + row0, h = r >= kTile / 2 ? 1 : 0;
            const int key = d.key0 + row;
            const bool valid = ok[h] && key >= d.lo && key < d.hi;
            const int64_t at = valid ? base[h] + lane_at + (r % (kTile / 2)) / kRows * row_step : 0;
            const uint32_t off = dst + tile_offset<D>(row, grp);
            copy16(off, a.k + at, valid);
            copy16(off + S::kMatrix, a.v + at, valid);
        }
    };
    // the queries of tile i's item (item number n of this CTA): this warp's share
    auto ask_queries = [&](int i, int n) {
        const Desc d = sm.desc[warp][i % kDescs];
        const int vecs = a.group * (D / 8);
        const __nv_bfloat16 *src = a.q + d.b * a.ldq + static_cast<int64_t>(d.kvh) * a.group * D;
        for (int x = warp * 32 + lane; x < vecs; x += kThreads)
            copy16(smem_u32(&sm.q[n % kQueries][0][0]) + x * 16, src + x * 8, true);
    };

    // Queries run one tile further ahead than codes: the barrier at the end of the item before
    // makes the other warps' shares visible.
    for (int i = 0; i < kIds; ++i)
        ask_pages(i);
    copy_commit();
    copy_wait<0>();
    __syncwarp();
    int asked_items = 0;
#pragma unroll
    for (int i = 0; i < S::kAhead; ++i) {
        ask_codes(i);
        if (i == 0)   // the queries of the items that open in the first kAhead + 1 tiles
            for (int j = 0; j <= S::kAhead; ++j) {
                const int flags = sm.desc[warp][j].flags;
                if ((flags & kFirst) && !(flags & kEnd))
                    ask_queries(j, asked_items++);
            }
        copy_commit();
    }
    // zero columns of the query ring that no head fills, once
    for (int x = tid; x < kQueries * (kCols - a.group) * (D / 2); x += kThreads) {
        const int per = (kCols - a.group) * (D / 2);
        reinterpret_cast<uint32_t *>(&sm.q[x / per][a.group][0])[x % per] = 0;
    }
    copy_wait<S::kAhead - 1>();
    __syncthreads();

    uint32_t qf[NT][D / 16][2];       // queries as the second operand
    float qc[NT][2];                  // scale * log2 e * the power of two taken out, of heads 2t, 2t + 1
    float o[NT][D / 16][4];           // [dimension 16 j + 2 g, + 1][head 2t, 2t + 1]
    float m[NT][2], l[NT][2];
    int item = -1;

    for (int i = 0;; ++i) {
        copy_wait<S::kAhead - 1>();
        __syncwarp();
        const Desc d = sm.desc[warp][i % kDescs];
        if (d.flags & kEnd)
            break;
        ask_codes(i + S::kAhead);
        {
            const int flags = sm.desc[warp][(i + S::kAhead + 1) % kDescs].flags;
            if ((flags & kFirst) && !(flags & kEnd))
                ask_queries(i + S::kAhead + 1, asked_items++);
        }
        ask_pages(i + kIds);
        copy_commit();
        const int stage = i % S::kStages;

        if (d.flags & kFirst) {
            ++item;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 *row = reinterpret_cast<const uint2 *>(&sm.q[item % kQueries][n * 8 + g][0]);
                uint2 raw[D / 16];
                uint32_t top = 0;     // the head's largest magnitude, bf16 bits
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    raw[ks] = row[ks * 4 + t];
                    top = max(top, max(max(raw[ks].x & 0x7fffu, (raw[ks].x >> 16) & 0x7fffu),
                                       max(raw[ks].y & 0x7fffu, (raw[ks].y >> 16) & 0x7fffu)));
                }
                top = max(top, __shfl_xor_sync(kFull, top, 1));
                top = max(top, __shfl_xor_sync(kFull, top, 2));
                // largest magnitude to [2^14, 2^15)
                const int e = top == 0 ? 0 : max(-120, static_cast<int>(top >> 7) - 127 - 14);
                const float down = pow2(-e);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    qf[n][ks][0] = pack_half(__uint_as_float(raw[ks].x << 16) * down, __uint_as_float(raw[ks].x & 0xffff0000u) * down);
                    qf[n][ks][1] = pack_half(__uint_as_float(raw[ks].y << 16) * down, __uint_as_float(raw[ks].y & 0xffff0000u) * down);
                }
                const float c = a.scale * kLog2e * pow2(e);
                // heads 2t and 2t + 1 are rows of lanes 8t and 8t + 4
                qc[n][0] = __shfl_sync(kFull, c, 8 * t);
                qc[n][1] = __shfl_sync(kFull, c, 8 * t + 4);
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        o[n][j][x] = 0.0f;
                m[n][0] = m[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.0f;
            }
        }

        if (d.flags & (kHalf0 | kHalf1)) {
            const float4 sc = sm.scale[warp][stage];
            const uint32_t ks_base = smem_u32(&sm.ring[warp][stage][0][0]);
            const uint32_t vs_base = ks_base + S::kMatrix;
            const int mrow = (lane & 7) + ((lane >> 3) & 1) * 8, mgrp = lane >> 4;   // ldmatrix: this lane's row
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
            const float sk[2] = {checked_scale(sc.x), checked_scale(sc.y)};
            const float sv[2] = {checked_scale(sc.z), checked_scale(sc.w)};
            // approximate to 2^-22: a page's weights are all off by the same factor, less than 2^-21
            const float lsv[2] = {log2_approx(sv[0]), log2_approx(sv[1])};
            const float rsv[2] = {rcp_approx(sv[0]), rcp_approx(sv[1])};
            const bool whole = (d.flags & kWhole) != 0;
            uint32_t pf[NT][2][2];    // weights as the second operand: [tile of 16][keys 0-7, 8-15]
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float mx[2] = {m[n][0], m[n][1]};
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
                    const float c[2] = {qc[n][0] * sk[mt], qc[n][1] * sk[mt]};
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        s[n][mt][x] = fmaf(s[n][mt][x], c[x & 1], lsv[mt]);
                }
                if (!whole) {
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int key = d.key0 + mt * 16 + g + (x >> 1) * 8;
                            if (key < d.lo || key >= d.hi)
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
                const float corr[2] = {exp2_approx(m[n][0] - mx[0]), exp2_approx(m[n][1] - mx[1])};
                const float ref[2] = {mx[0] - kWeightExp, mx[1] - kWeightExp};
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        s[n][mt][x] = exp2_approx(s[n][mt][x] - ref[x & 1]);
                        sum[x & 1] = fmaf(s[n][mt][x], rsv[mt], sum[x & 1]);
                    }
                    pf[n][mt][0] = transpose8x8(pack_half(s[n][mt][0], s[n][mt][1]));
                    pf[n][mt][1] = transpose8x8(pack_half(s[n][mt][2], s[n][mt][3]));
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    l[n][h] = fmaf(l[n][h], corr[h], sum[h]);
                    m[n][h] = mx[h];
                }
                // outputs so far to the new maximum (factors of one change nothing)
                if (!(d.flags & kFirst)) {
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

        if (d.flags & kLast) {
            // this warp's state to its (consumed) stage, then the eight states added in warp order
            float *mine = reinterpret_cast<float *>(&sm.ring[warp][stage][0][0]);
            __syncwarp();   // every lane has read the stage's codes
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x = l[n][h];
                    x += __shfl_xor_sync(kFull, x, 4);
                    x += __shfl_xor_sync(kFull, x, 8);
                    x += __shfl_xor_sync(kFull, x, 16);
                    const int head = n * 8 + 2 * t + h;
                    if (g == 0)
                        sm.ml[warp][head] = make_float2(m[n][h], x);
                    if (head < a.group) {
#pragma unroll
                        for (int j = 0; j < D / 16; ++j)
                            *reinterpret_cast<float2 *>(mine + out_offset<D>(head, 16 * j + 2 * g)) =
                                make_float2(o[n][j][h], o[n][j][2 + h]);
                    }
                }
            }
            __syncthreads();
            constexpr int kPairs = D / 2;
            for (int x = tid; x < a.group * kPairs; x += kThreads) {
                const int head = x / kPairs, dd = (x % kPairs) * 2;
                float mx = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    mx = fmaxf(mx, sm.ml[w][head].x);
                float sum = 0.0f;
                float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 ml = sm.ml[w][head];
                    const float2 v = *reinterpret_cast<const float2 *>(
                        reinterpret_cast<const float *>(&sm.ring[w][stage][0][0]) + out_offset<D>(head, dd));
                    const float f = exp2_approx(ml.x - mx);
                    sum = fmaf(ml.y, f, sum);
                    acc.x = fmaf(v.x, f, acc.x);
                    acc.y = fmaf(v.y, f, acc.y);
                }
                const int64_t row = static_cast<int64_t>(d.b) * a.hq + d.kvh * a.group + head;
                if (d.chunks == 1) {
                    const bool bad = (d.flags & kBad) != 0, empty = d.hi <= d.lo;
                    const float r0 = bad ? NAN : empty ? 0.0f : acc.x / sum, r1 = bad ? NAN : empty ? 0.0f : acc.y / sum;
                    *reinterpret_cast<__nv_bfloat162 *>(a.out + d.b * a.ldo + static_cast<int64_t>(d.kvh * a.group + head) * D + dd) =
                        __floats2bfloat162_rn(r0, r1);
                    if (a.lse && dd == 0)
                        a.lse[row] = bad ? NAN : empty ? -INFINITY : (mx - kWeightExp + log2f(sum)) * kLn2;
                } else {
                    const int64_t at = row * a.chunks + d.chunk;
                    *reinterpret_cast<float2 *>(a.part + at * D + dd) = acc;
                    if (dd == 0)
                        a.part_ml[at] = make_float2(mx, sum);
                }
            }
            __syncthreads();   // the stages are refilled from the next tile on
        }
    }
    bi_kv::launch_dependents();
}

// The chunks of one query head added in ascending order; sequences of one chunk are done already.
// kSlices groups of D threads take consecutive runs of chunks, whose sums are then added in order.
constexpr int kSlices = 4;

template <int D>
__global__ void __launch_bounds__(D * kSlices) paged_merge_kernel(const __grid_constant__ AttnArgs a)
{
    __shared__ float2 ml_s[kMaxChunks];
    __shared__ float acc_s[kSlices][D], sum_s[kSlices];
    const int64_t row = blockIdx.x;
    const int b = static_cast<int>(row / a.hq), h = static_cast<int>(row % a.hq);
    const int tid = threadIdx.x, slice = tid / D, dd = tid % D;
    bi_kv::dependency_wait();
    const Span s = span_of(a.lens[b], a);
    if (s.chunks == 1)
        return;
    if (tid < s.chunks)
        ml_s[tid] = a.part_ml[row * a.chunks + tid];
    __syncthreads();
    float mx = -INFINITY;
    for (int c = 0; c < s.chunks; ++c)
        mx = fmaxf(mx, ml_s[c].x);
    const int per = (s.chunks + kSlices - 1) / kSlices;
    const int lo = slice * per, hi = min(lo + per, s.chunks);
    const float *part = a.part + row * a.chunks * D + dd;
    float sum = 0.0f, acc = 0.0f;
#pragma unroll 8
    for (int c = lo; c < hi; ++c) {
        const float f = exp2_approx(ml_s[c].x - mx);
        sum = fmaf(ml_s[c].y, f, sum);
        acc = fmaf(part[static_cast<int64_t>(c) * D], f, acc);
    }
    acc_s[slice][dd] = acc;
    if (dd == 0)
        sum_s[slice] = sum;
    __syncthreads();
    if (slice == 0) {
        acc = (acc_s[0][dd] + acc_s[1][dd]) + (acc_s[2][dd] + acc_s[3][dd]);
        sum = (sum_s[0] + sum_s[1]) + (sum_s[2] + sum_s[3]);
        a.out[b * a.ldo + static_cast<int64_t>(h) * D + dd] = __float2bfloat16_rn(acc / sum);
        if (a.lse && dd == 0)
            a.lse[row] = (mx - kWeightExp + log2f(sum)) * kLn2;
    }
}

// Chunks a sequence of up to max_len positions can have.
int64_t most_chunks(int64_t max_len)
{
    const int64_t steps = (max_len + kStep - 1) / kStep;
    return steps < 1 ? 1 : steps < kMaxChunks ? steps : kMaxChunks;
}

template <int D, int NT>
bi_status_t run_attention(const AttnArgs &a, int dev, int sms, cudaStream_t stream)
{
    static std::mutex mu;
    static bool set[64] = {};
    {
        std::lock_guard<std::mutex> lock(mu);
        if (!set[dev]) {
            if (cudaFuncSetAttribute(paged_attention_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(sizeof(Shared<D, NT>))) != cudaSuccess) {
                cudaGetLastError();
                return BI_ERR_CUDA;
            }
            set[dev] = true;
        }
    }
    // no more CTAs than there can be items
    const int64_t items = static_cast<int64_t>(a.b) * a.heads * a.chunks;
    const unsigned grid = static_cast<unsigned>(items < sms ? items : sms);
    bi_status_t st = bi_kv::launch(paged_attention_kernel<D, NT>, dim3(grid), dim3(kThreads), sizeof(Shared<D, NT>), stream, 1, a);
    if (st != BI_OK || a.chunks == 1)
        return st;
    return bi_kv::launch(paged_merge_kernel<D>, dim3(static_cast<unsigned>(a.b * a.hq)), dim3(D * kSlices), 0, stream, 1, a);
}

} // namespace

extern "C" {

size_t bi_paged_decode_attention_workspace_bytes(int64_t B, int Hq, int D, int64_t max_len)
{
    if (B < 1 || Hq < 1 || D < 1 || max_len < 1)
        return 0;
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
    if (max_len > (INT64_C(1) << 30) || B * cache->num_heads > (INT64_C(1) << 30) / most_chunks(max_len))
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
    a.k = static_cast<const uint8_t *>(cache->k);
    a.v = static_cast<const uint8_t *>(cache->v);
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.table = block_table;
    a.lens = seq_lens;
    a.out = static_cast<__nv_bfloat16 *>(O);
    a.lse = lse;
    a.ldq = ldq;
    a.ldo = ldo;
    a.ld_table = ld_table;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.window = window;
    a.num_pages = static_cast<int>(cache->num_pages);
    a.max_len = static_cast<int>(max_len);
    a.b = static_cast<int>(B);
    a.hq = Hq;
    a.heads = cache->num_heads;
    a.group = Hq / cache->num_heads;
    a.page_shift = bi_kv::log2_of(cache->page_size);
    a.chunks = static_cast<int>(most_chunks(max_len));
    a.scale = scale;
    a.part = static_cast<float *>(workspace);
    a.part_ml = reinterpret_cast<float2 *>(a.part + B * Hq * a.chunks * cache->head_dim);
    if (cache->head_dim == 128)
        return a.group <= 8 ? run_attention<128, 1>(a, dev, sms, stream) : run_attention<128, 2>(a, dev, sms, stream);
    return a.group <= 8 ? run_attention<64, 1>(a, dev, sms, stream) : run_attention<64, 2>(a, dev, sms, stream);
}

} // extern "C"
