// bi_kv_cache.cu -- the paged 8-bit cache's block tables and the write into it
// (include/bi_kv_cache.h).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "bi_kv_cache.h"
#include "bi_kv_common.cuh"

namespace {

using bi_kv::kFull;

// ---------------------------------------------------------------------------------------------
// Block tables and slot maps.  One cluster of one to sixteen CTAs; every CTA reads all lengths and
// scans them by itself (new tokens, new pages, returned pages), so the CTAs share no partial sums,
// and after one cluster barrier -- every input that an output may alias has been read -- each writes
// its share.  Latency bound: a few hundred KB at most.  Threads find the request of their token or
// page by a binary search in the scanned sums, which sit in shared memory, once for four consecutive
// tokens, and again where requests without new tokens lie between them.  (A search for every token kept
// eight SMs busy for 9 us over 51k tokens; steps alone took 90 us with 16 of 8192 requests in use, now 16.)
// ---------------------------------------------------------------------------------------------

constexpr int kTableThreads = 1024;
constexpr int kTableTokens = 4;      // consecutive tokens of a thread
constexpr int kTableSteps = 4;       // requests it steps over from one to the next before it searches again
constexpr int kMaxRequests = 8192;   // four int32 arrays of it in shared memory: 128 KB
constexpr int32_t kMostItems = 1 << 30;   // tokens of a call, pages on the stack

struct TableArgs {
    const int32_t *ctx_lens, *new_lens, *free_count;
    int32_t *free_pages, *block_table, *seq_lens, *token_offsets, *slot_map, *positions, *free_left, *status;
    int64_t free_capacity, ld_table, max_pages, max_tokens;
    int b, page_shift;
};

// Sums that stop at 2^31 - 1 (no valid call reaches it), so that no lengths make them wrap.
struct Sums {
    uint32_t tokens, need, back;
};

__device__ __forceinline__ uint32_t capped(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }
__device__ __forceinline__ Sums operator+(Sums a, Sums b)
{
    return {capped(a.tokens, b.tokens), capped(a.need, b.need), capped(a.back, b.back)};
}

__device__ __forceinline__ Sums shfl_up(Sums s, int off)
{
    return {__shfl_up_sync(kFull, s.tokens, off), __shfl_up_sync(kFull, s.need, off), __shfl_up_sync(kFull, s.back, off)};
}
__device__ __forceinline__ Sums shfl(Sums s, int from)
{
    return {__shfl_sync(kFull, s.tokens, from), __shfl_sync(kFull, s.need, from), __shfl_sync(kFull, s.back, from)};
}
__device__ __forceinline__ Sums warp_scan(Sums s)   // inclusive
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Sums y = shfl_up(s, off);
        if ((threadIdx.x & 31) >= off)
            s = s + y;
    }
    return s;
}

// What request i adds: ctx tokens in the cache, `add` new ones, 2^shift tokens a page.
__device__ __forceinline__ Sums request(int64_t ctx, int64_t add, int shift, int64_t max_pages)
{
    const int64_t page = INT64_C(1) << shift;
    const int64_t have = (ctx + page - 1) >> shift, end = (ctx + (add > 0 ? add : 0) + page - 1) >> shift;
    Sums s = {static_cast<uint32_t>(add > 0 ? add : 0), static_cast<uint32_t>(add >= 0 ? end - have : 0),
              static_cast<uint32_t>(add < 0 ? have : 0)};
    if (end > max_pages)   // does not fit: more tokens than any call may have
        s.tokens = 0x7fffffffu;
    return s;
}

// The last i in [0, n) with sums[i] <= x, for ascending sums with sums[0] = 0 <= x < sums[n]: the
// request that owns item x (requests without items are passed over).
__device__ __forceinline__ int owner(const int32_t *sums, int n, int32_t x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__global__ void __launch_bounds__(kTableThreads, 1) kv_tables_kernel(TableArgs a)
{
    extern __shared__ int32_t table_smem[];
    int32_t *ctx_s = table_smem;                // [b]
    int32_t *tok_s = ctx_s + a.b;               // [b + 1] exclusive sums
    int32_t *need_s = tok_s + a.b + 1;          // [b + 1]
    int32_t *back_s = need_s + a.b + 1;         // [b + 1]
    __shared__ Sums warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int page = 1 << a.page_shift;
    bi_kv::dependency_wait();

    // each thread owns `per` consecutive requests
    const int per = (a.b + kTableThreads - 1) / kTableThreads;
    const int lo = min(tid * per, a.b), hi = min(lo + per, a.b);
    Sums mine = {0, 0, 0};
    bool bad = false;
    for (int i = lo; i < hi; ++i) {
        const int ctx = a.ctx_lens[i], add = a.new_lens[i];
        bad |= ctx < 0 || add < -1;
        ctx_s[i] = ctx;
        tok_s[i] = add;   // the sums take its place below
        mine = mine + request(ctx, add, a.page_shift, a.max_pages);
    }
    const int64_t count = *a.free_count;
    const Sums incl = warp_scan(mine);
    if (lane == 31)
        warp_sums[warp] = incl;
    const bool any_bad = __syncthreads_or(bad);
    const Sums warps = warp_scan(warp_sums[lane]), total = shfl(warps, 31);
    const Sums before = shfl(warps, max(warp - 1, 0));
    int status = BI_OK;
    if (any_bad || count < 0 || count > a.free_capacity)
        status = BI_ERR_INVALID_ARG;
    else if (total.tokens > a.max_tokens || count + total.back > a.free_capacity || total.need > count + total.back)
        status = BI_ERR_UNSUPPORTED_SHAPE;
    if (status == BI_OK) {   // no sum has reached its cap
        Sums run = {incl.tokens - mine.tokens, incl.need - mine.need, incl.back - mine.back};
        if (warp > 0)
            run = run + before;
        for (int i = lo; i < hi; ++i) {
            const Sums r = request(ctx_s[i], tok_s[i], a.page_shift, a.max_pages);
            tok_s[i] = run.tokens;
            need_s[i] = run.need;
            back_s[i] = run.back;
            run = run + r;
        }
        if (tid == 0) {
            tok_s[a.b] = total.tokens;
            need_s[a.b] = total.need;
            back_s[a.b] = total.back;
        }
    }
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kTableThreads + tid;
    const int64_t gsize = static_cast<int64_t>(gridDim.x) * kTableThreads;
    cluster_barrier();   // every CTA's shared memory is ready, and every CTA has read the lengths

    if (status != BI_OK) {
        for (int64_t i = gid; i <= a.b; i += gsize) {
            if (i < a.b)
                a.seq_lens[i] = ctx_s[i];
            a.token_offsets[i] = 0;
        }
        for (int64_t t = gid; t < a.max_tokens; t += gsize) {
            a.slot_map[t] = -1;
            if (a.positions)
                a.positions[t] = -1;
        }
        if (gid == 0) {
            *a.free_left = static_cast<int32_t>(count);
            *a.status = status;
        }
        return;
    }

    const int32_t back = static_cast<int32_t>(total.back), need = static_cast<int32_t>(total.need);
    const int32_t tokens = static_cast<int32_t>(total.tokens);
    if (back > 0) {   // uniform over the cluster
        for (int64_t r = gid; r < back; r += gsize) {
            const int i = owner(back_s, a.b, static_cast<int32_t>(r));
            a.free_pages[count + r] = a.block_table[i * a.ld_table + (r - back_s[i])];
        }
        cluster_barrier();   // the pushed pages can be popped
    }
    const int64_t top = count + back;
    for (int64_t r = gid; r < need; r += gsize) {
        const int i = owner(need_s, a.b, static_cast<int32_t>(r));
        const int64_t have = (static_cast<int64_t>(ctx_s[i]) + page - 1) >> a.page_shift;
        a.block_table[i * a.ld_table + have + (r - need_s[i])] = __ldcg(a.free_pages + (top - 1 - r));
    }
    const bool vec = ((reinterpret_cast<uintptr_t>(a.slot_map) | reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
    for (int64_t t0 = kTableTokens * gid; t0 < a.max_tokens; t0 += kTableTokens * gsize) {
        int32_t pos[kTableTokens], id[kTableTokens], slots[kTableTokens];
        int i = t0 < tokens ? owner(tok_s, a.b, static_cast<int32_t>(t0)) : 0;
#pragma unroll
        for (int j = 0; j < kTableTokens; ++j) {
            const int64_t t = t0 + j;
            pos[j] = -1;
            id[j] = -1;
            if (t < tokens) {
                // a few steps to the request of the next token, then a search, which passes over idle ones
                for (int step = 0; tok_s[i + 1] <= t; ++step) {   // t < tok_s[b]
                    if (step == kTableSteps) {
                        i = owner(tok_s, a.b, static_cast<int32_t>(t));
                        break;
                    }
                    ++i;
                }
                pos[j] = ctx_s[i] + static_cast<int32_t>(t - tok_s[i]);   // below max_pages * page
                const int32_t p = pos[j] >> a.page_shift;
                const int32_t have = static_cast<int32_t>((static_cast<int64_t>(ctx_s[i]) + page - 1) >> a.page_shift);
                // a page of this call is read from the stack, not from the entry another CTA may still write
                const int32_t *from = p < have ? a.block_table + i * a.ld_table + p : a.free_pages + (top - 1 - (need_s[i] + (p - have)));
                id[j] = __ldcg(from);
            }
        }
#pragma unroll
        for (int j = 0; j < kTableTokens; ++j) {
            const int64_t slot = (static_cast<int64_t>(id[j]) << a.page_shift) + (pos[j] & (page - 1));
            slots[j] = id[j] < 0 || slot > INT32_MAX ? -1 : static_cast<int32_t>(slot);
        }
        if (vec && t0 + kTableTokens <= a.max_tokens) {
            *reinterpret_cast<int4 *>(a.slot_map + t0) = make_int4(slots[0], slots[1], slots[2], slots[3]);
            if (a.positions)
                *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int j = 0; j < kTableTokens && t0 + j < a.max_tokens; ++j) {
                a.slot_map[t0 + j] = slots[j];
                if (a.positions)
                    a.positions[t0 + j] = pos[j];
            }
        }
    }
    for (int64_t i = gid; i <= a.b; i += gsize) {
        a.token_offsets[i] = tok_s[i];
        // an ended request that held pages gets 0; one without pages held no tokens
        if (i < a.b)
            a.seq_lens[i] = back_s[i + 1] > back_s[i] ? 0 : ctx_s[i] + (tok_s[i + 1] - tok_s[i]);
    }
    if (gid == 0) {
        *a.free_left = static_cast<int32_t>(top - need);
        *a.status = BI_OK;
    }
}

size_t table_smem_bytes(int64_t b) { return (4 * static_cast<size_t>(b) + 3) * sizeof(int32_t); }

// Once per device: shared memory for the most requests, whatever this call has, since host threads
// that each set their own call's amount would undo one another's; and the largest cluster, 16 CTAs
// where the device can place them, else the portable 8.
bi_status_t prepare_tables(int dev, int *largest)
{
    static std::mutex mu;
    static int most[bi_kv::kMaxDevices] = {};
    std::lock_guard<std::mutex> lock(mu);
    if (!most[dev]) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 16;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kTableThreads);
        cfg.dynamicSmemBytes = table_smem_bytes(kMaxRequests);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaFuncSetAttribute(kv_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(table_smem_bytes(kMaxRequests))) != cudaSuccess ||
            cudaFuncSetAttribute(kv_tables_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&clusters, kv_tables_kernel, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return BI_ERR_CUDA;
        }
        most[dev] = clusters > 0 ? 16 : 8;
    }
    *largest = most[dev];
    return BI_OK;
}

// ---------------------------------------------------------------------------------------------
// The write into the cache.  A run -- rows with consecutive slots of one page -- has at most
// page_size tokens.  A group of warps, one for each 16 tokens of a page (eight for pages of 256), takes
// one head of K or of V and the runs that begin in a block of up to 32 rows: those inside the first 16
// rows together in one warp, and those inside the other 16 (a decode step's are one token each), then
// the remaining ones in turn, a share of the page a warp.  The tokens stay in registers between the
// pass that finds the largest magnitudes and the one that rounds.  Only when a page's exponent grows
// are its earlier codes read and moved.  The warps of a CTA take neighbouring heads, whose rows lie
// side by side.  Memory bound for prompts, latency bound for a decode step.
// ---------------------------------------------------------------------------------------------

constexpr int kAppendWarps = 8;

struct AppendArgs {
    const __nv_bfloat16 *x[2];   // K, V
    int64_t ld[2];
    uint8_t *codes[2];
    float *scale[2];
    const int32_t *slots;
    int64_t num_slots, page_stride, token_stride, head_stride;
    int t, rows, heads, page_shift;
};

// R of include/bi_kv_cache.h on a value already divided by the scale, as the e4m3 byte.
__device__ __forceinline__ uint32_t code_of(float y)
{
    const uint32_t bits = __float_as_uint(y);
    if ((bits & 0x7fffffffu) >= 0x7f800000u)
        return 0x7fu;                            // infinity and NaN: NaN
    // nearest even at 4 significant bits (3 stored ones): add half of the last kept place, ties
    // down when that place is even, and clear what is below
    float r = __uint_as_float((bits + 0x7ffffu + ((bits >> 20) & 1u)) & 0xfff00000u);
    if (fabsf(r) < 0.015625f)                    // below 2^-6: cut to a multiple of 2^-9
        r = truncf(r * 512.0f) * 0.001953125f;
    r = fminf(fmaxf(r, -448.0f), 448.0f);
    // r is an e4m3 value: the conversion is exact
    return static_cast<uint32_t>(__nv_cvt_float_to_fp8(r, __NV_SATFINITE, __NV_E4M3)) |
           ((bits >> 24) & 0x80u);
}

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The smallest e with amax <= 448 * 2^e, in [-64, 64], from amax's bf16 bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ int exponent_of(uint32_t amax_bits)
{
    const int e = static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
    return max(bi_kv::kScaleExpMin, min(bi_kv::kScaleExpMax, e));
}

// Magnitudes of two bf16 at or above this round up to infinity at 4 significant bits, or are not finite.
constexpr uint32_t kHuge = 0x7f78u;

// The magnitude of f * |x| cut to a multiple of 2^-9: (|x| f + 2^14, cut) - 2^14, for 2^-9 is the
// unit in the last place from 2^14 on.  Values of 4 significant bits from 2^-6 on are such multiples
// and stay what they are, so the cut of R needs no case.
__device__ __forceinline__ float cut(float x, float f) { return __fmaf_rz(fabsf(x), f, 16384.0f) - 16384.0f; }

// Two non-negative values as e4m3 bytes: exact for values of R up to 448, saturating, NaN stays.
__device__ __forceinline__ uint32_t bytes_of(float lo, float hi)
{
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
    return y;
}

// R(x * inv) of four bf16 values below kHuge (two words), as four e4m3 bytes.  Rounding to 4
// significant bits works on the bf16 bits of a pair at once (dividing by a power of two changes no
// significant bit); the sign bits are the high bits of the bf16s' high bytes.
__device__ __forceinline__ uint32_t codes_of(uint32_t a, uint32_t b, float inv)
{
    const uint32_t ra = (a + 0x00070007u + ((a >> 4) & 0x00010001u)) & 0xfff0fff0u;
    const uint32_t rb = (b + 0x00070007u + ((b >> 4) & 0x00010001u)) & 0xfff0fff0u;
    const uint32_t lo = bytes_of(cut(__uint_as_float(ra << 16), inv), cut(__uint_as_float(ra & 0xffff0000u), inv));
    const uint32_t hi = bytes_of(cut(__uint_as_float(rb << 16), inv), cut(__uint_as_float(rb & 0xffff0000u), inv));
    return __byte_perm(lo, hi, 0x5410) | (__byte_perm(a, b, 0x7531) & 0x80808080u);
}

// Four e4m3 codes moved to a scale 1 / f times theirs: R(code * f).
__device__ __forceinline__ uint32_t moved(uint32_t codes, float f)
{
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes >> (16 * j))));
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        out[j] = bytes_of(cut(v.x, f), cut(v.y, f));
    }
    const uint32_t r = __byte_perm(out[0], out[1], 0x5410);
    // a NaN keeps no sign, as when it was written
    uint32_t sign = codes & 0x80808080u;
    if (__vcmpeq4(codes & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0)
        sign &= ~__vcmpeq4(codes & 0x7f7f7f7fu, 0x7f7f7f7fu);
    return r | sign;
}

// Largest of two bf16 magnitudes so far and in a word, packed.
__device__ __forceinline__ uint32_t magnitudes(uint32_t best, uint32_t two) { return __vmaxu2(best, two & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t finite_magnitude(uint32_t best, uint32_t two)
{
    const uint32_t lo = two & 0x7fffu, hi = (two >> 16) & 0x7fffu;
    best = lo < 0x7f80u ? max(best, lo) : best;
    return hi < 0x7f80u ? max(best, hi) : best;
}

// One group's warps (G of them, named barrier 1 + group); nothing to wait for in a group of one.
template <int G>
__device__ __forceinline__ void group_sync(int group)
{
    if constexpr (G > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * G) : "memory");
}

// The exponent that a stored scale's bits stand for.
__device__ __forceinline__ int exponent_of_scale(uint32_t bits)
{
    return max(bi_kv::kScaleExpMin, min(bi_kv::kScaleExpMax, static_cast<int>((bits >> 23) & 0xffu) - 127));
}

// The codes of places [begin, end) of a page's head move from exponent `from` to the larger `to`.
template <int D>
__device__ __forceinline__ void move_codes(uint8_t *codes, int64_t token_stride, int begin, int end, int from, int to)
{
    constexpr int kGroups = D / 16, kRows = 32 / kGroups, kMoves = 4;   // loads in flight
    const float f = pow2(max(from - to, -126));
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int base = begin + lane / kGroups; base < end; base += kMoves * kRows) {   // a lane past the end leaves
        uint8_t *at = codes + base * token_stride + lane % kGroups * 16;
        uint4 q[kMoves];
#pragma unroll
        for (int j = 0; j < kMoves; ++j)
            if (base + j * kRows < end)
                q[j] = *reinterpret_cast<const uint4 *>(at + j * kRows * token_stride);
#pragma unroll
        for (int j = 0; j < kMoves; ++j)
            if (base + j * kRows < end)
                *reinterpret_cast<uint4 *>(at + j * kRows * token_stride) =
                    make_uint4(moved(q[j].x, f), moved(q[j].y, f), moved(q[j].z, f), moved(q[j].w, f));
    }
    __syncwarp();
}

__device__ __forceinline__ uint32_t larger_half(uint32_t two) { return max(two & 0xffffu, two >> 16); }
__device__ __forceinline__ uint32_t row_magnitudes(const uint4 &v)
{
    return magnitudes(magnitudes(magnitudes(magnitudes(0u, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint32_t row_finite(const uint4 &v)
{
    return finite_magnitude(finite_magnitude(finite_magnitude(finite_magnitude(0u, v.x), v.y), v.z), v.w);
}
__device__ __forceinline__ uint2 row_codes(const uint4 &v, float inv)
{
    return make_uint2(codes_of(v.x, v.y, inv), codes_of(v.z, v.w, inv));
}

// The codes at `to` of 8 values some of which codes_of does not take (the largest finite ones,
// infinities, NaN), one value at a time: rare, so short rather than fast.
__device__ __forceinline__ void write_huge(uint8_t *to, const uint4 *from, float inv)
{
    const uint4 v = __ldg(from);
    if (larger_half(row_magnitudes(v)) < kHuge)
        return;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
    for (int y = 0; y < 8; ++y) {
        to[y] = static_cast<uint8_t>(code_of(__uint_as_float(w[0] << 16) * inv));
        w[0] = __funnelshift_r(w[0], w[1], 16);
        w[1] = __funnelshift_r(w[1], w[2], 16);
        w[2] = __funnelshift_r(w[2], w[3], 16);
        w[3] >>= 16;
    }
}

// Blocks of an SM: tokens of a warp are held in registers.
__host__ __device__ constexpr int append_blocks(int piece) { return piece == 16 ? 3 : 2; }

// G warps a group, kPiece tokens a warp: G * kPiece = page_size.
template <int D, int G, int kPiece>
__global__ void __launch_bounds__(32 * kAppendWarps, append_blocks(kPiece)) kv_append_kernel(const __grid_constant__ AppendArgs a)
{
    constexpr int kVecs = D / 8;             // 16-byte vectors of a row's head
    constexpr int kTokens = 32 / kVecs;      // tokens one load instruction covers
    constexpr int kLoads = kPiece / kTokens;
    __shared__ uint32_t top_s[2][kAppendWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / G, part = warp % G;
    const int page = 1 << a.page_shift;
    bi_kv::dependency_wait();
    // unit: a block of rows, K or V, a head
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kAppendWarps / G) + group;
    const int h = static_cast<int>(unit % a.heads), kv = static_cast<int>(unit / a.heads % 2);
    const int64_t t0 = unit / a.heads / 2 * a.rows;
    if (t0 >= a.t)
        return;
    const int64_t ld = a.ld[kv];
    const __nv_bfloat16 *x = a.x[kv] + t0 * ld + static_cast<int64_t>(h) * D + lane % kVecs * 8;
    uint8_t *pool = a.codes[kv] + h * a.head_stride;
    float *scales = a.scale[kv] + h;

    // The slots of the block's rows and of a page of rows behind them, all asked for at once.  Bit l of
    // follows[k]: row t0 + 32 k + l continues the run of the row before.
    constexpr int kWords = (G * kPiece + 31) / 32 + 1;
    int mine[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        const int64_t t = t0 + 32 * k + lane;
        mine[k] = t < a.t ? a.slots[t] : -1;
    }
    int before = t0 > 0 ? a.slots[t0 - 1] : -1;
    uint32_t follows[kWords], begins = 0;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        int prev = __shfl_up_sync(kFull, mine[k], 1);
        prev = lane == 0 ? before : prev;
        before = __shfl_sync(kFull, mine[k], 31);
        const bool valid = mine[k] >= 0 && mine[k] < a.num_slots;
        const bool next = valid && (mine[k] & (page - 1)) != 0 && prev == mine[k] - 1;
        follows[k] = __ballot_sync(kFull, next);
        if (k == 0)
            begins = __ballot_sync(kFull, valid && !next);
    }
    const uint32_t block = a.rows == 32 ? kFull : (1u << a.rows) - 1u;   // rows whose runs are this unit's
    if ((begins & block) == 0)
        return;   // the whole group

    // The run of this lane's row: its first row and the row behind its last (33: behind the first 32).
    const bool in_run = ((begins | follows[0]) >> lane) & 1u;
    const uint32_t below = begins & (lane == 31 ? kFull : (2u << lane) - 1u);
    const int start = in_run && below != 0 ? 31 - __clz(below) : -1;
    const uint32_t breaks = lane == 31 ? 0u : ~follows[0] >> (lane + 1);
    const int end = breaks != 0 ? lane + __ffs(breaks) : (follows[1] & 1u) ? 33 : 32;
    const bool ours = start >= 0 && ((block >> start) & 1u);
    const bool inside = ours && end <= start / kPiece * kPiece + kPiece;   // its kPiece rows
    const uint32_t short_rows = __ballot_sync(kFull, inside);
    uint32_t on = __ballot_sync(kFull, ours && lane == start && !inside);   // first rows of the others

#pragma unroll 1
    for (int row0 = 0; row0 < 32; row0 += kPiece) {   // the first warp's work
        const uint32_t here = kPiece == 32 ? short_rows : short_rows >> row0 & ((1u << (kPiece & 31)) - 1u);
        if (part != 0 || here == 0)
            continue;
        uint4 v[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            const int tok = j * kTokens + lane / kVecs;
            v[j] = make_uint4(0, 0, 0, 0);
            if ((here >> tok) & 1u)
                v[j] = __ldg(reinterpret_cast<const uint4 *>(x + (row0 + tok) * ld));
        }
        const bool used = lane >= row0 && lane < row0 + kPiece && ((short_rows >> lane) & 1u), leads = used && lane == start;
        const int slot = mine[0], off = slot & (page - 1);
        float *scale = scales + static_cast<int64_t>(slot >> a.page_shift) * a.heads;
        const uint32_t old_scale = leads && off != 0 ? __float_as_uint(*scale) : 0u;
        uint32_t top = 0;   // of this lane's token
        bool huge = false;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if ((here >> (j * kTokens)) & ((1u << kTokens) - 1u)) {
                uint32_t y = larger_half(row_magnitudes(v[j]));
                if (y >= kHuge) {
                    huge = true;
                    y = row_finite(v[j]);
                }
#pragma unroll
                for (int m = kVecs / 2; m > 0; m >>= 1)
                    y = max(y, __shfl_xor_sync(kFull, y, m));
                y = __shfl_sync(kFull, y, lane % kTokens * kVecs);
                top = (lane - row0) / kTokens == j ? y : top;
            }
        // the run's largest, at its last row and from there to all of it
#pragma unroll
        for (int m = 1; m < kPiece; m <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, top, m);
            if (used && lane - m >= start)
                top = max(top, y);
        }
        top = __shfl_sync(kFull, top, used ? end - 1 : lane);
        const int run_off = __shfl_sync(kFull, off, used ? start : lane);
        const int old = exponent_of_scale(__shfl_sync(kFull, old_scale, used ? start : lane));
        int e = exponent_of(top);
        const bool grows = run_off != 0 && e > old;
        if (run_off != 0 && !grows)
            e = old;
        for (uint32_t move = __ballot_sync(kFull, leads && grows); move != 0; move &= move - 1) {
            const int l = __ffs(move) - 1;
            const int64_t id = __shfl_sync(kFull, slot, l) >> a.page_shift;
            move_codes<D>(pool + id * a.page_stride, a.token_stride, 0, __shfl_sync(kFull, off, l), __shfl_sync(kFull, old, l),
                          __shfl_sync(kFull, e, l));
        }
        if (leads)
            *scale = pow2(e);
        auto place = [&](int tok, float *inv) {   // of token tok's 8 codes
            const int to = __shfl_sync(kFull, slot, row0 + tok);
            *inv = pow2(-__shfl_sync(kFull, e, row0 + tok));
            return pool + static_cast<int64_t>(to >> a.page_shift) * a.page_stride + (to & (page - 1)) * a.token_stride +
                   lane % kVecs * 8;
        };
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if ((here >> (j * kTokens)) & ((1u << kTokens) - 1u)) {
                const int tok = j * kTokens + lane / kVecs;
                float inv;
                uint8_t *to = place(tok, &inv);
                if ((here >> tok) & 1u)
                    *reinterpret_cast<uint2 *>(to) = row_codes(v[j], inv);
            }
        if (__any_sync(kFull, huge))
#pragma unroll 1
            for (int j = 0; j < kLoads; ++j) {
                const int tok = j * kTokens + lane / kVecs;
                float inv;
                uint8_t *to = place(tok, &inv);
                if ((here >> tok) & 1u)
                    write_huge(to, reinterpret_cast<const uint4 *>(x + (row0 + tok) * ld), inv);
            }
    }

    int turn = 0;
#pragma unroll 1
    for (; on != 0; on &= on - 1, turn ^= 1) {
        const int i = __ffs(on) - 1;   // the run's first row
        int n = 32 * kWords - i;       // up to the first row behind it that does not follow
#pragma unroll
        for (int k = kWords - 1; k >= 0; --k) {
            const uint32_t stop = k == 0 ? ~follows[0] & (i == 31 ? 0u : 0xfffffffeu << i) : ~follows[k];
            if (stop != 0)
                n = 32 * k + __ffs(stop) - 1 - i;
        }
        const int slot = __shfl_sync(kFull, mine[0], i), off = slot & (page - 1);
        const int64_t p = slot >> a.page_shift;
        uint8_t *codes = pool + p * a.page_stride;
        float *scale = scales + p * a.heads;
        // this warp's tokens of the run
        const int begin = part * kPiece, count = min(n - begin, kPiece);
        const __nv_bfloat16 *from = x + (i + begin + lane / kVecs) * ld;
        uint4 v[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            if (j * kTokens + lane / kVecs < count)
                v[j] = __ldg(reinterpret_cast<const uint4 *>(from + j * kTokens * ld));
        }
        const uint32_t old_scale = off != 0 ? __float_as_uint(*scale) : 0u;
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            best = __vmaxu2(best, row_magnitudes(v[j]));
        uint32_t top = larger_half(best);
        const bool huge = top >= kHuge;
        if (huge) {
            top = 0;
#pragma unroll
            for (int j = 0; j < kLoads; ++j)
                top = max(top, row_finite(v[j]));
        }
        top = __reduce_max_sync(kFull, top);
        if constexpr (G > 1) {
            if (lane == 0)
                top_s[turn][warp] = top;
            group_sync<G>(group);   // also: every warp has read the scale
#pragma unroll
            for (int w = 0; w < G; ++w)
                top = max(top, top_s[turn][group * G + w]);
        }
        int e = exponent_of(top);
        if (off != 0) {
            const int old = exponent_of_scale(old_scale);
            if (e > old)
                move_codes<D>(codes, a.token_stride, begin, min(off, begin + kPiece), old, e);
            else
                e = old;
        }
        if (part == 0 && lane == 0)
            *scale = pow2(e);
        const float inv = pow2(-e);
        uint8_t *to = codes + (off + begin + lane / kVecs) * a.token_stride + lane % kVecs * 8;
#pragma unroll
        for (int j = 0; j < kLoads; ++j)
            if (j * kTokens + lane / kVecs < count)
                *reinterpret_cast<uint2 *>(to + j * kTokens * a.token_stride) = row_codes(v[j], inv);
        if (huge)
#pragma unroll 1
            for (int j = 0; j < kLoads; ++j)
                if (j * kTokens + lane / kVecs < count)
                    write_huge(to + j * kTokens * a.token_stride, reinterpret_cast<const uint4 *>(from + j * kTokens * ld), inv);
    }
}

template <int D, int G, int kPiece>
bi_status_t run_append(const AppendArgs &a, int64_t blocks_of_rows, cudaStream_t stream)
{
    const int64_t units = blocks_of_rows * 2 * a.heads, per = kAppendWarps / G;
    return bi_kv::launch(kv_append_kernel<D, G, kPiece>, dim3(static_cast<unsigned>((units + per - 1) / per)),
                         dim3(32 * kAppendWarps), 0, stream, 1, a);
}

template <int D>
bi_status_t run_append(const AppendArgs &a, int page_size, int64_t blocks_of_rows, cudaStream_t stream)
{
    switch (page_size) {
    case 16: return run_append<D, 1, 16>(a, blocks_of_rows, stream);
    case 32: return run_append<D, 2, 16>(a, blocks_of_rows, stream);
    case 64: return run_append<D, 4, 16>(a, blocks_of_rows, stream);
    case 128: return run_append<D, 8, 16>(a, blocks_of_rows, stream);
    default: return run_append<D, 8, 32>(a, blocks_of_rows, stream);
    }
}

} // namespace

extern "C" {

bi_status_t bi_kv_block_tables(const int32_t *ctx_lens, const int32_t *new_lens, int64_t B,
                               int page_size, int32_t *free_pages, int64_t free_capacity,
                               const int32_t *free_count, int32_t *block_table, int64_t ld_table,
                               int64_t max_pages, int32_t *seq_lens, int32_t *token_offsets,
                               int32_t *slot_map, int32_t *positions, int64_t max_tokens,
                               int32_t *free_left, int32_t *status, cudaStream_t stream)
{
    if (B < 0 || free_capacity < 0 || max_pages < 0 || ld_table < max_pages || max_tokens < 0)
        return BI_ERR_INVALID_ARG;
    if (!bi_kv::valid_page_size(page_size) || B > kMaxRequests || max_pages > INT32_MAX / page_size ||
        max_tokens > kMostItems || free_capacity > kMostItems || ld_table > (INT64_C(1) << 40))
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (!free_count || !free_left || !status || !token_offsets || (B > 0 && (!ctx_lens || !new_lens || !seq_lens)) ||
        (B > 0 && max_pages > 0 && !block_table) || (free_capacity > 0 && !free_pages) || (max_tokens > 0 && !slot_map))
        return BI_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(ctx_lens), static_cast<const void *>(new_lens),
                          static_cast<const void *>(free_pages), static_cast<const void *>(free_count),
                          static_cast<const void *>(block_table), static_cast<const void *>(seq_lens),
                          static_cast<const void *>(token_offsets), static_cast<const void *>(slot_map),
                          static_cast<const void *>(positions), static_cast<const void *>(free_left),
                          static_cast<const void *>(status)})
        if (!bi_kv::aligned(p, 4))
            return BI_ERR_ALIGNMENT;
    int dev = 0, sms = 0;
    bi_status_t st = bi_kv::current_device(&dev, &sms);
    if (st != BI_OK)
        return st;
    TableArgs a = {};
    a.ctx_lens = ctx_lens;
    a.new_lens = new_lens;
    a.free_count = free_count;
    a.free_pages = free_pages;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.token_offsets = token_offsets;
    a.slot_map = slot_map;
    a.positions = positions;
    a.free_left = free_left;
    a.status = status;
    a.free_capacity = free_capacity;
    a.ld_table = ld_table;
    a.max_pages = max_pages;
    a.max_tokens = max_tokens;
    a.b = static_cast<int>(B);
    a.page_shift = bi_kv::log2_of(page_size);
    int largest = 0;
    st = prepare_tables(dev, &largest);
    if (st != BI_OK)
        return st;
    const size_t smem = table_smem_bytes(B);
    // CTAs: one for every 4096 tokens, up to the largest cluster.  51k tokens of 1000 requests took
    // 10.3 us with 8 CTAs and 8.0 with 16, 69k of 33 prompts 8.1 and 6.3 (8.4 and 6.6 since threads search
    // again).  Eight tokens a thread: 9.3.
    int cluster = 1;
    while (cluster < largest && static_cast<int64_t>(cluster) * kTableThreads * kTableTokens < (max_tokens > B ? max_tokens : B))
        cluster *= 2;
    return bi_kv::launch(kv_tables_kernel, dim3(cluster), dim3(kTableThreads), smem, stream, cluster, a);
}

bi_status_t bi_kv_append_e4m3(const bi_kv_cache_t *cache, const void *K, int64_t ldk, const void *V,
                              int64_t ldv, const int32_t *slot_map, int64_t T, cudaStream_t stream)
{
    bi_status_t st = bi_kv::check_cache(cache);
    if (st != BI_OK)
        return st;
    const int64_t row = static_cast<int64_t>(cache->num_heads) * cache->head_dim;
    if (T < 0 || ldk < row || ldv < row)
        return BI_ERR_INVALID_ARG;
    if (T == 0)
        return BI_OK;
    if (!K || !V || !slot_map)
        return BI_ERR_INVALID_ARG;
    if (!bi_kv::aligned(K, 16) || !bi_kv::aligned(V, 16) || ldk % 8 || ldv % 8 || !bi_kv::aligned(slot_map, 4))
        return BI_ERR_ALIGNMENT;
    if (T > INT32_MAX || ldk > (INT64_C(1) << 30) || ldv > (INT64_C(1) << 30))
        return BI_ERR_UNSUPPORTED_SHAPE;
    int dev = 0, sms = 0;
    if ((st = bi_kv::current_device(&dev, &sms)) != BI_OK)
        return st;
    AppendArgs a = {};
    a.x[0] = static_cast<const __nv_bfloat16 *>(K);
    a.x[1] = static_cast<const __nv_bfloat16 *>(V);
    a.ld[0] = ldk;
    a.ld[1] = ldv;
    a.codes[0] = static_cast<uint8_t *>(cache->k);
    a.codes[1] = static_cast<uint8_t *>(cache->v);
    a.scale[0] = cache->k_scale;
    a.scale[1] = cache->v_scale;
    a.slots = slot_map;
    a.num_slots = cache->num_pages * cache->page_size;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.t = static_cast<int>(T);
    a.heads = cache->num_heads;
    a.page_shift = bi_kv::log2_of(cache->page_size);
    // Rows per block: one, so that the runs of a decode step are written side by side, while all warps
    // are resident at once (64 tokens, 8 heads, pages of 64: two rows 3.1 us, one 4.9 us; 160 tokens,
    // pages of 256: sixteen rows 5.6 us, eight 7.7 us); at most a warp's 32.
    const int64_t groups = 2 * static_cast<int64_t>(cache->num_heads);
    const int warps = cache->page_size == 256 ? 8 : cache->page_size / 16;
    const int resident = kAppendWarps * append_blocks(cache->page_size == 256 ? 32 : 16);
    a.rows = 1;
    while (a.rows < 32 && (T + a.rows - 1) / a.rows * groups * warps > resident * static_cast<int64_t>(sms))
        a.rows *= 2;
    const int64_t blocks = (T + a.rows - 1) / a.rows;
    if (blocks > INT32_MAX / groups)
        return BI_ERR_UNSUPPORTED_SHAPE;
    return cache->head_dim == 128 ? run_append<128>(a, cache->page_size, blocks, stream)
                                  : run_append<64>(a, cache->page_size, blocks, stream);
}

} // extern "C"
