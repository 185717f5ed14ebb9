// bi_kv_cache.cu -- the paged 8-bit cache's block tables and the write into it
// (include/bi_kv_cache.h).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bi_kv_cache.h"
#include "bi_kv_common.cuh"

namespace {

using bi_kv::kFull;

// ---------------------------------------------------------------------------------------------
// Block tables and slot maps.  One cluster; every CTA reads all lengths and scans them by itself
// (new tokens, new pages, returned pages), so the CTAs share no partial sums, and after one
// cluster barrier -- every input that an output may alias has been read -- each writes its share.
// Latency bound: a few hundred KB at most.  Threads find the request of their token or page by a
// binary search in the scanned sums, which sit in shared memory.
// ---------------------------------------------------------------------------------------------

constexpr int kTableThreads = 1024;
constexpr int kTableCluster = 8;
constexpr int kMaxRequests = 8192;   // four int32 arrays of it in shared memory: 128 KB

struct TableArgs {
    const int32_t *ctx_lens, *new_lens, *free_count;
    int32_t *free_pages, *block_table, *seq_lens, *token_offsets, *slot_map, *positions, *free_left, *status;
    int64_t free_capacity, ld_table, max_pages, max_tokens;
    int b, page_shift;
};

struct Sums {
    int64_t tokens, need, back;
};

__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.tokens + b.tokens, a.need + b.need, a.back + b.back}; }

__device__ __forceinline__ Sums shfl_up(Sums s, int off)
{
    return {__shfl_up_sync(kFull, s.tokens, off), __shfl_up_sync(kFull, s.need, off), __shfl_up_sync(kFull, s.back, off)};
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
    bool bad = false, wide = false;
    for (int i = lo; i < hi; ++i) {
        const int64_t ctx = a.ctx_lens[i], add = a.new_lens[i];
        bad |= ctx < 0 || add < -1;
        const int64_t have = (ctx + page - 1) >> a.page_shift;
        const int64_t end = (ctx + (add > 0 ? add : 0) + page - 1) >> a.page_shift;
        wide |= end > a.max_pages;
        ctx_s[i] = static_cast<int32_t>(ctx);
        mine = mine + Sums{add > 0 ? add : 0, add >= 0 ? end - have : 0, add < 0 ? have : 0};
    }
    Sums incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Sums y = shfl_up(incl, off);
        if (lane >= off)
            incl = incl + y;
    }
    if (lane == 31)
        warp_sums[warp] = incl;
    const bool any_bad = __syncthreads_or(bad);
    const bool any_wide = __syncthreads_or(wide);
    Sums before = {0, 0, 0}, total = {0, 0, 0};
    for (int w = 0; w < kTableThreads / 32; ++w) {
        if (w == warp)
            before = total;
        total = total + warp_sums[w];
    }
    const int64_t count = *a.free_count;
    int status = BI_OK;
    if (any_bad || count < 0 || count > a.free_capacity)
        status = BI_ERR_INVALID_ARG;
    else if (any_wide || total.tokens > a.max_tokens || count + total.back > a.free_capacity ||
             total.need > count + total.back)
        status = BI_ERR_UNSUPPORTED_SHAPE;
    if (status == BI_OK) {   // every sum is below 2^31
        Sums run = {before.tokens + incl.tokens - mine.tokens, before.need + incl.need - mine.need,
                    before.back + incl.back - mine.back};
        for (int i = lo; i < hi; ++i) {
            const int64_t ctx = ctx_s[i], add = a.new_lens[i];
            const int64_t have = (ctx + page - 1) >> a.page_shift;
            tok_s[i] = static_cast<int32_t>(run.tokens);
            need_s[i] = static_cast<int32_t>(run.need);
            back_s[i] = static_cast<int32_t>(run.back);
            run.tokens += add > 0 ? add : 0;
            run.need += add >= 0 ? ((ctx + add + page - 1) >> a.page_shift) - have : 0;
            run.back += add < 0 ? have : 0;
        }
        if (tid == 0) {
            tok_s[a.b] = static_cast<int32_t>(total.tokens);
            need_s[a.b] = static_cast<int32_t>(total.need);
            back_s[a.b] = static_cast<int32_t>(total.back);
        }
    }
    // whether request i has ended, before seq_lens (which may be ctx_lens) is written
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
    for (int64_t t = gid; t < a.max_tokens; t += gsize) {
        int64_t slot = -1, pos = -1;
        if (t < tokens) {
            const int i = owner(tok_s, a.b, static_cast<int32_t>(t));
            pos = static_cast<int64_t>(ctx_s[i]) + (t - tok_s[i]);
            const int64_t p = pos >> a.page_shift;
            const int64_t have = (static_cast<int64_t>(ctx_s[i]) + page - 1) >> a.page_shift;
            // a page of this call is read from the stack, not from the entry another CTA may still write
            const int64_t id = p < have ? a.block_table[i * a.ld_table + p]
                                        : __ldcg(a.free_pages + (top - 1 - (need_s[i] + (p - have))));
            slot = (id << a.page_shift) + (pos & (page - 1));
            if (id < 0 || slot > INT32_MAX)
                slot = -1;
        }
        a.slot_map[t] = static_cast<int32_t>(slot);
        if (a.positions)
            a.positions[t] = static_cast<int32_t>(pos);
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

// ---------------------------------------------------------------------------------------------
// The write into the cache.  A run -- rows with consecutive slots of one page -- belongs to the
// CTA that owns its first row; it takes one head of K or of V.  The new exponent is the maximum of
// the page's old one and the run's, so one pass over the run finds it and a second one (from L1)
// rounds and stores; only when the exponent grows are the page's earlier codes read and moved.
// Memory bound for prompts, latency bound for a decode step.
// ---------------------------------------------------------------------------------------------

constexpr int kAppendThreads = 256;

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
        return 0x7fu | ((bits >> 24) & 0x80u);   // infinity and NaN: NaN
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

__device__ __forceinline__ uint32_t amax2(uint32_t best, uint32_t pair)
{
    const uint32_t lo = pair & 0x7fffu, hi = (pair >> 16) & 0x7fffu;
    best = lo < 0x7f80u ? max(best, lo) : best;
    return hi < 0x7f80u ? max(best, hi) : best;
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(AppendArgs a)
{
    constexpr int kVecs = D / 8;   // 16-byte vectors of a row's head
    __shared__ uint32_t red[kAppendThreads / 32];
    __shared__ int run_end;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int h = blockIdx.y, kv = blockIdx.z;
    const int page = 1 << a.page_shift;
    bi_kv::dependency_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * a.rows;
    const int64_t last = min(first + a.rows, static_cast<int64_t>(a.t));
    for (int64_t t = first; t < last; ++t) {   // uniform over the CTA
        const int64_t slot = a.slots[t];
        if (slot < 0 || slot >= a.num_slots)
            continue;
        const int off = static_cast<int>(slot & (page - 1));
        if (off != 0 && t > 0 && a.slots[t - 1] == slot - 1)
            continue;   // inside a run
        // the run's length: rows t + i with slot + i, up to the page's end
        if (tid == 0)
            run_end = static_cast<int>(min(static_cast<int64_t>(page - off), a.t - t));
        __syncthreads();
        if (tid < page - off && t + tid < a.t && a.slots[t + tid] != slot + tid)
            atomicMin(&run_end, tid);
        __syncthreads();
        const int n = run_end;
        const __nv_bfloat16 *x = a.x[kv] + t * a.ld[kv] + static_cast<int64_t>(h) * D;
        uint32_t amax = 0;
        for (int i = tid; i < n * kVecs; i += kAppendThreads) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(x + (i / kVecs) * a.ld[kv]) + i % kVecs);
            amax = amax2(amax2(amax2(amax2(amax, v.x), v.y), v.z), v.w);
        }
        amax = __reduce_max_sync(kFull, amax);
        if (lane == 0)
            red[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kAppendThreads / 32; ++w)
            amax = max(amax, red[w]);
        const int64_t p = slot >> a.page_shift;
        float *scale = a.scale[kv] + p * a.heads + h;
        uint8_t *codes = a.codes[kv] + p * a.page_stride + h * a.head_stride;
        int e = exponent_of(amax);
        if (off != 0) {
            int old = static_cast<int>((__float_as_uint(*scale) >> 23) & 0xffu) - 127;
            old = max(bi_kv::kScaleExpMin, min(bi_kv::kScaleExpMax, old));
            if (e > old) {   // the earlier codes move to the new scale
                const float f = pow2(max(old - e, -126));
                for (int i = tid; i < off * (D / 16); i += kAppendThreads) {
                    uint4 *at = reinterpret_cast<uint4 *>(codes + (i / (D / 16)) * a.token_stride) + i % (D / 16);
                    uint4 v = *at;
                    uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t out = 0;
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            __nv_fp8_e4m3 c;
                            c.__x = static_cast<uint8_t>(w[j] >> (8 * b));
                            out |= code_of(static_cast<float>(c) * f) << (8 * b);
                        }
                        w[j] = out;
                    }
                    *at = v;
                }
            } else {
                e = old;
            }
        }
        __syncthreads();   // everyone has read the scale
        if (tid == 0)
            *scale = pow2(e);
        const float inv = pow2(-e);
        for (int i = tid; i < n * kVecs; i += kAppendThreads) {
            const int row = i / kVecs, vec = i % kVecs;
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(x + row * a.ld[kv]) + vec);
            const uint32_t in[4] = {v.x, v.y, v.z, v.w};
            uint32_t out[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = code_of(__uint_as_float(in[j] << 16) * inv);
                const uint32_t hi = code_of(__uint_as_float(in[j] & 0xffff0000u) * inv);
                out[j >> 1] |= (lo | (hi << 8)) << (16 * (j & 1));
            }
            *reinterpret_cast<uint2 *>(codes + (off + row) * a.token_stride + vec * 8) = make_uint2(out[0], out[1]);
        }
        __syncthreads();   // the shared words are free for the next run
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
        max_tokens > INT32_MAX || free_capacity > INT32_MAX || ld_table > (INT64_C(1) << 40))
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
    const size_t smem = (4 * static_cast<size_t>(B) + 3) * sizeof(int32_t);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kv_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess) {
        cudaGetLastError();
        return BI_ERR_CUDA;
    }
    return bi_kv::launch(kv_tables_kernel, dim3(kTableCluster), dim3(kTableThreads), smem, stream, kTableCluster, a);
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
    // rows per CTA: 1 while that gives no more than 16 CTAs per SM, at most 32
    const int64_t per_row = 2 * static_cast<int64_t>(cache->num_heads);
    a.rows = 1;
    while (a.rows < 32 && (T + a.rows - 1) / a.rows * per_row > 16 * static_cast<int64_t>(sms))
        a.rows *= 2;
    const dim3 grid(static_cast<unsigned>((T + a.rows - 1) / a.rows), cache->num_heads, 2);
    return cache->head_dim == 128
               ? bi_kv::launch(kv_append_kernel<128>, grid, dim3(kAppendThreads), 0, stream, 1, a)
               : bi_kv::launch(kv_append_kernel<64>, grid, dim3(kAppendThreads), 0, stream, 1, a);
}

} // extern "C"
