// bi_paged_attention.cu -- decode attention over the paged 8-bit cache
// (include/bi_paged_attention.h).  One CTA per (sequence, query head) walks the positions in blocks
// of 128 with an online softmax: thread i scores position i of the block, then thread d sums
// dimension d of the values.  All sums are fp32 in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "bi_kv_common.cuh"
#include "bi_paged_attention.h"

namespace {

using bi_kv::kFull;

constexpr int kBlock = 128;
constexpr int kMaxGroup = 16;

struct AttnArgs {
    const __nv_bfloat16 *q;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const int32_t *table, *lens;
    __nv_bfloat16 *out;
    float *lse;
    int64_t ldq, ldo, ld_table, num_pages, page_stride, token_stride, head_stride, max_len, window;
    int hq, heads, group, page_shift;
    float scale;
};

__device__ __forceinline__ float value_of(uint8_t code)
{
    __nv_fp8_e4m3 c;
    c.__x = code;
    return static_cast<float>(c);
}

// NaN unless 2^-64 <= s <= 2^64.
__device__ __forceinline__ float checked_scale(float s)
{
    return s >= 0x1p-64f && s <= 0x1p64f ? s : NAN;
}

template <int D>
__global__ void __launch_bounds__(kBlock) paged_attention_kernel(AttnArgs a)
{
    __shared__ float q_s[D], p_s[kBlock], red[kBlock / 32];
    __shared__ int64_t base_s[kBlock];   // byte of the position's codes, or -1
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x / a.hq;
    const int h = static_cast<int>(blockIdx.x % a.hq), kvh = h / a.group;
    bi_kv::dependency_wait();
    const int64_t len = a.lens[b];
    const bool bad = len < 0 || len > a.max_len;
    const int64_t hi = bad ? 0 : len;
    const int64_t lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
    if (tid < D)
        q_s[tid] = __bfloat162float(a.q[b * a.ldq + static_cast<int64_t>(h) * D + tid]);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, acc = 0.0f;
    for (int64_t j0 = lo & ~static_cast<int64_t>(kBlock - 1); j0 < hi; j0 += kBlock) {
        const int64_t j = j0 + tid;
        float s = -INFINITY, sv = 0.0f;
        int64_t at = -1;
        if (j >= lo && j < hi) {
            const int64_t p = a.table[b * a.ld_table + (j >> a.page_shift)];
            if (p < 0 || p >= a.num_pages) {
                s = NAN;
            } else {
                at = p * a.page_stride + (j & ((1 << a.page_shift) - 1)) * a.token_stride + kvh * a.head_stride;
                const float sk = checked_scale(a.k_scale[p * a.heads + kvh]);
                sv = checked_scale(a.v_scale[p * a.heads + kvh]);
                float dot = 0.0f;
                for (int d = 0; d < D; ++d)
                    dot = fmaf(q_s[d], value_of(a.k[at + d]), dot);
                s = sv == sv ? dot * (sk * a.scale) : NAN;
            }
        }
        float mb = s;
        for (int off = 16; off > 0; off >>= 1)
            mb = fmaxf(mb, __shfl_xor_sync(kFull, mb, off));
        if (lane == 0)
            red[warp] = mb;
        __syncthreads();
        for (int w = 0; w < kBlock / 32; ++w)
            mb = fmaxf(mb, red[w]);
        const float m_new = fmaxf(m, mb);
        const float ref = m_new == -INFINITY ? 0.0f : m_new;
        const float p = expf(s - ref);
        const float corr = expf(m - ref);
        p_s[tid] = at >= 0 || s != s ? p * (s != s ? 1.0f : sv) : 0.0f;
        base_s[tid] = at;
        float ps = p;
        for (int off = 16; off > 0; off >>= 1)
            ps += __shfl_xor_sync(kFull, ps, off);
        __syncthreads();
        if (lane == 0)
            red[warp] = ps;
        __syncthreads();
        l = l * corr;
        for (int w = 0; w < kBlock / 32; ++w)
            l += red[w];
        acc *= corr;
        if (tid < D)
            for (int i = 0; i < kBlock; ++i)
                if (base_s[i] >= 0)
                    acc = fmaf(p_s[i], value_of(a.v[base_s[i] + tid]), acc);
        m = m_new;
        __syncthreads();
    }
    if (bad)
        l = NAN;
    if (tid < D)
        a.out[b * a.ldo + static_cast<int64_t>(h) * D + tid] = __float2bfloat16_rn(l == 0.0f ? 0.0f : acc / l);
    if (tid == 0 && a.lse)
        a.lse[b * a.hq + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

} // namespace

extern "C" {

size_t bi_paged_decode_attention_workspace_bytes(int64_t B, int Hq, int D, int64_t max_len)
{
    (void)B, (void)Hq, (void)D, (void)max_len;
    return 0;
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
        B > INT32_MAX / Hq || ldq > (INT64_C(1) << 40) || ldo > (INT64_C(1) << 40) || ld_table > (INT64_C(1) << 40))
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (B == 0)
        return BI_OK;
    if (!Q || !O || !seq_lens || (max_pages > 0 && !block_table))
        return BI_ERR_INVALID_ARG;
    if (!bi_kv::aligned(Q, 16) || !bi_kv::aligned(O, 16) || ldq % 8 || ldo % 8 || !bi_kv::aligned(block_table, 4) ||
        !bi_kv::aligned(seq_lens, 4) || !bi_kv::aligned(lse, 4))
        return BI_ERR_ALIGNMENT;
    const size_t need = bi_paged_decode_attention_workspace_bytes(B, Hq, cache->head_dim, max_pages * cache->page_size);
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
    a.num_pages = cache->num_pages;
    a.page_stride = cache->page_stride;
    a.token_stride = cache->token_stride;
    a.head_stride = cache->head_stride;
    a.max_len = max_pages * cache->page_size;
    a.window = window;
    a.hq = Hq;
    a.heads = cache->num_heads;
    a.group = Hq / cache->num_heads;
    a.page_shift = bi_kv::log2_of(cache->page_size);
    a.scale = scale;
    const dim3 grid(static_cast<unsigned>(B * Hq));
    return cache->head_dim == 128 ? bi_kv::launch(paged_attention_kernel<128>, grid, dim3(kBlock), 0, stream, 1, a)
                                  : bi_kv::launch(paged_attention_kernel<64>, grid, dim3(kBlock), 0, stream, 1, a);
}

} // extern "C"
