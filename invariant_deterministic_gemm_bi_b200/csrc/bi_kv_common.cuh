// bi_kv_common.cuh -- what the paged cache's host and device code share: the checks of a cache
// handle, the device probe, launches as programmatic dependents, and the limits of a scale.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "bi_kv_cache.h"

namespace bi_kv {

constexpr int kScaleExpMin = -64;   // exponents of a page's scale
constexpr int kScaleExpMax = 64;
constexpr unsigned kFull = 0xffffffffu;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline bool valid_page_size(int ps) { return ps == 16 || ps == 32 || ps == 64 || ps == 128 || ps == 256; }

inline int log2_of(int power_of_two)
{
    int s = 0;
    while ((1 << s) < power_of_two)
        ++s;
    return s;
}

// The cache handle's own checks, host arithmetic only.
inline bi_status_t check_cache(const bi_kv_cache_t *c)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || c->num_pages < 1 || c->num_heads < 1)
        return BI_ERR_INVALID_ARG;
    if (!valid_page_size(c->page_size) || (c->head_dim != 64 && c->head_dim != 128) ||
        c->num_pages > INT32_MAX / c->page_size || c->num_heads > 65535)
        return BI_ERR_UNSUPPORTED_SHAPE;
    const int64_t d = c->head_dim, big = (INT64_C(1) << 40) - 16;
    if (c->token_stride < d || c->head_stride < d)
        return BI_ERR_INVALID_ARG;
    if (c->token_stride > big || c->head_stride > big || c->page_stride > big)
        return BI_ERR_UNSUPPORTED_SHAPE;
    if (c->page_stride < (c->page_size - 1) * c->token_stride + (c->num_heads - 1) * c->head_stride + d)
        return BI_ERR_INVALID_ARG;
    // a token's heads beside one another, or a head's tokens: anything else overlaps
    if (c->num_heads > 1 && c->token_stride < (c->num_heads - 1) * c->head_stride + d &&
        c->head_stride < (c->page_size - 1) * c->token_stride + d)
        return BI_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
        c->token_stride % 16 || c->head_stride % 16 || c->page_stride % 16)
        return BI_ERR_ALIGNMENT;
    return BI_OK;
}

constexpr int kMaxDevices = 64;

// The current device and its SM count.  The properties are read once per device.
inline bi_status_t current_device(int *dev_out, int *num_sms)
{
    struct Info {
        bool probed, ok;
        int sms;
    };
    static std::mutex mu;
    static Info info[kMaxDevices] = {};
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver ? BI_ERR_NO_DEVICE : BI_ERR_CUDA;
    }
    std::lock_guard<std::mutex> lock(mu);
    Info &d = info[dev];
    if (!d.probed) {
        int count = 0, major = 0, sms = 0;
        if (cudaGetDeviceCount(&count) != cudaSuccess || count <= 0) {
            cudaGetLastError();
            return BI_ERR_NO_DEVICE;
        }
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
            cudaGetLastError();
            return BI_ERR_CUDA;
        }
        d.ok = major == 10;
        d.sms = sms;
        d.probed = true;
    }
    if (!d.ok)
        return BI_ERR_NO_DEVICE;
    *dev_out = dev;
    *num_sms = d.sms;
    return BI_OK;
}

// The tensor map of one pool, [page][head][position][dimension], whose boxes are 16 positions (pages
// of 16) or 32 of one page and head, in the swizzle that spreads rows of 64 or 128 bytes over the banks.
inline bi_status_t page_map(CUtensorMap *map, const bi_kv_cache_t *c, void *pool)
{
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                               const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<Encode>(fn) : nullptr;
    }();
    if (!encode)
        return BI_ERR_CUDA;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->head_dim), static_cast<cuuint64_t>(c->page_size),
                                static_cast<cuuint64_t>(c->num_heads), static_cast<cuuint64_t>(c->num_pages)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c->token_stride), static_cast<cuuint64_t>(c->head_stride),
                                   static_cast<cuuint64_t>(c->page_stride)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(c->head_dim), c->page_size == 16 ? 16u : 32u, 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pool, dims, strides, box, ones,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              c->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? BI_OK : BI_ERR_CUDA;
}

// Launch as a programmatic dependent of the previous kernel in the stream: the grid may start
// while that kernel finishes and calls dependency_wait() before it touches global memory.
template <typename... Params, typename... Args>
bi_status_t launch(void (*fn)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                   int cluster, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, fn, args...) != cudaSuccess) {
        cudaGetLastError();
        return BI_ERR_CUDA;
    }
    return BI_OK;
}

__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

} // namespace bi_kv
