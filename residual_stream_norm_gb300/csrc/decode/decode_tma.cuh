// decode_tma.cuh -- TMA gathers of cache rows by slot.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "beam_tma.cuh"
#include "decode_kernels.h"

namespace beam {

// Maps of the K and V caches as matrices [num_slots, n_kv * 128] for copies of 128 bytes of one
// head's row (64 BF16 or 128 FP8 elements), 128-byte swizzle: of four rows by slot (k, v), and of
// kRun rows of consecutive slots (k_run, v_run).  A warp issues a gather of four rows about every 50
// cycles and a copy of 16 rows every 32 (16 KB tiles out of the L2 cache: 2550 against 1250 cycles), so
// runs of slots, which is what a paged allocator hands out, go as one copy.
constexpr int kRun = 16;

struct CacheMaps {
    CUtensorMap k, v, k_run, v_run;
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Four rows (any slots; one outside the matrix gives zeros) of 128 bytes from column x to dst, dst +
// 128, ...; dst a multiple of 512 in a buffer on a 1024-byte boundary.  512 bytes of transactions.
__device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap *map, int x, int y0, int y1,
                                        int y2, int y3, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y0), "r"(y1), "r"(y2), "r"(y3), "r"(smem_addr(bar))
        : "memory");
}

// kRun rows of consecutive slots from y on, to dst, a multiple of 1024:
// kRun * 128 bytes of transactions.
__device__ __forceinline__ void copy_run(uint32_t dst, const CUtensorMap *map, int x, int y,
                                         uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_tiled()
{
    static EncodeTiled fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiled>(f);
    }();
    return fn;
}

inline cudaError_t make_cache_maps(CacheMaps &maps, const AttnArgs &a)
{
    const EncodeTiled encode = encode_tiled();
    if (!encode)
        return cudaErrorNotSupported;
    const bool fp8 = a.fp8;
    // without a slot no key is seen and nothing is read: any address does for the map
    const void *k = a.num_slots > 0 ? a.k_cache : a.workspace;
    const void *v = a.num_slots > 0 ? a.v_cache : a.workspace;
    const cuuint64_t cols = (cuuint64_t)a.n_kv * 128;
    const cuuint64_t dims[2] = {cols, (cuuint64_t)(a.num_slots > 0 ? a.num_slots : 1)};
    const cuuint64_t strides[1] = {cols * (fp8 ? 1 : 2)};
    const cuuint32_t ones[2] = {1u, 1u};
    CUtensorMap *all[4] = {&maps.k, &maps.v, &maps.k_run, &maps.v_run};
    for (int i = 0; i < 4; ++i) {
        const cuuint32_t box[2] = {fp8 ? 128u : 64u, i < 2 ? 1u : (cuuint32_t)kRun};
        if (encode(all[i],
                   fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                   const_cast<void *>(i & 1 ? v : k), dims, strides, box, ones,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

}  // namespace beam
