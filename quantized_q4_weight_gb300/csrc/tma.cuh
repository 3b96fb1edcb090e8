// tma.cuh -- tiled copies by tensor maps, for the kernels that read a paged cache
// by them (attn_tc.cu, kv8_attn.cuh).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "qgemv_internal.cuh"

namespace qg {

// A box of the 4-D tensor at (x, row, head, page) into shared memory, counted on `bar`.
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap *map, int x, int row, int head, int page,
                                          uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(row), "r"(head), "r"(page), "r"(smem_addr(bar))
        : "memory");
}

// The driver's encoder of tensor maps, looked up once.
inline PFN_cuTensorMapEncodeTiled_v12000 map_encoder()
{
    static std::atomic<void *> fn{nullptr};
    void *f = fn.load(std::memory_order_acquire);
    if (!f) {
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        fn.store(f, std::memory_order_release);
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
}

}  // namespace qg
