// bulk.cuh -- plain (untiled) bulk copies global -> shared memory.
#pragma once
#include "ptx.cuh"

namespace ccv3d {

// `bytes` bytes from global memory to this CTA's shared memory, completing on
// mbarrier `bar`.  Both addresses and `bytes` are multiples of 16.
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes,
                                         uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar) : "memory");
}

}  // namespace ccv3d
