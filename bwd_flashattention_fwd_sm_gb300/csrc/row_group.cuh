// Groups of threads that share a row, several of them in a block.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gbattn {

constexpr int kMaxStages = 8;  // of a group's ring

// Lets a kernel take `smem` bytes of dynamic shared memory.  Always the same limit, because calls from two
// threads may set it in turn before either launches.
template <class K>
cudaError_t allow_shared(K kernel, size_t smem) {
  if (smem <= 32 * 1024) return cudaSuccess;  // 48 KB, its static shared memory included, need no leave
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
}

// Whether x holds for any of a group's kRow threads; a barrier of the group.
template <int kRow, int kGroups>
__device__ __forceinline__ bool group_any(int group, bool x) {
  if constexpr (kRow == 32) {
    return __any_sync(0xffffffffu, x);
  } else if constexpr (kGroups == 1) {
    return __syncthreads_or(x);
  } else {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(1 + group), "n"(kRow)
        : "memory");
    return r != 0;
  }
}

}  // namespace gbattn
