// Groups of threads that share a row, several of them in a block; blocks of a cluster that do.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ptx.cuh"

namespace gbattn {

constexpr int kMaxStages = 8;  // of a group's ring

// Stages of a ring whose stage takes `stage_bytes`: an SM's shared memory over its blocks, less what they hold beside
// the ring, over a block's groups.
__host__ __device__ constexpr int ring_stages(int blocks, int groups, int stage_bytes) {
  const int n = (224 * 1024 / blocks - 2048) / groups / stage_bytes;
  return n < kMaxStages ? n : kMaxStages;
}

// Lets a kernel take `smem` bytes of dynamic shared memory.  Always the same limit, because calls from two
// threads may set it in turn before either launches.
template <class K>
cudaError_t allow_shared(K kernel, size_t smem) {
  if (smem <= 32 * 1024) return cudaSuccess;  // 48 KB, its static shared memory included, need no leave
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
}

// Whether x holds for any of a group's kRow threads; a barrier of the group, which orders their memory too.
template <int kRow, int kGroups>
__device__ __forceinline__ bool group_any(int group, bool x) {
  if constexpr (kRow == 32) {
    __syncwarp();  // a vote orders no memory
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

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// x to the place of `here`, and 4 bytes to the count of the barrier at the place of `bar`, in the
// block `rank` of the cluster.  (Not a cluster barrier: that would wait for the stores of dr and dx.)
__device__ __forceinline__ void cluster_send(void* here, uint64_t* bar, uint32_t rank, float x) {
  uint32_t to, count;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(ptx::smem_u32(here)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(count) : "r"(ptx::smem_u32(bar)), "r"(rank));
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(to),
               "r"(__float_as_uint(x)), "r"(count)
               : "memory");
}

}  // namespace gbattn
