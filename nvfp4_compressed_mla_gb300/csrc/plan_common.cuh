// plan_common.cuh -- what the kernels that work on block tables and the stack of
// free pages share: cluster barriers, prefix sums, division by the page size, launches.
#pragma once

#include "common.cuh"

namespace nvfp4_mla {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMaxCluster = 8;  // largest portable cluster

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t rank, int32_t v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// Inclusive prefix sum over the block's threads plus `carry`; `carry` becomes
// the total. `warp_sums` holds kPlanWarps values.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t& carry, int64_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  __syncthreads();  // the previous scan's sums have been read
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  int64_t w = warp_sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, w, d);
    if (lane >= d) w += o;
  }
  const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  const int64_t total = __shfl_sync(0xffffffffu, w, 31);
  v += carry + (warp > 0 ? before : 0);
  carry += total;
  return v;
}

// Division of n < 2^31 by the page size, by a product (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994): with l =
// ceil(log2 d) and m = ceil(2^(31 + l) / d), m d exceeds 2^(31 + l) by less than
// d <= 2^l, so that n m / 2^(31 + l) exceeds n / d by less than 1 / d.
struct PageSize {
  int32_t size;
  uint32_t mul, shift;
  __device__ __forceinline__ int32_t block(int32_t n) const {
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
  }
  __device__ __forceinline__ int32_t blocks(int32_t tokens) const {  // pages of 0 .. 2^31 - 1 tokens
    return tokens > 0 ? block(tokens - 1) + 1 : 0;
  }
};
PageSize page_division(int32_t size) {
  uint32_t l = 0;
  while (l < 31 && (1u << l) < static_cast<uint32_t>(size)) ++l;
  const uint64_t m = ((uint64_t{1} << (31 + l)) + size - 1) / size;  // 2^31 .. 2^32 - 1
  return {size, static_cast<uint32_t>(m), 31 + l};
}

// With `smem` bytes of dynamic shared memory, at most `most`. The kernel's limit
// is the process's: calls of other threads rely on it, so that it is the same one
// in every call that needs it.
template <typename Params>
int32_t launch_cluster_smem(void (*kernel)(Params), const Params& p, int ctas, size_t smem,
                            size_t most, cudaStream_t stream) {
  // what a kernel has beside it counts towards the 48 KB that need no setting
  if (smem > 40 * 1024 &&
      cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(most)) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return NVFP4_MLA_ERR_LAUNCH;
  }
  return NVFP4_MLA_OK;
}

// With `per_seq` bytes of shared memory a sequence.
template <typename Params>
int32_t launch_cluster(void (*kernel)(Params), const Params& p, int ctas, size_t per_seq,
                       cudaStream_t stream) {
  return launch_cluster_smem(kernel, p, ctas, per_seq * static_cast<size_t>(p.num_seqs),
                             per_seq * NVFP4_MLA_MAX_PLAN_SEQS, stream);
}

bool plan_shape_ok(int32_t num_seqs, int32_t max_blocks, int32_t page_size,
                   int32_t free_capacity) {
  return num_seqs > 0 && num_seqs <= NVFP4_MLA_MAX_PLAN_SEQS && max_blocks > 0 && page_size > 0 &&
         page_size <= (1 << 20) && static_cast<int64_t>(max_blocks) * page_size <= INT32_MAX &&
         free_capacity >= 0;
}

}  // namespace
}  // namespace nvfp4_mla
