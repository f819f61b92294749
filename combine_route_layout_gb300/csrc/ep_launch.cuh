// Launches whose start overlaps the end of the kernel before them (programmatic
// dependent launch). The kernel calls begin_overlapped() before its first access
// to global memory: what comes ahead of it (barriers, TMEM, constant operands) is
// set up while the kernel before still runs, everything after it sees that
// kernel's writes. A kernel that is followed by one of these lets it start as
// soon as all of its own CTAs have.
#pragma once

#include <atomic>

#include "ep_kernels.cuh"

namespace ep {

#ifdef __CUDACC__
__device__ __forceinline__ void begin_overlapped() {
  pdl_launch_dependents();
  pdl_wait();
}

// 16 bytes that this SM reads once.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
#endif

template <typename... Params, typename... Args>
inline cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, int block, size_t smem,
                                     cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Raise the kernel's shared-memory limit to `most`, all that any launch of it takes, once
// on each device (`raised`: the kernel's own). A limit of each launch's own size could
// be lowered by one host thread between another's and its launch.
template <typename Kernel>
inline cudaError_t raise_shared_limit(Kernel* kernel, size_t most, std::atomic<uint64_t>* raised) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (raised->load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
  if (e == cudaSuccess) raised->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace ep
