// Launches of the dense operators, which follow one another within microseconds: a kernel's blocks come
// as soon as the blocks of the kernel before it have ended, prepare (barriers, tensor memory) and wait,
// before they touch any global memory, until that kernel is complete and its writes are visible.
// Back to back that takes 2 to 5 us off a call (norm gradient at 8192 x 768: 37 -> 32 us). Letting blocks
// come while the earlier kernel's still run gains another 0.7 us on a linear layer, but two kernels in
// turn then hold each other's places: 45 us for the same norm gradient.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace sol {

// By every thread that goes on to global memory, before it does: waits for all earlier kernels of the stream.
__device__ __forceinline__ void chained_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// A kernel's dynamic shared memory is allowed once per device, at the largest size that any of its launches
// takes: the attribute is the kernel's, so a launch that set its own size would take it from another thread's.
template <auto Kernel>
cudaError_t allow_smem(int most) {
  constexpr int kDevices = 64;
  static std::atomic<bool> done[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < kDevices && done[dev].load(std::memory_order_relaxed))) return e;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e == cudaSuccess && dev < kDevices) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

}  // namespace sol
