// Launch helper shared by the block-sparse step's kernels.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace pa {

// Once per device: let `Kernel` take as much dynamic shared memory as a CTA
// can have, and run in clusters of more than 8 CTAs.
template <auto Kernel>
cudaError_t allow_large() {
  static std::atomic<uint64_t> done{0};  // a bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit & done.load(std::memory_order_acquire)) return cudaSuccess;
  const void* k = reinterpret_cast<const void*>(Kernel);
  cudaFuncAttributes a;
  e = cudaFuncGetAttributes(&a, k);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             227 * 1024 - (int)a.sharedSizeBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// Launch `Kernel` as a programmatic dependent of the stream's previous
// kernel (its CTAs may start before that one ends; each waits with
// griddepcontrol.wait before its first global access) in clusters of
// `cluster` CTAs along x.
template <auto Kernel, typename... Args>
cudaError_t launch_dependent(dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, Kernel, args...);
  const cudaError_t last = cudaGetLastError();  // a refused launch leaves no error behind
  return e != cudaSuccess ? e : last;
}

}  // namespace pa
