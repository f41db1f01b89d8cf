// Host helpers: kernels whose blocks go on over their work until it is done, and kernels of one call
// that follow each other.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

namespace ssd {
namespace {   // of its own in every library: a process may hold the normal and the checked one

// Blocks of `kernel` that the device holds at once (looked up once per kernel and device).
template <typename K>
cudaError_t resident_blocks(K* kernel, int threads, int smem, int* out) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, int> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_pair(reinterpret_cast<const void*>(kernel), dev);
  const auto it = known.find(key);
  if (it != known.end()) {
    *out = it->second;
    return cudaSuccess;
  }
  int sms = 0, per = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && smem > 0)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *out = known[key] = sms * std::max(per, 1);
  return cudaSuccess;
}

// Launch of a kernel that follows another one of the same call on the stream: its blocks may take their
// places while that one ends, and wait in follow() for all its writes.  Saves about a
// microsecond of each of a call's launches behind the first.
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

#ifdef __CUDACC__
// At the start of every kernel of a call that launches more than one: waits for the kernel before (at
// once, where there is none or it was launched plainly), then lets the next one's blocks come.  Every
// thread calls it before it touches memory, so a kernel's end implies the end of all before it.  What the
// kernels before have written is read with plain loads, never through the read-only path.
__device__ __forceinline__ void follow() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
#endif

}  // namespace
}  // namespace ssd
