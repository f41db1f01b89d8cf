// Host helpers: kernels whose blocks go on over their work until it is done, and kernels of one call
// that follow each other.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

namespace ssd {
namespace {   // of its own in every library: a process may hold the normal and the checked one

// Blocks of `kernel` that the device holds at once (looked up once per kernel and device; throws nothing).
cudaError_t resident_blocks(const void* kernel, int threads, int smem, int* out) {
  struct Known {
    const void* kernel;
    int dev, blocks;
  };
  constexpr int kMost = 256;   // more kernels than a translation unit has; beyond it, looked up every time
  static Known known[kMost];
  static int count = 0;
  static std::atomic_flag busy = ATOMIC_FLAG_INIT;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  while (busy.test_and_set(std::memory_order_acquire)) {
  }
  int blocks = 0;
  for (int k = 0; k < count; ++k)
    if (known[k].kernel == kernel && known[k].dev == dev) blocks = known[k].blocks;
  if (blocks == 0) {
    int sms = 0, per = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && smem > 0)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
    if (e == cudaSuccess) {
      blocks = sms * std::max(per, 1);
      if (count < kMost) known[count++] = {kernel, dev, blocks};
    }
  }
  busy.clear(std::memory_order_release);
  *out = blocks;
  return e;
}
template <typename... P>
cudaError_t resident_blocks(void (*kernel)(P...), int threads, int smem, int* out) {
  return resident_blocks(reinterpret_cast<const void*>(kernel), threads, smem, out);
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
