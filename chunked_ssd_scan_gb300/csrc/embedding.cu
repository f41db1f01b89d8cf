// Token embedding with scaling and the gradient of its table (declarations in include/ssdscan.h):
//   out[i] = scale * table[ids[i]],  dtable[v] = scale * sum_{ids[i] = v} dout[i].
#include <math.h>
#include <string.h>

#include "common.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

template <typename Id>
__device__ __forceinline__ int64_t row_of(const Id* ids, int64_t i, int64_t V) {
  const int64_t v = (int64_t)ids[i];
  return v >= 0 && v < V ? v : -1;
}

// One warp per token.
template <typename T, typename Id>
__global__ void __launch_bounds__(kThreads) embed_forward_kernel(const Id* ids, int64_t n, const T* table,
                                                                 int64_t V, int64_t D, float scale, T* out) {
  const int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (i >= n) return;
  const int64_t v = row_of(ids, i, V);
  for (int64_t d = threadIdx.x % 32; d < D; d += 32)
    st_from_f32(out + i * D + d, v >= 0 ? scale * ld_f32(table + v * D + d) : 0.f);
}

// One block per row of the table: the block looks through all ids and adds its row's tokens in
// their order.
template <typename T, typename Id>
__global__ void __launch_bounds__(kThreads) embed_backward_kernel(const Id* ids, int64_t n, const T* dout,
                                                                  int64_t V, int64_t D, float scale,
                                                                  float* dtable) {
  __shared__ int64_t hits[kThreads];
  __shared__ int warp_count[kThreads / 32];
  const int64_t v = blockIdx.x;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int64_t d = threadIdx.x; d < D; d += kThreads) dtable[v * D + d] = 0.f;
  for (int64_t i0 = 0; i0 < n; i0 += kThreads) {
    const int64_t i = i0 + threadIdx.x;
    const bool hit = i < n && row_of(ids, i, V) == v;
    const unsigned ball = __ballot_sync(0xffffffffu, hit);
    if (lane == 0) warp_count[warp] = __popc(ball);
    if (__syncthreads_or(hit)) {
      int at = __popc(ball & ((1u << lane) - 1)), total = 0;
      for (int k = 0; k < kThreads / 32; ++k) {
        if (k < warp) at += warp_count[k];
        total += warp_count[k];
      }
      if (hit) hits[at] = i;
      __syncthreads();
      for (int64_t d = threadIdx.x; d < D; d += kThreads) {
        float s = dtable[v * D + d];
        for (int k = 0; k < total; ++k) s += scale * ld_f32(dout + hits[k] * D + d);
        dtable[v * D + d] = s;
      }
    }
    __syncthreads();
  }
}

constexpr int64_t kMaxElems = (int64_t)1 << 40;

ssd_status check_sizes(int64_t n, int64_t V, int64_t D) {
  if (n < 0 || V < 1 || D < 1) return SSD_ERR_INVALID_ARG;
  if (n > 0x7fffffffLL || V > 0x7fffffffLL || D > kMaxElems / V || (n > 0 && D > kMaxElems / n))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
ssd_status done(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

template <typename T, typename Id>
cudaError_t launch_forward(const void* ids, int64_t n, const void* table, int64_t V, int64_t D, float scale,
                           void* out, cudaStream_t st) {
  constexpr int kWarps = kThreads / 32;
  embed_forward_kernel<T, Id><<<(unsigned)((n + kWarps - 1) / kWarps), kThreads, 0, st>>>(
      static_cast<const Id*>(ids), n, static_cast<const T*>(table), V, D, scale, static_cast<T*>(out));
  return cudaGetLastError();
}

template <typename T, typename Id>
cudaError_t launch_backward(const void* ids, int64_t n, const void* dout, int64_t V, int64_t D, float scale,
                            float* dtable, cudaStream_t st) {
  embed_backward_kernel<T, Id><<<(unsigned)V, kThreads, 0, st>>>(
      static_cast<const Id*>(ids), n, static_cast<const T*>(dout), V, D, scale, dtable);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status embedding_forward(const void* ids, int32_t ids_bits, int64_t n, const void* table,
                             int64_t vocab, int64_t dim, int32_t io_dtype, float scale, void* out,
                             void* stream) {
  const ssd_status bad = check_sizes(n, vocab, dim);
  if (bad != SSD_OK) return bad;
  if ((ids_bits != 32 && ids_bits != 64) || (io_dtype != SSD_F32 && io_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  const bool bf16 = io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  if (n > 0 && (!ids || !table || !out)) return SSD_ERR_INVALID_ARG;
  if (misaligned(ids, ids_bits / 8) || misaligned(table, e) || misaligned(out, e))
    return SSD_ERR_INVALID_ARG;
  if (n == 0) return SSD_OK;
  auto f = bf16 ? (ids_bits == 64 ? launch_forward<__nv_bfloat16, int64_t> : launch_forward<__nv_bfloat16, int32_t>)
                : (ids_bits == 64 ? launch_forward<float, int64_t> : launch_forward<float, int32_t>);
  return done(f(ids, n, table, vocab, dim, scale, out, static_cast<cudaStream_t>(stream)));
}

size_t embedding_backward_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  return check_sizes(n, vocab, dim) == SSD_OK ? sizeof(WsHeader) : 0;
}

ssd_status embedding_backward(const void* ids, int32_t ids_bits, int64_t n, const void* dout,
                              int64_t vocab, int64_t dim, int32_t io_dtype, float scale,
                              float* dtable, void* workspace, size_t workspace_bytes,
                              void* stream) {
  const ssd_status bad = check_sizes(n, vocab, dim);
  if (bad != SSD_OK) return bad;
  if ((ids_bits != 32 && ids_bits != 64) || (io_dtype != SSD_F32 && io_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  const bool bf16 = io_dtype == SSD_BF16;
  if (!dtable || (n > 0 && (!ids || !dout))) return SSD_ERR_INVALID_ARG;
  if (misaligned(ids, ids_bits / 8) || misaligned(dout, bf16 ? 2 : 4) || misaligned(dtable, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, kWsAlign) ||
      workspace_bytes < embedding_backward_workspace_bytes(n, vocab, dim))
    return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0)
    return done(cudaMemsetAsync(dtable, 0, sizeof(float) * (size_t)(vocab * dim), st));
  auto f = bf16 ? (ids_bits == 64 ? launch_backward<__nv_bfloat16, int64_t> : launch_backward<__nv_bfloat16, int32_t>)
                : (ids_bits == 64 ? launch_backward<float, int64_t> : launch_backward<float, int32_t>);
  return done(f(ids, n, dout, vocab, dim, scale, dtable, st));
}

}  // extern "C"
