// Group norm with an activation, channels last (declarations in include/ssdscan.h):
//   xhat = (x - mean) rstd, z = xhat w + b, y = act(z), statistics over the S * C/G values of a
//   sample's group; reverse mode, dz = dy act'(z), q = dz w:
//   dx = rstd (q - mean(q) - xhat mean(q xhat)), dw = sum dz xhat, db = sum dz.
#include <math.h>
#include <string.h>

#include "common.cuh"

namespace ssd {
namespace {

struct NormParams {
  const void *x, *dy;
  const float *w, *bias, *mean_in, *rstd_in;
  void *y, *dx;
  float *mean, *rstd, *dw, *db;
  int64_t N, S, C, G, cg;
  int64_t xs[2], ds[2];
  float eps;
  int32_t act;
};

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
  for (int k = 0; k < kThreads / 32; ++k) s += part[k];
  return s;
}

// Compensated sum: a thread may add millions of values of one sign.
struct Sum {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float v) {
    const float y = v - c, t = s + y;
    c = (t - s) - y;
    s = t;
  }
};

__device__ __forceinline__ float act_fwd(float z, int act) {
  return act == SSD_ACT_SILU ? z / (1.f + expf(-z)) : z;
}
// act'(z)
__device__ __forceinline__ float act_grad(float z, int act) {
  if (act != SSD_ACT_SILU) return 1.f;
  const float s = 1.f / (1.f + expf(-z));
  return s * (1.f + z * (1.f - s));
}

// One block per (sample, group).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(NormParams p) {
  const int64_t n = blockIdx.x / p.G, g = blockIdx.x % p.G, c0 = g * p.cg;
  const T* x = static_cast<const T*>(p.x) + n * p.xs[0] + c0;
  T* y = static_cast<T*>(p.y) + n * p.S * p.C + c0;
  const int64_t count = p.S * p.cg;
  Sum s, v;
  for (int64_t k = threadIdx.x; k < count; k += kThreads)
    s.add(ld_f32(x + k / p.cg * p.xs[1] + k % p.cg));
  const float mean = block_sum(s.s) / (float)count;
  for (int64_t k = threadIdx.x; k < count; k += kThreads) {
    const float d = ld_f32(x + k / p.cg * p.xs[1] + k % p.cg) - mean;
    v.add(d * d);
  }
  const float rstd = 1.f / sqrtf(block_sum(v.s) / (float)count + p.eps);
  for (int64_t k = threadIdx.x; k < count; k += kThreads) {
    const int64_t r = k / p.cg, c = k % p.cg;
    float z = (ld_f32(x + r * p.xs[1] + c) - mean) * rstd;
    z = z * (p.w ? p.w[c0 + c] : 1.f) + (p.bias ? p.bias[c0 + c] : 0.f);
    st_from_f32(y + r * p.C + c, act_fwd(z, p.act));
  }
  if (threadIdx.x == 0 && p.mean) {
    p.mean[blockIdx.x] = mean;
    p.rstd[blockIdx.x] = rstd;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(NormParams p) {
  const int64_t n = blockIdx.x / p.G, g = blockIdx.x % p.G, c0 = g * p.cg;
  const T* x = static_cast<const T*>(p.x) + n * p.xs[0] + c0;
  const T* dy = static_cast<const T*>(p.dy) + n * p.ds[0] + c0;
  T* dx = static_cast<T*>(p.dx) + n * p.S * p.C + c0;
  const float mean = p.mean_in[blockIdx.x], rstd = p.rstd_in[blockIdx.x];
  const int64_t count = p.S * p.cg;
  Sum sq, sqx;
  float mq = 0.f, mqx = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int64_t k = threadIdx.x; k < count; k += kThreads) {
      const int64_t r = k / p.cg, c = k % p.cg;
      const float w = p.w ? p.w[c0 + c] : 1.f;
      const float xh = (ld_f32(x + r * p.xs[1] + c) - mean) * rstd;
      const float z = xh * w + (p.bias ? p.bias[c0 + c] : 0.f);
      const float q = ld_f32(dy + r * p.ds[1] + c) * act_grad(z, p.act) * w;
      if (pass == 0) {
        sq.add(q);
        sqx.add(q * xh);
      } else {
        st_from_f32(dx + r * p.C + c, rstd * (q - mq - xh * mqx));
      }
    }
    if (pass == 0) {
      mq = block_sum(sq.s) / (float)count;
      mqx = block_sum(sqx.s) / (float)count;
    }
  }
}

// One block per channel.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_param_grad_kernel(NormParams p) {
  const int64_t c = blockIdx.x, g = c / p.cg;
  const float w = p.w ? p.w[c] : 1.f, bias = p.bias ? p.bias[c] : 0.f;
  Sum sw, sb;
  for (int64_t k = threadIdx.x; k < p.N * p.S; k += kThreads) {
    const int64_t n = k / p.S, r = k % p.S;
    const float xh = (ld_f32(static_cast<const T*>(p.x) + n * p.xs[0] + r * p.xs[1] + c) -
                      p.mean_in[n * p.G + g]) * p.rstd_in[n * p.G + g];
    const float dz = ld_f32(static_cast<const T*>(p.dy) + n * p.ds[0] + r * p.ds[1] + c) *
                     act_grad(xh * w + bias, p.act);
    sw.add(dz * xh);
    sb.add(dz);
  }
  const float dw = block_sum(sw.s), db = block_sum(sb.s);
  if (threadIdx.x == 0) {
    if (p.dw) p.dw[c] = dw;
    if (p.db) p.db[c] = db;
  }
}

constexpr int64_t kMaxElems = (int64_t)1 << 40;

ssd_status check_shape(const group_norm_shape* s, bool backward) {
  if (!s || s->batch < 0 || s->rows < 0 || s->channels < 1 || s->groups < 1 ||
      s->channels % s->groups != 0)
    return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_F32 && s->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (s->activation != SSD_ACT_NONE && s->activation != SSD_ACT_SILU) return SSD_ERR_INVALID_ARG;
  if (!(s->eps >= 0.f) || !isfinite(s->eps)) return SSD_ERR_INVALID_ARG;
  for (int k = 0; k < 2; ++k)
    if (s->x_stride[k] < 0 || (backward && s->dy_stride[k] < 0)) return SSD_ERR_INVALID_ARG;
  if (s->channels > 0x7fffffffLL || s->rows > kMaxElems / s->channels ||
      (s->rows > 0 && s->batch > kMaxElems / s->channels / s->rows))
    return SSD_ERR_UNSUPPORTED;
  if (s->batch > 0x7fffffffLL / s->groups) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

NormParams norm_params(const group_norm_shape* s) {
  NormParams p;
  memset(&p, 0, sizeof(p));
  p.N = s->batch;
  p.S = s->rows;
  p.C = s->channels;
  p.G = s->groups;
  p.cg = s->channels / s->groups;
  p.eps = s->eps;
  p.act = s->activation;
  memcpy(p.xs, s->x_stride, sizeof(p.xs));
  memcpy(p.ds, s->dy_stride, sizeof(p.ds));
  return p;
}

ssd_status done(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t group_norm_workspace_bytes(const group_norm_shape* shape, int32_t backward) {
  (void)backward;
  return check_shape(shape, false) == SSD_OK ? sizeof(WsHeader) : 0;
}

ssd_status group_norm_forward(const group_norm_shape* shape, const void* x, const float* weight,
                              const float* bias, void* y, float* mean, float* rstd,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const ssd_status bad = check_shape(shape, false);
  if (bad != SSD_OK) return bad;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  const bool empty = shape->batch == 0 || shape->rows == 0;
  if ((!empty && (!x || !y)) || (mean == nullptr) != (rstd == nullptr)) return SSD_ERR_INVALID_ARG;
  if (misaligned(x, e) || misaligned(y, e) || misaligned(weight, 4) || misaligned(bias, 4) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, kWsAlign) ||
      workspace_bytes < group_norm_workspace_bytes(shape, 0))
    return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) return SSD_OK;
  NormParams p = norm_params(shape);
  p.x = x;
  p.w = weight;
  p.bias = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  const unsigned grid = (unsigned)(p.N * p.G);
  if (bf16) norm_forward_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
  else norm_forward_kernel<float><<<grid, kThreads, 0, st>>>(p);
  return done(cudaGetLastError());
}

ssd_status group_norm_backward(const group_norm_shape* shape, const void* x, const void* dy,
                               const float* mean, const float* rstd, const float* weight,
                               const float* bias, void* dx, float* dweight, float* dbias,
                               void* workspace, size_t workspace_bytes, void* stream) {
  const ssd_status bad = check_shape(shape, true);
  if (bad != SSD_OK) return bad;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  const bool empty = shape->batch == 0 || shape->rows == 0;
  if (!empty && (!x || !dy || !dx || !mean || !rstd)) return SSD_ERR_INVALID_ARG;
  if (misaligned(x, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(weight, 4) ||
      misaligned(bias, 4) || misaligned(mean, 4) || misaligned(rstd, 4) ||
      misaligned(dweight, 4) || misaligned(dbias, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, kWsAlign) ||
      workspace_bytes < group_norm_workspace_bytes(shape, 1))
    return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) {
    for (float* d : {dweight, dbias})
      if (d && cudaMemsetAsync(d, 0, sizeof(float) * (size_t)shape->channels, st) != cudaSuccess)
        return SSD_ERR_CUDA;
    return SSD_OK;
  }
  NormParams p = norm_params(shape);
  p.x = x;
  p.dy = dy;
  p.mean_in = mean;
  p.rstd_in = rstd;
  p.w = weight;
  p.bias = bias;
  p.dx = dx;
  p.dw = dweight;
  p.db = dbias;
  const unsigned grid = (unsigned)(p.N * p.G);
  if (bf16) norm_backward_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
  else norm_backward_kernel<float><<<grid, kThreads, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SSD_ERR_CUDA;
  if (dweight || dbias) {
    if (bf16) norm_param_grad_kernel<__nv_bfloat16><<<(unsigned)p.C, kThreads, 0, st>>>(p);
    else norm_param_grad_kernel<float><<<(unsigned)p.C, kThreads, 0, st>>>(p);
  }
  return done(cudaGetLastError());
}

}  // extern "C"
