// Gated linear recurrence, elementwise per channel (declarations in include/ssdscan.h):
//   h_t = a_t h_{t-1} + m_t i_t x_t,  a = e^l, l = -c softplus(decay) sigmoid(gate_a),
//   m = sqrt(1 - a^2) = sqrt(-expm1(2 l)), i = sigmoid(gate_x)
// and its reverse mode, G_t = dy_t + a_{t+1} G_{t+1}:
//   dx = G m i; dgate_x = G m x i (1 - i); k = a (h_{t-1} - a i x / m);
//   dgate_a = G k l (1 - r); ddecay = sum G k (-c r) sigmoid(decay).
#include <math.h>
#include <string.h>

#include "common.cuh"

namespace ssd {
namespace {

constexpr int kChunk = GATED_RECURRENCE_CHUNK;

struct RecParams {
  const void *x, *ga, *gx, *dy;
  const float *decay, *init, *states_in, *dfinal;
  void *y, *dx, *dga, *dgx;
  float *final_state, *states_out, *ddecay, *dinit, *partial;
  int64_t batch, T, D, nch;
  int64_t xs[2], as[2], gs[2], ds[2];
  float c;
};

__device__ __forceinline__ float softplus(float d) { return fmaxf(d, 0.f) + log1pf(expf(-fabsf(d))); }

// The decay is carried as w = a - 1 = expm1(l), and a step is h + (w h + b): near one, a itself has an
// absolute rounding error of 2^-25 whose bias a channel with memory 1 / (1 - a) multiplies by
// that memory, while w's error is relative to 1 - a.
struct Gates {
  float l, r, w, m, i;
};
__device__ __forceinline__ Gates gates(float ga, float gx, float rate) {
  Gates g;
  g.r = 1.f / (1.f + expf(-ga));
  g.i = 1.f / (1.f + expf(-gx));
  g.l = -rate * g.r;
  g.w = expm1f(g.l);
  g.m = sqrtf(-g.w * (2.f + g.w));   // 1 - a^2
  return g;
}
__device__ __forceinline__ float decayed(const Gates& g, float h, float b) { return h + fmaf(g.w, h, b); }

// One thread per (sequence, channel), the steps in order.
template <typename T>
__global__ void rec_forward_kernel(RecParams p) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= p.batch * p.D) return;
  const int64_t b = id / p.D, d = id % p.D;
  const float rate = p.c * softplus(p.decay[d]);
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + d;
  const T* ga = static_cast<const T*>(p.ga) + b * p.as[0] + d;
  const T* gx = static_cast<const T*>(p.gx) + b * p.gs[0] + d;
  T* y = p.y ? static_cast<T*>(p.y) + b * p.T * p.D + d : nullptr;
  float h = p.init ? p.init[id] : 0.f;
  for (int64_t t = 0; t < p.T; ++t) {
    if (p.states_out && t % kChunk == 0) p.states_out[(b * p.nch + t / kChunk) * p.D + d] = h;
    const Gates g = gates(ld_f32(ga + t * p.as[1]), ld_f32(gx + t * p.gs[1]), rate);
    h = decayed(g, h, g.m * g.i * ld_f32(x + t * p.xs[1]));
    if (y) st_from_f32(y + t * p.D, h);
  }
  if (p.final_state) p.final_state[id] = h;
}

// One thread per (sequence, channel): chunks from the last to the first, each recomputed from the
// state before it.
template <typename T>
__global__ void rec_backward_kernel(RecParams p) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= p.batch * p.D) return;
  const int64_t b = id / p.D, d = id % p.D;
  const float rate = p.c * softplus(p.decay[d]);
  const T* x = static_cast<const T*>(p.x) + b * p.xs[0] + d;
  const T* ga = static_cast<const T*>(p.ga) + b * p.as[0] + d;
  const T* gx = static_cast<const T*>(p.gx) + b * p.gs[0] + d;
  const T* dy = static_cast<const T*>(p.dy) + b * p.ds[0] + d;
  const int64_t o = b * p.T * p.D + d;
  float carry = p.dfinal ? p.dfinal[id] : 0.f, sum = 0.f, comp = 0.f;
  float prev[kChunk];
  for (int64_t k = p.nch - 1; k >= 0; --k) {
    const int64_t t0 = k * kChunk;
    const int n = (int)min((int64_t)kChunk, p.T - t0);
    float h = p.states_in[(b * p.nch + k) * p.D + d];
    for (int j = 0; j < n; ++j) {
      const int64_t t = t0 + j;
      prev[j] = h;
      const Gates g = gates(ld_f32(ga + t * p.as[1]), ld_f32(gx + t * p.gs[1]), rate);
      h = decayed(g, h, g.m * g.i * ld_f32(x + t * p.xs[1]));
    }
    for (int j = n - 1; j >= 0; --j) {
      const int64_t t = t0 + j;
      const Gates g = gates(ld_f32(ga + t * p.as[1]), ld_f32(gx + t * p.gs[1]), rate);
      const float xv = ld_f32(x + t * p.xs[1]);
      const float G = ld_f32(dy + t * p.ds[1]) + carry;
      const float a = 1.f + g.w;
      const float k1 = G * a * (prev[j] - (g.m > 0.f ? a * g.i * xv / g.m : 0.f));
      const float mi = g.m * g.i;
      st_from_f32(static_cast<T*>(p.dx) + o + t * p.D, G * mi);
      st_from_f32(static_cast<T*>(p.dgx) + o + t * p.D, G * mi * xv * (1.f - g.i));
      st_from_f32(static_cast<T*>(p.dga) + o + t * p.D, k1 * g.l * (1.f - g.r));
      const float add = k1 * g.r - comp, s = sum + add;   // compensated sum over the steps
      comp = (s - sum) - add;
      sum = s;
      carry = decayed(g, G, 0.f);
    }
  }
  p.partial[id] = sum;
  if (p.dinit) p.dinit[id] = carry;
}

__global__ void rec_ddecay_kernel(RecParams p) {
  const int64_t d = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (d >= p.D) return;
  float s = 0.f;
  for (int64_t b = 0; b < p.batch; ++b) s += p.partial[b * p.D + d];
  p.ddecay[d] = -p.c * s / (1.f + expf(-p.decay[d]));
}

template <typename T>
__global__ void rec_step_kernel(RecParams p) {
  const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= p.batch * p.D) return;
  const int64_t b = id / p.D, d = id % p.D;
  const Gates g = gates(ld_f32(static_cast<const T*>(p.ga) + b * p.as[0] + d),
                        ld_f32(static_cast<const T*>(p.gx) + b * p.gs[0] + d),
                        p.c * softplus(p.decay[d]));
  const float h = decayed(g, p.init ? p.init[id] : 0.f,
                          g.m * g.i * ld_f32(static_cast<const T*>(p.x) + b * p.xs[0] + d));
  p.final_state[id] = h;
  st_from_f32(static_cast<T*>(p.y) + id, h);
}

constexpr int64_t kMaxElems = (int64_t)1 << 40;

ssd_status check_shape(const gated_recurrence_shape* s, bool backward) {
  if (!s || s->batch < 0 || s->seqlen < 0 || s->d_model < 1) return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_F32 && s->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (!(s->c > 0.f) || !isfinite(s->c)) return SSD_ERR_INVALID_ARG;
  for (int k = 0; k < 2; ++k)
    if (s->x_stride[k] < 0 || s->gate_a_stride[k] < 0 || s->gate_x_stride[k] < 0 ||
        (backward && s->dy_stride[k] < 0))
      return SSD_ERR_INVALID_ARG;
  if (s->d_model > kMaxElems || s->batch > kMaxElems / s->d_model ||
      (s->batch > 0 && s->seqlen > kMaxElems / s->d_model / s->batch))
    return SSD_ERR_UNSUPPORTED;
  if ((s->batch * s->d_model + 127) / 128 > 0x7fffffffLL) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

RecParams rec_params(const gated_recurrence_shape* s) {
  RecParams p;
  memset(&p, 0, sizeof(p));
  p.batch = s->batch;
  p.T = s->seqlen;
  p.D = s->d_model;
  p.nch = (s->seqlen + kChunk - 1) / kChunk;
  p.c = s->c;
  memcpy(p.xs, s->x_stride, sizeof(p.xs));
  memcpy(p.as, s->gate_a_stride, sizeof(p.as));
  memcpy(p.gs, s->gate_x_stride, sizeof(p.gs));
  memcpy(p.ds, s->dy_stride, sizeof(p.ds));
  return p;
}

struct RecLayout {
  size_t states = 0, partial = 0, total = 0;
};
RecLayout rec_layout(const gated_recurrence_shape* s, bool backward) {
  RecLayout L;
  size_t off = sizeof(WsHeader);
  if (backward) {
    L.states = off;
    const int64_t nch = (s->seqlen + kChunk - 1) / kChunk;
    off = align_up(off + sizeof(float) * (size_t)(s->batch * nch * s->d_model), kWsAlign);
    L.partial = off;
    off = align_up(off + sizeof(float) * (size_t)(s->batch * s->d_model), kWsAlign);
  }
  L.total = off;
  return L;
}

cudaError_t set_rows(float* dst, const float* src, int64_t n, cudaStream_t st) {
  if (!dst || n == 0) return cudaSuccess;
  return src ? cudaMemcpyAsync(dst, src, sizeof(float) * (size_t)n, cudaMemcpyDeviceToDevice, st)
             : cudaMemsetAsync(dst, 0, sizeof(float) * (size_t)n, st);
}

cudaError_t launch_forward(const RecParams& p, bool bf16, cudaStream_t st) {
  const unsigned grid = (unsigned)((p.batch * p.D + 127) / 128);
  if (bf16) rec_forward_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(p);
  else rec_forward_kernel<float><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}

ssd_status done(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t gated_recurrence_workspace_bytes(const gated_recurrence_shape* shape, int32_t backward) {
  if (check_shape(shape, false) != SSD_OK) return 0;
  return rec_layout(shape, backward != 0).total;
}

ssd_status gated_recurrence_forward(const gated_recurrence_shape* shape, const void* x,
                                    const void* gate_a, const void* gate_x, const float* decay,
                                    const float* init_state, void* y, float* final_state,
                                    float* states, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  const ssd_status bad = check_shape(shape, false);
  if (bad != SSD_OK) return bad;
  const size_t e = shape->io_dtype == SSD_BF16 ? 2 : 4;
  const bool empty = shape->batch == 0 || shape->seqlen == 0;
  if (!empty && (!x || !gate_a || !gate_x || !decay)) return SSD_ERR_INVALID_ARG;
  if (misaligned(x, e) || misaligned(gate_a, e) || misaligned(gate_x, e) || misaligned(y, e) ||
      misaligned(decay, 4) || misaligned(init_state, 4) || misaligned(final_state, 4) ||
      misaligned(states, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, kWsAlign) ||
      workspace_bytes < rec_layout(shape, false).total)
    return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) return done(set_rows(final_state, init_state, shape->batch * shape->d_model, st));
  RecParams p = rec_params(shape);
  p.x = x;
  p.ga = gate_a;
  p.gx = gate_x;
  p.decay = decay;
  p.init = init_state;
  p.y = y;
  p.final_state = final_state;
  p.states_out = states;
  return done(launch_forward(p, shape->io_dtype == SSD_BF16, st));
}

ssd_status gated_recurrence_backward(const gated_recurrence_shape* shape, const void* x,
                                     const void* gate_a, const void* gate_x, const float* decay,
                                     const float* init_state, const float* states, const void* dy,
                                     const float* dfinal, void* dx, void* dgate_a, void* dgate_x,
                                     float* ddecay, float* dinit, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const ssd_status bad = check_shape(shape, true);
  if (bad != SSD_OK) return bad;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  const bool empty = shape->batch == 0 || shape->seqlen == 0;
  if (!ddecay ||
      (!empty && (!x || !gate_a || !gate_x || !decay || !dy || !dx || !dgate_a || !dgate_x)))
    return SSD_ERR_INVALID_ARG;
  if (misaligned(x, e) || misaligned(gate_a, e) || misaligned(gate_x, e) || misaligned(dy, e) ||
      misaligned(dx, e) || misaligned(dgate_a, e) || misaligned(dgate_x, e) ||
      misaligned(decay, 4) || misaligned(init_state, 4) || misaligned(states, 4) ||
      misaligned(dfinal, 4) || misaligned(ddecay, 4) || misaligned(dinit, 4))
    return SSD_ERR_INVALID_ARG;
  const RecLayout L = rec_layout(shape, true);
  if (!workspace || misaligned(workspace, kWsAlign) || workspace_bytes < L.total)
    return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) {
    const cudaError_t ce = set_rows(ddecay, nullptr, shape->d_model, st);
    if (ce != cudaSuccess) return SSD_ERR_CUDA;
    return done(set_rows(dinit, dfinal, shape->batch * shape->d_model, st));
  }
  char* ws = static_cast<char*>(workspace);
  RecParams p = rec_params(shape);
  p.x = x;
  p.ga = gate_a;
  p.gx = gate_x;
  p.decay = decay;
  p.init = init_state;
  if (!states) {
    RecParams f = p;
    f.states_out = reinterpret_cast<float*>(ws + L.states);
    if (launch_forward(f, bf16, st) != cudaSuccess) return SSD_ERR_CUDA;
    states = f.states_out;
  }
  p.states_in = states;
  p.dy = dy;
  p.dfinal = dfinal;
  p.dx = dx;
  p.dga = dgate_a;
  p.dgx = dgate_x;
  p.ddecay = ddecay;
  p.dinit = dinit;
  p.partial = reinterpret_cast<float*>(ws + L.partial);
  const unsigned grid = (unsigned)((p.batch * p.D + 127) / 128);
  if (bf16) rec_backward_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(p);
  else rec_backward_kernel<float><<<grid, 128, 0, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SSD_ERR_CUDA;
  rec_ddecay_kernel<<<(unsigned)((p.D + 127) / 128), 128, 0, st>>>(p);
  return done(cudaGetLastError());
}

ssd_status gated_recurrence_step(const gated_recurrence_shape* shape, const void* x,
                                 const void* gate_a, const void* gate_x, const float* decay,
                                 const float* state, void* y, float* state_out, void* stream) {
  const ssd_status bad = check_shape(shape, false);
  if (bad != SSD_OK) return bad;
  if (shape->seqlen != 1) return SSD_ERR_INVALID_ARG;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  if (shape->batch == 0) return SSD_OK;
  if (!x || !gate_a || !gate_x || !decay || !y || !state_out) return SSD_ERR_INVALID_ARG;
  if (misaligned(x, e) || misaligned(gate_a, e) || misaligned(gate_x, e) || misaligned(y, e) ||
      misaligned(decay, 4) || misaligned(state, 4) || misaligned(state_out, 4))
    return SSD_ERR_INVALID_ARG;
  RecParams p = rec_params(shape);
  p.x = x;
  p.ga = gate_a;
  p.gx = gate_x;
  p.decay = decay;
  p.init = state;
  p.y = y;
  p.final_state = state_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)((p.batch * p.D + 127) / 128);
  if (bf16) rec_step_kernel<__nv_bfloat16><<<grid, 128, 0, st>>>(p);
  else rec_step_kernel<float><<<grid, 128, 0, st>>>(p);
  return done(cudaGetLastError());
}

}  // extern "C"
