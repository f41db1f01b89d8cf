// Root-mean-square norm of rows with the residual's addition and an 8-bit output, and its reverse mode
// (declarations in include/ssdscan.h):
//   h = x + residual, r = 1 / sqrt(mean h^2 + eps), y = h r w;  8 bits: scale = max |y| / 448, q = y / scale
//   dx = r (w dy - xh mean(w dy xh)) + dresidual, xh = h r;  dw = sum over rows of dy xh
// Memory bounds it: every value is read once and written once.  A row's values stay in the registers of the threads
// that loaded them while its sum is formed, a thread keeps its channels (and their weights, and the sums of dw) for
// all rows of its block, and the next row's loads are on their way meanwhile.
#include <cuda_fp8.h>
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "launch.h"
#include "pack.cuh"

namespace ssd {
namespace {

constexpr float kMost = 448.f;
constexpr int kBlock = RMS_NORM_BLOCK;
constexpr int kWideThreads = 512;
constexpr int kRowThreads = 512;   // of a block whose rows stay in registers at most; one vector a thread is held to 64
                                   // registers all the same (16384 x 2048 bf16 backward 51 us, with what it likes 56)

struct NormParams {
  const void *x, *res, *dy;     // backward: x is h, res is dresidual
  const float *w, *rstd_in;
  void *y, *h;                  // backward: y is dx
  float *rstd, *scale, *partial, *dw;
  int64_t N, C, xs, rs, ds, blocks;   // blocks of channels with a scale of their own
  int64_t part_rows;            // backward: rows that the workspace has for partial sums of dw
  float eps;
  int tpr;                      // threads a row
  WsHeader* hdr;                // backward
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Sum and maximum over a row's threads (whole warps), the same in each of them.  `buf` alternates, so one barrier a
// row is enough.
struct RowReduce {
  float sum[2][32], most[2][32];
};
template <bool kMax>
__device__ __forceinline__ void row_reduce(RowReduce& sm, int buf, int tpr, float& s, float& m) {
  s = warp_sum(s);
  if (kMax) m = warp_max(m);
  if (tpr == 32) return;
  const int warp = threadIdx.x >> 5, per = tpr >> 5, first = warp / per * per;
  if ((threadIdx.x & 31) == 0) {
    sm.sum[buf][warp] = s;
    if (kMax) sm.most[buf][warp] = m;
  }
  __syncthreads();
  s = 0.f;
  for (int i = 0; i < per; ++i) {
    s += sm.sum[buf][first + i];
    if (kMax) m = fmaxf(m, sm.most[buf][first + i]);
  }
}

__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Quotients y / scale as a division rounds them, by Markstein's theorem (IBM Journal of Research and Development 34, 1990):
// with a reciprocal that is rounded to nearest, one step by the remainder makes of their product the quotient rounded to
// nearest.  (A division for every value: 62 us for 16384 x 2048 bf16 where this takes 56; the product alone, which rounds
// twice, 50.)  Both are brought to a middle size first: a scale below 2^-128 has no reciprocal in fp32 (zeros would become NaN
// and all else 448), and a remainder of far smaller values would lose bits.
struct Quotient {
  float scale, inv, by;
  __device__ __forceinline__ explicit Quotient(float s) {
    by = s < 0x1p-64f ? 0x1p96f : s > 0x1p64f ? 0x1p-96f : 1.f;
    scale = s * by;
    inv = 1.f / scale;
    if (s == INFINITY) scale = 0.f;   // q is 0 then, or NaN
  }
  __device__ __forceinline__ float operator()(float y) const {
    y *= by;
    const float q = y * inv;
    return fmaf(fmaf(-q, scale, y), inv, q);
  }
};
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t* to, const float2 (&f)[(V + 1) / 2], const Quotient& by) {
  uint32_t u[(V + 1) / 2];
#pragma unroll
  for (int k = 0; k < (V + 1) / 2; ++k) u[k] = e4m3_pair(by(f[k].x), by(f[k].y));
  if constexpr (V == 8) *reinterpret_cast<uint2*>(to) = make_uint2(u[0] | u[1] << 16, u[2] | u[3] << 16);
  else if constexpr (V == 4) *reinterpret_cast<uint32_t*>(to) = u[0] | u[1] << 16;
  else if constexpr (V == 2) *reinterpret_cast<uint16_t*>(to) = (uint16_t)u[0];
  else *to = (uint8_t)u[0];
}

__device__ __forceinline__ float scale_of(float most) {
  const float s = most / kMost;
  return s > 0.f ? s : 1.f;
}

// Rows whose vectors fit the registers: N_ vectors of V values a thread.
template <typename T, int V, int N_, int Q>
__global__ void __launch_bounds__(N_ == 1 ? 1024 : kRowThreads) rms_forward_kernel(const __grid_constant__ NormParams p) {
  using K = Pack<T, V>;
  __shared__ RowReduce sm;
  const int tpr = p.tpr, rows = blockDim.x / tpr, sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int64_t nvec = p.C / V, step = (int64_t)gridDim.x * rows;
  int64_t row = (int64_t)blockIdx.x * rows + sub;
  float2 w[N_][K::P];
  typename K::Raw x[N_], r[N_];
  const T* xp = static_cast<const T*>(p.x);
  const T* rp = static_cast<const T*>(p.res);
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int n = 0; n < N_; ++n) {
      const int64_t c = (int64_t)n * tpr + t;
      const bool in = at < p.N && c < nvec;
      x[n] = in ? K::raw(xp + at * p.xs + c * V) : K::none();
      r[n] = in && rp ? K::raw(rp + at * p.rs + c * V) : K::none();
    }
  };
  fetch(row);
#pragma unroll
  for (int n = 0; n < N_; ++n) {
    const int64_t c = (int64_t)n * tpr + t;
    if (c < nvec) K::param(p.w, c * V, 1.f, w[n]);
    else K::zero(w[n]);
  }
  const float over = 1.f / (float)p.C;
  int buf = 0;
  for (int64_t first = (int64_t)blockIdx.x * rows; first < p.N; first += step, row += step, buf ^= 1) {
    float2 h[N_][K::P];
    float s = 0.f, most = 0.f;
#pragma unroll
    for (int n = 0; n < N_; ++n) {
      float2 a[K::P], b[K::P];
      K::unpack(x[n], a);
      K::unpack(r[n], b);
#pragma unroll
      for (int k = 0; k < K::P; ++k) {
        h[n][k] = rp ? make_float2(a[k].x + b[k].x, a[k].y + b[k].y) : a[k];
        s = fmaf(h[n][k].x, h[n][k].x, s);
        s = fmaf(h[n][k].y, h[n][k].y, s);
        if (Q == SSD_QUANT_TOKEN) most = fmaxf(most, fmaxf(fabsf(h[n][k].x * w[n][k].x), fabsf(h[n][k].y * w[n][k].y)));
      }
    }
    fetch(row + step);
    row_reduce<Q == SSD_QUANT_TOKEN>(sm, buf, tpr, s, most);
    const float rstd = rsqrtf(fmaf(s, over, p.eps));
    const bool live = row < p.N;
    if (live && t == 0 && p.rstd) p.rstd[row] = rstd;
    float sc = 1.f;
    if (Q == SSD_QUANT_TOKEN) {
      sc = scale_of(most * rstd);
      if (live && t == 0) p.scale[row] = sc;
    }
#pragma unroll
    for (int n = 0; n < N_; ++n) {
      const int64_t c = (int64_t)n * tpr + t;
      const bool in = live && c < nvec;
      float2 y[K::P];
      if (in && p.h) K::store(static_cast<T*>(p.h) + row * p.C + c * V, h[n]);
#pragma unroll
      for (int k = 0; k < K::P; ++k) y[k] = make_float2(h[n][k].x * rstd * w[n][k].x, h[n][k].y * rstd * w[n][k].y);
      if constexpr (Q == SSD_QUANT_BLOCK) {   // 128 / V neighbouring lanes hold a block
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < K::P; ++k) m = fmaxf(m, fmaxf(fabsf(y[k].x), fabsf(y[k].y)));
#pragma unroll
        for (int o = kBlock / V / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        sc = scale_of(rstd == rstd ? m : 0.f);
        if (in && c % (kBlock / V) == 0) p.scale[row * p.blocks + c / (kBlock / V)] = sc;
      }
      if (!in) continue;
      if constexpr (Q == SSD_QUANT_NONE) K::store(static_cast<T*>(p.y) + row * p.C + c * V, y);
      else store_e4m3<V>(static_cast<uint8_t*>(p.y) + row * p.C + c * V, y, Quotient(sc));
    }
  }
}

__device__ __forceinline__ float block_sum(float v, float* sm) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kWideThreads / 32; ++i) s += sm[i];
  return s;
}

// Any row: a block, value by value, from global memory (the caches) for every pass.
template <typename T, int Q>
__global__ void __launch_bounds__(kWideThreads) rms_forward_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[32];
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.xs;
    const T* res = p.res ? static_cast<const T*>(p.res) + row * p.rs : nullptr;
    T* hp = p.h ? static_cast<T*>(p.h) + row * p.C : nullptr;
    auto value = [&](int64_t c) { return ld_f32(x + c) + (res ? ld_f32(res + c) : 0.f); };
    auto weight = [&](int64_t c) { return p.w ? __ldg(p.w + c) : 1.f; };
    float s = 0.f, most = 0.f;
    for (int64_t c = tid; c < p.C; c += kWideThreads) {
      const float h = value(c);
      s = fmaf(h, h, s);
      if (Q == SSD_QUANT_TOKEN) most = fmaxf(most, fabsf(h * weight(c)));
    }
    s = block_sum(s, sm);
    const float rstd = rsqrtf(fmaf(s, 1.f / (float)p.C, p.eps));
    if (tid == 0 && p.rstd) p.rstd[row] = rstd;
    float sc = 1.f;
    if (Q == SSD_QUANT_TOKEN) {
      most = warp_max(most);
      __syncthreads();
      if ((tid & 31) == 0) sm[tid >> 5] = most;
      __syncthreads();
      for (int i = 0; i < kWideThreads / 32; ++i) most = fmaxf(most, sm[i]);
      sc = scale_of(most * rstd);
      if (tid == 0) p.scale[row] = sc;
    }
    if constexpr (Q == SSD_QUANT_BLOCK) {   // a warp a block, four values a lane
      for (int64_t blk = tid >> 5; blk < p.blocks; blk += kWideThreads / 32) {
        float y[4], h[4], m = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t c = blk * kBlock + j * 32 + (tid & 31);
          h[j] = c < p.C ? value(c) : 0.f;
          y[j] = c < p.C ? h[j] * rstd * weight(c) : 0.f;
          m = fmaxf(m, fabsf(y[j]));
        }
        sc = scale_of(rstd == rstd ? warp_max(m) : 0.f);
        if ((tid & 31) == 0) p.scale[row * p.blocks + blk] = sc;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t c = blk * kBlock + j * 32 + (tid & 31);
          if (c >= p.C) continue;
          if (hp) st_from_f32(hp + c, h[j]);
          static_cast<uint8_t*>(p.y)[row * p.C + c] = (uint8_t)e4m3_pair(Quotient(sc)(y[j]), 0.f);
        }
      }
    } else {
      for (int64_t c = tid; c < p.C; c += kWideThreads) {
        const float h = value(c), y = h * rstd * weight(c);
        if (Q == SSD_QUANT_NONE) st_from_f32(static_cast<T*>(p.y) + row * p.C + c, y);
        else static_cast<uint8_t*>(p.y)[row * p.C + c] = (uint8_t)e4m3_pair(Quotient(sc)(y), 0.f);
        if (hp) st_from_f32(hp + c, h);   // the same thread has read what this may overwrite
      }
    }
  }
}

template <typename T, int V, int N_>
__global__ void __launch_bounds__(N_ == 1 ? 1024 : kRowThreads) rms_backward_kernel(const __grid_constant__ NormParams p) {
  using K = Pack<T, V>;
  __shared__ RowReduce sm;
  const int tpr = p.tpr, rows = blockDim.x / tpr, sub = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int64_t nvec = p.C / V, step = (int64_t)gridDim.x * rows;
  int64_t row = (int64_t)blockIdx.x * rows + sub;
  float2 w[N_][K::P], dw[N_][K::P];
  typename K::Raw x[N_], r[N_], d[N_];
  float rstd = 0.f;
  const T* rp = static_cast<const T*>(p.res);
  auto fetch = [&](int64_t at) {
#pragma unroll
    for (int n = 0; n < N_; ++n) {
      const int64_t c = (int64_t)n * tpr + t;
      const bool in = at < p.N && c < nvec;
      x[n] = in ? K::raw(static_cast<const T*>(p.x) + at * p.xs + c * V) : K::none();
      d[n] = in ? K::raw(static_cast<const T*>(p.dy) + at * p.ds + c * V) : K::none();
      r[n] = in && rp ? K::raw(rp + at * p.rs + c * V) : K::none();
    }
    rstd = at < p.N ? __ldg(p.rstd_in + at) : 0.f;
  };
  fetch(row);
#pragma unroll
  for (int n = 0; n < N_; ++n) {
    const int64_t c = (int64_t)n * tpr + t;
    if (c < nvec) K::param(p.w, c * V, 1.f, w[n]);
    else K::zero(w[n]);
    K::zero(dw[n]);
  }
  const float over = 1.f / (float)p.C;
  int buf = 0;
  for (int64_t first = (int64_t)blockIdx.x * rows; first < p.N; first += step, row += step, buf ^= 1) {
    float2 xh[N_][K::P], q[N_][K::P], rr[N_][K::P];
    float s = 0.f, none = 0.f;
    const float rs = rstd;
#pragma unroll
    for (int n = 0; n < N_; ++n) {
      float2 a[K::P], b[K::P];
      K::unpack(x[n], a);
      K::unpack(d[n], b);
      K::unpack(r[n], rr[n]);
#pragma unroll
      for (int k = 0; k < K::P; ++k) {
        xh[n][k] = make_float2(a[k].x * rs, a[k].y * rs);
        dw[n][k].x = fmaf(b[k].x, xh[n][k].x, dw[n][k].x);
        dw[n][k].y = fmaf(b[k].y, xh[n][k].y, dw[n][k].y);
        q[n][k] = make_float2(b[k].x * w[n][k].x, b[k].y * w[n][k].y);
        s = fmaf(q[n][k].x, xh[n][k].x, s);
        s = fmaf(q[n][k].y, xh[n][k].y, s);
      }
    }
    fetch(row + step);
    row_reduce<false>(sm, buf, tpr, s, none);
    const float mean = s * over;
#pragma unroll
    for (int n = 0; n < N_; ++n) {
      const int64_t c = (int64_t)n * tpr + t;
      float2 dx[K::P];
#pragma unroll
      for (int k = 0; k < K::P; ++k)
        dx[k] = make_float2(fmaf(rs, fmaf(-xh[n][k].x, mean, q[n][k].x), rr[n][k].x),
                            fmaf(rs, fmaf(-xh[n][k].y, mean, q[n][k].y), rr[n][k].y));
      if (row < p.N && c < nvec && SSD_INDEX_OK(p.hdr, row * p.C + c * V + V - 1, p.N * p.C, 2101))
        K::store(static_cast<T*>(p.y) + row * p.C + c * V, dx);
    }
  }
  if (!p.partial) return;
  float* part = p.partial + ((int64_t)blockIdx.x * rows + sub) * p.C;
#pragma unroll
  for (int n = 0; n < N_; ++n) {
    const int64_t c = (int64_t)n * tpr + t;
    if (c >= nvec || !SSD_INDEX_OK(p.hdr, part - p.partial + c * V + V - 1, p.part_rows * p.C, 2102)) continue;
#pragma unroll
    for (int k = 0; k < K::P; ++k) {
      part[c * V + 2 * k] = dw[n][k].x;
      if (V > 1) part[c * V + 2 * k + 1] = dw[n][k].y;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) rms_backward_wide_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[32];
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.xs;
    const T* dy = static_cast<const T*>(p.dy) + row * p.ds;
    const T* res = p.res ? static_cast<const T*>(p.res) + row * p.rs : nullptr;
    const float rstd = __ldg(p.rstd_in + row);
    auto weight = [&](int64_t c) { return p.w ? __ldg(p.w + c) : 1.f; };
    float s = 0.f;
    for (int64_t c = tid; c < p.C; c += kWideThreads) s = fmaf(ld_f32(dy + c) * weight(c), ld_f32(x + c) * rstd, s);
    const float mean = block_sum(s, sm) / (float)p.C;
    for (int64_t c = tid; c < p.C; c += kWideThreads) {
      const float xh = ld_f32(x + c) * rstd, q = ld_f32(dy + c) * weight(c);
      if (SSD_INDEX_OK(p.hdr, row * p.C + c, p.N * p.C, 2103)) st_from_f32(static_cast<T*>(p.y) + row * p.C + c, fmaf(rstd, fmaf(-xh, mean, q), res ? ld_f32(res + c) : 0.f));
    }
  }
}

// Sums of dw over a share of the rows, for rows too wide for the registers: a thread a channel.
template <typename T>
__global__ void __launch_bounds__(128) rms_weight_grad_kernel(const __grid_constant__ NormParams p, int64_t per) {
  const int64_t c = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (c >= p.C) return;
  const int64_t end = min(p.N, (blockIdx.y + 1) * per);
  float s = 0.f;
  for (int64_t row = blockIdx.y * per; row < end; ++row)
    s = fmaf(ld_f32(static_cast<const T*>(p.dy) + row * p.ds + c),
             ld_f32(static_cast<const T*>(p.x) + row * p.xs + c) * __ldg(p.rstd_in + row), s);
  if (SSD_INDEX_OK(p.hdr, blockIdx.y * p.C + c, p.part_rows * p.C, 2104)) p.partial[blockIdx.y * p.C + c] = s;
}

// dw from the partial rows, in a fixed order: 32 channels a block, 32 threads a channel.
__global__ void __launch_bounds__(1024) rms_join_kernel(const float* partial, float* dw, int64_t rows, int64_t C,
                                                        WsHeader* hdr) {
  __shared__ float sm[32][33];
  follow();
  const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const int part = threadIdx.x >> 5;
  float s = 0.f;
  if (c < C)
    for (int64_t r = part; r < rows; r += 32) s += partial[r * C + c];
  sm[part][threadIdx.x & 31] = s;
  __syncthreads();
  s = warp_sum(sm[threadIdx.x & 31][part]);
  const int64_t to = (int64_t)blockIdx.x * 32 + part;
  if ((threadIdx.x & 31) == 0 && to < C && SSD_INDEX_OK(hdr, to, C, 2105)) dw[to] = s;
}

// ------------------------------------------------------------------------------------------------ host
bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
ssd_status done(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

ssd_status check_shape(const rms_norm_shape* s, bool back) {
  if (!s || s->rows < 0 || s->channels < 1 || s->x_stride < 0 || s->res_stride < 0 || (back && s->dy_stride < 0))
    return SSD_ERR_INVALID_ARG;
  if (!(s->eps >= 0.f) || !isfinite(s->eps)) return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_F32 && s->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (!back && (s->quantize < SSD_QUANT_NONE || s->quantize > SSD_QUANT_BLOCK)) return SSD_ERR_INVALID_ARG;
  if (s->channels > INT32_MAX || (s->rows > 0 && s->channels > INT64_MAX / 16 / s->rows)) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

// Vectors of the widest size that every row starts on and C divides, threads a row and vectors a thread; 0 vectors:
// a row does not fit the registers.  At most 256 threads a row where more vectors a thread avoid more (us, forward and
// backward of bf16 rows: 10007 x 2560 by 160 threads 43 / 45, by 320 45 / 56; 16384 x 4096 by 256 90 / 83, by 512 88 / 120;
// 4000 x 8192 by 256 45, by 512 49), and no fewer than one vector needs (16384 x 2048 by 256 46 / 52, by 128 47 / 51).
struct Form {
  int v, n, tpr, rows;
};
Form form_of(uint64_t bits, size_t e, int64_t C, int most_n, bool block_scales) {
  Form f = {1, 0, 32, 1};
  for (int v = 16 / (int)e; v > 1; v /= 2)
    if (bits % (v * e) == 0 && C % v == 0 && v != (e == 2 ? 4 : 2)) {
      f.v = v;
      break;
    }
  if (block_scales && kBlock / f.v > 32) return f;
  const int64_t nvec = C / f.v;
  for (int n = 1; n <= most_n; n *= 2) {
    const int64_t tpr = ((nvec + n - 1) / n + 31) / 32 * 32;
    if (tpr > (n < most_n ? kRowThreads / 2 : kRowThreads)) continue;
    f.n = n;
    f.tpr = (int)tpr;
    break;
  }
  f.rows = std::max(1, 256 / f.tpr);
  return f;
}

constexpr int64_t kMaxPartials = 152 * 8;   // partial rows of dw, however many rows there are

template <typename T, int Q>
cudaError_t launch_forward(NormParams p, uint64_t bits, cudaStream_t st) {
  const Form f = form_of(bits, sizeof(T), p.C, 4, Q == SSD_QUANT_BLOCK);
  if (f.n == 0) {
    rms_forward_wide_kernel<T, Q><<<(unsigned)std::min<int64_t>(p.N, 152 * 4), kWideThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  p.tpr = f.tpr;
  const int threads = f.tpr * f.rows;
  void (*kernel)(NormParams) = nullptr;
  constexpr int W = 16 / (int)sizeof(T);
  auto pick = [&](auto v) {
    constexpr int V = decltype(v)::value;
    if constexpr (Q != SSD_QUANT_BLOCK || kBlock / V <= 32)
      kernel = f.n == 1 ? rms_forward_kernel<T, V, 1, Q> : f.n == 2 ? rms_forward_kernel<T, V, 2, Q> : rms_forward_kernel<T, V, 4, Q>;
  };
  if (f.v == W) pick(std::integral_constant<int, W>{});
  else if (f.v == 1) pick(std::integral_constant<int, 1>{});
  else if constexpr (sizeof(T) == 2) pick(std::integral_constant<int, 2>{});
  int most = 0;
  cudaError_t e = resident_blocks(kernel, threads, 0, &most);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)std::min<int64_t>((p.N + f.rows - 1) / f.rows, most), threads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_backward(NormParams p, uint64_t bits, cudaStream_t st) {
  const Form f = form_of(bits, sizeof(T), p.C, 2, false);
  cudaError_t e;
  int64_t partials;
  if (f.n == 0) {
    rms_backward_wide_kernel<T><<<(unsigned)std::min<int64_t>(p.N, 152 * 4), kWideThreads, 0, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || !p.dw) return e;
    const int64_t cols = (p.C + 127) / 128;
    partials = std::max<int64_t>(1, std::min<int64_t>({p.N, 152 * 8 / cols, kMaxPartials}));
    const int64_t per = (p.N + partials - 1) / partials;
    partials = (p.N + per - 1) / per;
    rms_weight_grad_kernel<T><<<dim3((unsigned)cols, (unsigned)partials), 128, 0, st>>>(p, per);
    e = cudaGetLastError();
  } else {
    p.tpr = f.tpr;
    const int threads = f.tpr * f.rows;
    void (*kernel)(NormParams) = nullptr;
    constexpr int W = 16 / (int)sizeof(T);
    auto pick = [&](auto v) {
      constexpr int V = decltype(v)::value;
      kernel = f.n == 1 ? rms_backward_kernel<T, V, 1> : rms_backward_kernel<T, V, 2>;
    };
    if (f.v == W) pick(std::integral_constant<int, W>{});
    else if (f.v == 1) pick(std::integral_constant<int, 1>{});
    else if constexpr (sizeof(T) == 2) pick(std::integral_constant<int, 2>{});
    int most = 0;
    e = resident_blocks(kernel, threads, 0, &most);
    if (e != cudaSuccess) return e;
    const int64_t grid = std::min<int64_t>({(p.N + f.rows - 1) / f.rows, (int64_t)most, kMaxPartials / f.rows});
    partials = grid * f.rows;
    kernel<<<(unsigned)grid, threads, 0, st>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !p.dw) return e;
  return launch_next(rms_join_kernel, dim3((unsigned)((p.C + 31) / 32)), 1024, 0, st, (const float*)p.partial, p.dw,
                     partials, p.C, p.hdr);
}

int64_t partial_rows(const rms_norm_shape* s) { return std::min(std::max<int64_t>(s->rows, 1) + 7, kMaxPartials); }
size_t workspace_total(const rms_norm_shape* s) {
  return sizeof(WsHeader) + align_up((size_t)partial_rows(s) * (size_t)s->channels * 4, kWsAlign);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t rms_norm_workspace_bytes(const rms_norm_shape* shape) {
  if (check_shape(shape, true) != SSD_OK) return 0;
  return workspace_total(shape);
}

ssd_status rms_norm_forward(const rms_norm_shape* shape, const void* x, const void* residual, const float* weight,
                            void* y, void* h, float* rstd, float* scale, void* stream) {
  const ssd_status bad = check_shape(shape, false);
  if (bad != SSD_OK) return bad;
  if (shape->rows == 0) return SSD_OK;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  const int32_t q = shape->quantize;
  if (!x || !y || (q != SSD_QUANT_NONE && !scale)) return SSD_ERR_INVALID_ARG;
  if (misaligned(x, e) || misaligned(residual, e) || misaligned(h, e) || (q == SSD_QUANT_NONE && misaligned(y, e)) ||
      misaligned(weight, 4) || misaligned(rstd, 4) || misaligned(scale, 4))
    return SSD_ERR_INVALID_ARG;
  NormParams p;
  memset(&p, 0, sizeof(p));
  p.x = x;
  p.res = residual;
  p.w = weight;
  p.y = y;
  p.h = h;
  p.rstd = rstd;
  p.scale = scale;
  p.N = shape->rows;
  p.C = shape->channels;
  p.xs = shape->x_stride;
  p.rs = shape->res_stride;
  p.eps = shape->eps;
  p.blocks = q == SSD_QUANT_BLOCK ? (p.C + kBlock - 1) / kBlock : 1;
  const uint64_t outs = reinterpret_cast<uintptr_t>(h) | (q == SSD_QUANT_NONE ? reinterpret_cast<uintptr_t>(y) : reinterpret_cast<uintptr_t>(y) * e);
  const uint64_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) | outs |
                        (uint64_t)(p.xs | (residual ? p.rs : 0)) * e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (bf16)
    return done(q == SSD_QUANT_NONE    ? launch_forward<__nv_bfloat16, SSD_QUANT_NONE>(p, bits, st)
                : q == SSD_QUANT_TOKEN ? launch_forward<__nv_bfloat16, SSD_QUANT_TOKEN>(p, bits, st)
                                       : launch_forward<__nv_bfloat16, SSD_QUANT_BLOCK>(p, bits, st));
  return done(q == SSD_QUANT_NONE    ? launch_forward<float, SSD_QUANT_NONE>(p, bits, st)
              : q == SSD_QUANT_TOKEN ? launch_forward<float, SSD_QUANT_TOKEN>(p, bits, st)
                                     : launch_forward<float, SSD_QUANT_BLOCK>(p, bits, st));
}

ssd_status rms_norm_backward(const rms_norm_shape* shape, const void* h, const void* dy, const float* rstd,
                             const float* weight, const void* dresidual, void* dx, float* dweight, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const ssd_status bad = check_shape(shape, true);
  if (bad != SSD_OK) return bad;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  if (shape->rows > 0 && (!h || !dy || !rstd || !dx)) return SSD_ERR_INVALID_ARG;
  if (misaligned(h, e) || misaligned(dy, e) || misaligned(dresidual, e) || misaligned(dx, e) || misaligned(rstd, 4) ||
      misaligned(weight, 4) || misaligned(dweight, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, kWsAlign) || workspace_bytes < workspace_total(shape)) return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->rows == 0)
    return done(dweight ? cudaMemsetAsync(dweight, 0, (size_t)shape->channels * 4, st) : cudaSuccess);
  NormParams p;
  memset(&p, 0, sizeof(p));
  p.x = h;
  p.dy = dy;
  p.rstd_in = rstd;
  p.w = weight;
  p.res = dresidual;
  p.y = dx;
  p.dw = dweight;
  p.hdr = static_cast<WsHeader*>(workspace);
  p.part_rows = partial_rows(shape);
  p.partial = dweight ? reinterpret_cast<float*>(static_cast<char*>(workspace) + sizeof(WsHeader)) : nullptr;
  p.N = shape->rows;
  p.C = shape->channels;
  p.xs = shape->x_stride;
  p.rs = shape->res_stride;
  p.ds = shape->dy_stride;
  const uint64_t bits = reinterpret_cast<uintptr_t>(h) | reinterpret_cast<uintptr_t>(dy) |
                        reinterpret_cast<uintptr_t>(dresidual) | reinterpret_cast<uintptr_t>(dx) |
                        (uint64_t)(p.xs | p.ds | (dresidual ? p.rs : 0)) * e;
  return done(bf16 ? launch_backward<__nv_bfloat16>(p, bits, st) : launch_backward<float>(p, bits, st));
}

}  // extern "C"
