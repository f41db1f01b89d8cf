// Group norm with an activation, channels last: what its translation units share.
#pragma once

#include <math.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "common.cuh"
#include "fp_helpers.cuh"
#include "launch.h"
#include "pack.cuh"

namespace ssd {
namespace norm {

struct NormParams {
  const void *x, *dy;
  const float *w, *bias, *mean_in, *rstd_in;
  void *y, *dx;
  float *mean, *rstd, *dw, *db;
  int64_t N, S, C, G, cg;
  int64_t xs[2], ds[2];
  float eps;
  int32_t act;
  int32_t lanes;        // token kernels: lanes of a group
  int32_t tile_groups;  // map kernels: groups of a column tile
  int32_t chunks;       // map kernels: pieces that a sample's positions are cut into
  int64_t chunk_rows;
  int64_t slots;        // map gradient sums: samples that are worked on side by side
  float *stats;         // map kernels: [N, G, chunks, 2], mean and M2 or the two gradient sums
  float *joined;        // [N, G, 2]
  float *part_w, *part_b;   // rows of parameter gradient partials [part_rows, C]
  int64_t part_rows;
  WsHeader* hdr;
};

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGridBlocks = 152;        // blocks that a map kernel is cut into: so many times what fits an SM
constexpr int kMapForward = 4, kMapBackward = 3;   // blocks of a map kernel on an SM
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
// The sigmoid by approximations: 2^x is good to 2^-22, its argument z log2 e adds |z| 2^-23 to e^-z, 1/x to 2^-23,
// so SiLU to about 2^-21 of itself.  The exact functions are several instructions each, of which the
// kernels issue 12 to 24 a value in all.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + e^-z)
__device__ __forceinline__ float2 sigmoid2(float2 z) {
  const float2 t = fp::mul2(z, dup(-kLog2e));
  const float2 d = fp::add2(make_float2(fp::ex2_approx(t.x), fp::ex2_approx(t.y)), dup(1.f));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
template <bool kSilu>
__device__ __forceinline__ float2 act2(float2 z) {
  return kSilu ? fp::mul2(z, sigmoid2(z)) : z;
}
// v act'(z); silu' = s + z (s - s^2)
template <bool kSilu>
__device__ __forceinline__ float2 times_act_grad2(float2 v, float2 z) {
  if (!kSilu) return v;
  const float2 s = sigmoid2(z);
  const float2 ss = fp::fma2(fp::mul2(s, dup(-1.f)), s, s);
  return fp::mul2(v, fp::fma2(z, ss, s));
}

// a - b, and 0 in the second place of a single value
template <int V>
__device__ __forceinline__ float2 minus2(float2 a, float b) {
  float2 d = fp::add2(a, dup(-b));
  if (V == 1) d.y = 0.f;
  return d;
}

constexpr int kTokenBlocks = 152 * 4;   // most blocks of the token backward, which writes a partial row each
constexpr int kTokenWidth = 4 * kThreads;   // vectors of a group that a token kernel holds in registers
// Most samples that a map kernel's gradient sums take side by side, each with a partial row: twice what the
// machine holds of its blocks.  Beyond it a block goes on to further samples and adds to its row (a row for
// every sample took 461 MB, now 55 MB, for 100000 x 2 x 512 bf16, and 2610 us, now 2455).
constexpr int kMapRows = 2 * kGridBlocks * kMapBackward;

// dweight and dbias of 32 channels from the partial rows, by a block of 32 warps: a warp adds every 32nd
// row, eight loads of each array in flight, and the warps are joined in their order.
static __device__ __forceinline__ void param_grad(const NormParams& p, int64_t cols) {
  __shared__ float2 sums[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = cols * 32 + lane;
  float2 s = make_float2(0.f, 0.f);
  if (c < p.C) {
    constexpr int U = 8;
    for (int64_t r = warp; r < p.part_rows; r += 32 * U) {
      const float *pw = p.part_w + r * p.C + c, *pb = p.part_b + r * p.C + c;
      float2 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = r + 32 * u < p.part_rows ? make_float2(__ldcg(pw + u * 32 * p.C), __ldcg(pb + u * 32 * p.C))
                                        : make_float2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < U; ++u) s = fp::add2(s, v[u]);
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.C) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 32; ++k) v = fp::add2(v, sums[k][lane]);
    if (p.dw) p.dw[c] = v.x;
    if (p.db) p.db[c] = v.y;
  }
}
static __global__ void __launch_bounds__(1024) norm_param_grad_kernel(NormParams p) {
  follow();
  param_grad(p, blockIdx.x);
}

// Joins the partial rows of the parameters' gradients.
static cudaError_t launch_param_grad(const NormParams& p, cudaStream_t st) {
  if (p.part_rows == 0) return cudaSuccess;
  return launch_next(norm_param_grad_kernel, dim3((unsigned)((p.C + 31) / 32)), 1024, 0, st, p);
}

// Runs a call with one position a sample whose rows start on 16 bytes, groups of kStraddleLeast bytes to
// kThreads channels, none of the vectors that divide them wider than 4 bytes.
constexpr int kStraddleLeast = 16;
template <typename T>
cudaError_t run_straddle(const NormParams& p, bool backward, cudaStream_t st);

// Runs a call with one position a sample; a group is at most kTokenWidth vectors of V values.
template <typename T, int V>
cudaError_t run_tokens(const NormParams& p, bool backward, cudaStream_t st);

}  // namespace norm
}  // namespace ssd
