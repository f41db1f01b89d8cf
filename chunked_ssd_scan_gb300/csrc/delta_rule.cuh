// What the kernels of the gated delta rule share (declarations in include/ssdscan.h).
#pragma once

#include <math.h>

#include "common.cuh"

namespace ssd {
namespace delta {

constexpr int kChunk = GATED_DELTA_RULE_CHUNK;
constexpr float kNoDecay = -200.f;   // e^-200 is zero in fp32; keeps differences of sums of g finite

struct Params {
  const void *q, *k, *v, *dy;
  const float *g, *beta, *init, *dfinal;
  const float* states_in;              // before every chunk (backward)
  void *y, *dq, *dk, *dv;
  float *final_state, *states_out, *dg, *dbeta, *dinit;
  float *err, *du;                     // [b,T,H,V]: v - S k of every step; gradient of u
  float* dstates;                      // [b,nch,H,V,K]: gradient of the state before every chunk
  float* partial;                      // [key blocks][b*nch*H][kChunk + 1]
  int64_t batch, T, Hk, H, K, V, nch;
  int64_t qs[3], ks[3], vs[3], ds[3], gs[2], bs[2];
  int64_t slices;                      // blocks side by side in V
  float scale;
  WsHeader* hdr;
};

__device__ __forceinline__ float decay_log(const Params& p, int64_t b, int64_t t, int64_t h) {
  const float g = p.g ? __ldg(p.g + b * p.gs[0] + t * p.gs[1] + h) : 0.f;
  return g < kNoDecay ? kNoDecay : g;
}

// Sums of g within a chunk as pairs of floats (double in parts), and what they make of it: thread i < 64 of
// the first two warps holds step i's g.  `last` is the chunk's last step.
struct ChunkDecay {
  float hi[kChunk], lo[kChunk];   // sum of g over the chunk's steps up to i
  float beta[kChunk];
  float from[kChunk], to[kChunk]; // e^(sum up to i), e^(sum behind i)
};

__device__ __forceinline__ float decay_between(const ChunkDecay& c, int i, int j) {   // j <= i
  return expf((c.hi[i] - c.hi[j]) + (c.lo[i] - c.lo[j]));
}

// By one whole warp; lane l holds the steps 2l and 2l + 1.
__device__ __forceinline__ void chunk_decay_warp(const Params& p, ChunkDecay& c, int64_t b, int64_t t0, int n,
                                                 int64_t h, int lane) {
  const int i0 = 2 * lane, i1 = i0 + 1;
  const double g0 = i0 < n ? (double)decay_log(p, b, t0 + i0, h) : 0.0;
  const double g1 = i1 < n ? (double)decay_log(p, b, t0 + i1, h) : 0.0;
  double sum = g0 + g1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double up = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += up;
  }
  const double total = __shfl_sync(0xffffffffu, sum, 31);
  const double c0 = sum - g1, c1 = sum;
  c.hi[i0] = (float)c0;
  c.lo[i0] = (float)(c0 - (double)(float)c0);
  c.hi[i1] = (float)c1;
  c.lo[i1] = (float)(c1 - (double)(float)c1);
  c.from[i0] = expf((float)c0);
  c.from[i1] = expf((float)c1);
  c.to[i0] = expf((float)(total - c0));
  c.to[i1] = expf((float)(total - c1));
  const float* bp = p.beta + b * p.bs[0] + h;
  c.beta[i0] = i0 < n ? __ldg(bp + (t0 + i0) * p.bs[1]) : 0.f;
  c.beta[i1] = i1 < n ? __ldg(bp + (t0 + i1) * p.bs[1]) : 0.f;
}

}  // namespace delta
}  // namespace ssd
