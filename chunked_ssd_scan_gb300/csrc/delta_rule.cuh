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
  float* partial;                      // [key blocks][b*nch*H][kChunk]: of dg
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

// Sums of g within a chunk as pairs of floats, and what they make of it.
struct ChunkDecay {
  float hi[kChunk], lo[kChunk];   // sum of g over the chunk's steps up to i
  float beta[kChunk];
  float from[kChunk], to[kChunk]; // e^(sum up to i), e^(sum behind i)
  float back[kChunk];             // e^-(sum up to i)
  int plain;                      // whether no sum of the chunk is beyond e^+-80: from[i] back[j] is the decay between
};

__device__ __forceinline__ float decay_between(const ChunkDecay& c, int i, int j) {   // j <= i
  return expf((c.hi[i] - c.hi[j]) + (c.lo[i] - c.lo[j]));
}

// (hi, lo) += (h, l): the exact sum of the first parts, and what its rounding left with the second ones.
__device__ __forceinline__ void add_pair(float& hi, float& lo, float h, float l) {
  const float s = hi + h, back = s - hi, rest = (hi - (s - back)) + (h - back) + (lo + l);
  hi = s + rest;
  lo = rest - (hi - s);
}

// e^(hi + lo).  (Without lo, up to half a step of hi, a decay between neighbours was off by up to 7.6e-6 at sums near 80.)
__device__ __forceinline__ float exp_pair(float hi, float lo) { return expf(hi) * (1.f + lo); }

// By one whole warp; lane l holds the steps 2l and 2l + 1.
__device__ __forceinline__ void chunk_decay_warp(const Params& p, ChunkDecay& c, int64_t b, int64_t t0, int n,
                                                 int64_t h, int lane) {
  const int i0 = 2 * lane, i1 = i0 + 1;
  const float g0 = i0 < n ? decay_log(p, b, t0 + i0, h) : 0.f, g1 = i1 < n ? decay_log(p, b, t0 + i1, h) : 0.f;
  // sums as pairs of floats (in fp64 this scan alone took 5000 cycles)
  float hi = g0, lo = 0.f;
  add_pair(hi, lo, g1, 0.f);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float uh = __shfl_up_sync(0xffffffffu, hi, o), ul = __shfl_up_sync(0xffffffffu, lo, o);
    if (lane >= o) add_pair(hi, lo, uh, ul);
  }
  const float th = __shfl_sync(0xffffffffu, hi, 31), tl = __shfl_sync(0xffffffffu, lo, 31);
  float h0 = hi, l0 = lo;
  add_pair(h0, l0, -g1, 0.f);
  c.hi[i0] = h0;
  c.lo[i0] = l0;
  c.hi[i1] = hi;
  c.lo[i1] = lo;
  c.from[i0] = exp_pair(h0, l0);
  c.from[i1] = exp_pair(hi, lo);
  c.back[i0] = exp_pair(-h0, -l0);
  c.back[i1] = exp_pair(-hi, -lo);
  const bool plain = __all_sync(0xffffffffu, fabsf(h0) <= 80.f && fabsf(hi) <= 80.f);
  if (lane == 0) c.plain = plain;
  c.to[i0] = expf((th - h0) + (tl - l0));
  c.to[i1] = expf((th - hi) + (tl - lo));
  const float* bp = p.beta + b * p.bs[0] + h;
  c.beta[i0] = i0 < n ? __ldg(bp + (t0 + i0) * p.bs[1]) : 0.f;
  c.beta[i1] = i1 < n ? __ldg(bp + (t0 + i1) * p.bs[1]) : 0.f;
}

}  // namespace delta
}  // namespace ssd
