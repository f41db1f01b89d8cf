// Carry of an elementwise linear recurrence along tiles that run on different blocks: a decoupled
// look-back whose words hold a value and its state together, so that no fence is needed.
//
// A tile of steps maps the state before it, h, to h + W h + H (W + 1 the product of its decays, kept
// minus one: W lies in [-1, 0]).  Its word is 64 bits: H in the low half, |W| in the high half,
// whose two top bits are free (|W| <= 1) and hold the word's state: 0 nothing (the words are
// cleared before the launch), 1 the tile's own map, 2 inclusive (H is the state after the tile).
// A reader evaluates the maps from the nearest inclusive word on, oldest first, with the very
// operations that made the inclusive words: the result has the same bits wherever it starts.
#pragma once

#include "common.cuh"
#include "fp_helpers.cuh"

namespace ssd {
namespace lookback {

constexpr uint32_t kMap = 1u, kInclusive = 2u;

__device__ __forceinline__ float apply(float W, float H, float h) { return h + fmaf(W, h, H); }

__device__ __forceinline__ float2 apply(float2 W, float2 H, float2 h) { return fp::add2(h, fp::fma2(W, h, H)); }

__device__ __forceinline__ uint64_t word(float W, float H, uint32_t state) {
  if (W != W) H = W, W = 0.f;   // a NaN decay: the state after it is NaN whatever came before
  const uint32_t hi = (__float_as_uint(W) & 0x3fffffffu) | (state << 30);
  return ((uint64_t)hi << 32) | __float_as_uint(H);
}

__device__ __forceinline__ void publish(uint64_t* p, const uint64_t (&v)[1]) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v[0]) : "memory");
}
__device__ __forceinline__ void publish(uint64_t* p, const uint64_t (&v)[2]) {
  asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};" ::"l"(p), "l"(v[0]), "l"(v[1]) : "memory");
}
__device__ __forceinline__ void peek(const uint64_t* p, uint64_t (&v)[1]) {
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v[0]) : "l"(p) : "memory");
}
__device__ __forceinline__ void peek(const uint64_t* p, uint64_t (&v)[2]) {
  asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "l"(p) : "memory");
}

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// State before a tile, for a warp whose lanes own N channels each: `words` is the lane's word of the
// nearest tile before it, `step` the (signed) distance in words to the next older one and `have`
// how many older tiles there are (at least one).  A try reads the K nearest words at once; the nearest is
// enough if it is inclusive, and the others are evaluated only once it holds anything.  The wait is
// bounded (1 s, then SSD_ERR_TIMEOUT is latched and the call's results are void).
template <int K, int N>
__device__ __forceinline__ void state_before(const uint64_t* words, int64_t step, int64_t have, float (&h)[N],
                                             WsHeader* hdr, int64_t site) {
  uint64_t t0 = 0;
  for (int tries = 0;; ++tries) {
    uint64_t v[K][N];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j < have) {
        peek(words + j * step, v[j]);
      } else {
#pragma unroll
        for (int c = 0; c < N; ++c) v[j][c] = 0;
      }
    }
    uint32_t least = kInclusive;   // the nearest words' least state
#pragma unroll
    for (int c = 0; c < N; ++c) {
      least = min(least, (uint32_t)(v[0][c] >> 62));
      h[c] = __uint_as_float((uint32_t)v[0][c]);
    }
    if (__all_sync(0xffffffffu, least == kInclusive)) return;
    if (__all_sync(0xffffffffu, least != 0)) {
      bool all = true;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        bool ok = false;
        h[c] = 0.f;
#pragma unroll
        for (int j = K - 1; j >= 0; --j) {
          const uint32_t hi = (uint32_t)(v[j][c] >> 32), state = hi >> 30;
          const float H = __uint_as_float((uint32_t)v[j][c]);
          const float W = -__uint_as_float(hi & 0x3fffffffu);
          h[c] = state == kInclusive ? H : apply(W, H, h[c]);
          ok = state == kInclusive || (ok && state == kMap);
        }
        all = all && ok;
      }
      if (__all_sync(0xffffffffu, all)) return;
    }
    if ((tries & 255) == 255) {
      const uint64_t t = now_ns();
      if (t0 == 0) t0 = t;
      const bool late = t - t0 > 1000000000ull;
      if (__any_sync(0xffffffffu, late)) {
        if (threadIdx.x % 32 == 0) latch_error(hdr, SSD_ERR_TIMEOUT, site);
        return;
      }
    }
  }
}

}  // namespace lookback
}  // namespace ssd
