// Carry of an elementwise linear recurrence along tiles that run on different blocks: a decoupled
// look-back (Merrill and Garland, Single-pass Parallel Prefix Scan with Decoupled Look-back, 2016) whose
// words hold a value and its state together, so that no fence is needed.
//
// A step, or a span of steps, maps the state before it, h, to a h + H.  Its decay a in [0, 1] is kept as one
// number c: near one as c = a - 1 < 0 (a itself has an absolute rounding error of 2^-25 that a channel with
// memory 1 / (1 - a) multiplies by that memory), and where a is small as c = a >= 0 (h + ((a - 1) h + H)
// would leave the rounding of a large h behind, 2^-24 |h|, where a h is long gone).  No decay is exactly
// one: c <= -kTiny.
//
// A tile's word is 64 bits: H in the low half, c, with |c| <= 1, in the high half, whose bit 30 (the top bit of
// the exponent) is free and set in every word that holds anything (the words are cleared before the
// launch).  An inclusive word, whose H is the state after the tile, has c = -0, which no map has: as a map
// it gives H whatever came before.  A reader evaluates the maps from the nearest inclusive word on,
// oldest first, with the very operations that made the inclusive words: the result has the same bits
// wherever it starts.
#pragma once

#include "common.cuh"
#include "fp_helpers.cuh"

namespace ssd {
namespace lookback {

constexpr uint32_t kMap = 1u << 30, kInclusive = 3u << 30;
constexpr float kInf = __builtin_huge_valf();

// a h + H.  NaN for an infinite h: inf - inf next to one, 0 inf where a is small.
__device__ __forceinline__ float apply(float c, float H, float h) {
  return fmaf(c < 0.f ? 1.f : 0.f, h, fmaf(c, h, H));
}
// The same, but an infinite h stays what it is (no decay is zero, if fp32 makes it so).  Where the results of
// a chain of apply are not NaN, this chain's are the same.
__device__ __forceinline__ float apply_safe(float c, float H, float h) { return fabsf(h) == kInf ? h + H : apply(c, H, h); }

__device__ __forceinline__ uint64_t inclusive(float h) { return ((uint64_t)kInclusive << 32) | __float_as_uint(h); }
__device__ __forceinline__ uint64_t map(float c, float H) {
  if (c != c) H = c, c = 0.f;   // a NaN decay: the state after it is NaN whatever came before
  return ((uint64_t)(__float_as_uint(c) | kMap) << 32) | __float_as_uint(H);
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
// bounded (1 s, then SSD_ERR_TIMEOUT is latched and the call's results are void).  Maps evaluated behind an
// infinite state, inclusive ones among them, may give a NaN that is none: with a NaN the try is not over
// before the nearest is inclusive.
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
    bool known = true, some = true;   // the nearest words are inclusive, hold anything
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const uint32_t hi = (uint32_t)(v[0][c] >> 32);
      known = known && hi == kInclusive;
      some = some && hi != 0;
      h[c] = __uint_as_float((uint32_t)v[0][c]);
    }
    if (__all_sync(0xffffffffu, known)) return;
    if (__all_sync(0xffffffffu, some)) {
      bool all = true;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        bool ok = false;
        h[c] = 0.f;
#pragma unroll
        for (int j = K - 1; j >= 0; --j) {
          const uint32_t hi = (uint32_t)(v[j][c] >> 32);
          const float H = __uint_as_float((uint32_t)v[j][c]), a = __uint_as_float(hi & ~kMap);
          h[c] = apply(a, H, h[c]);
          ok = hi == kInclusive || (ok && hi != 0);
        }
        all = all && ok && h[c] == h[c];
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
