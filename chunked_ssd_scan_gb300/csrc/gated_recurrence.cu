// Gated linear recurrence, elementwise per channel (declarations in include/ssdscan.h):
//   h_t = a_t h_{t-1} + m_t i_t x_t,  a = e^l, l = -c softplus(decay) sigmoid(gate_a),
//   m = sqrt(1 - a^2) = sqrt(-expm1(2 l)), i = sigmoid(gate_x)
// and its reverse mode, G_t = dy_t + a_{t+1} G_{t+1}:
//   dx = G m i; dgate_x = G m x i (1 - i); k = a (h_{t-1} - a i x / m);
//   dgate_a = G k l (1 - r); ddecay = sum G k (-c r) sigmoid(decay).
#include <math.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "fp_helpers.cuh"
#include "launch.h"
#include "lookback.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace ssd {
namespace {

constexpr int kChunk = GATED_RECURRENCE_CHUNK;

struct RecParams {
  CUtensorMap map[4];   // x, gate_a, gate_x, dy in tiles (TMA kernels)
  const void *x, *ga, *gx, *dy;
  const float *decay, *init, *states_in, *dfinal;
  void *y, *dx, *dga, *dgx;
  float *final_state, *states_out, *ddecay, *dinit, *partial;
  int64_t batch, T, D, nch;
  int64_t xs[2], as[2], gs[2], ds[2];
  float c;
  int64_t ntile;     // tiles in time
  uint32_t cols;     // tiles side by side in the channels of one sequence
  uint32_t tiles;    // tiles in all
  uint32_t* ticket;  // tickets taken, blocks done; NULL where the order of the tiles does not matter
  uint64_t* words;
  WsHeader* hdr;
};

__device__ __forceinline__ float softplus(float d) { return fmaxf(d, 0.f) + log1pf(expf(-fabsf(d))); }

// A decay is kept as one number c (lookback.cuh): a - 1 = expm1(l) < 0 next to one, where a step is
// h + (c h + b), and a itself below e^-1/4, where it is c h + b.  A warp whose channels cannot decay
// faster than e^-1/4 a step does the first for all its values; others choose value by value (8 x 4096 x
// 2048 bf16: 111 us forward, 234 us backward, where the first takes 103 and 215).  Both make NaN of an
// infinite state next to one (inf - inf): an odd tile, one that meets values of kHuge or more, or NaN, is finished
// by a function that goes through its steps once more, one by one, in a third form that does not (all tiles
// odd: 217 us forward).  It is called, not part of the kernels: with its code inline they ran out of
// registers (forward 145 us).
constexpr float kInf = lookback::kInf;
enum Form { kSlow, kMixed, kSafe };
template <int F>
__device__ __forceinline__ float step(float c, float b, float h) {   // a h + b
  if (F == kSafe) return lookback::apply_safe(c, b, h);
  if (F == kMixed) return lookback::apply(c, b, h);
  return h + fmaf(c, h, b);
}
template <int F>
__device__ __forceinline__ float2 step(float2 c, float2 b, float2 h) {
  if (F == kSafe) return make_float2(lookback::apply_safe(c.x, b.x, h.x), lookback::apply_safe(c.y, b.y, h.y));
  float2 t = fp::fma2(c, h, b);
  if (F == kSlow) return fp::add2(h, t);
  if (c.x < 0.f) t.x += h.x;
  if (c.y < 0.f) t.y += h.y;
  return t;
}
template <int F>
__device__ __forceinline__ float decayed(float c, float v) {   // a v
  if (F == kSafe && fabsf(v) == kInf) return v;
  return fmaf(c, v, F == kSlow || c < 0.f ? v : 0.f);
}
template <int F>
__device__ __forceinline__ float2 decayed(float2 c, float2 v) {
  if (F == kSlow) return fp::fma2(c, v, v);
  return make_float2(decayed<F>(c.x, v.x), decayed<F>(c.y, v.y));
}
constexpr float kHuge = 1e30f;   // what a tile makes of its maps stays finite below it
__device__ __forceinline__ bool huge2(float2 v) { return !(fabsf(v.x) + fabsf(v.y) < kHuge); }   // or NaN
__device__ __forceinline__ bool rarely(bool v) { return __builtin_expect(v, 0); }

// ------------------------------------------------------------------------------------------------
// Forward.
//
// The work is cut into tiles of kSteps steps by one 128-byte row of channels.  A block takes tiles
// by ticket, time-major, so a tile only ever waits for tiles with smaller tickets, which blocks
// hold that are running: every wait ends.  The next tile's rows are in flight while this one is
// computed.  A warp owns SPW consecutive steps of the tile, forms c and b = m i x once, in
// registers, and composes its steps into one map (its decay from the sum of the l); the maps of the
// block's warps and, by look-back, of earlier tiles give the state before the warp's first step, and a
// second walk over the registers writes y.  Every input byte is read once.
//
// 8 x 4096 x 2048 bf16 with states: 103 us, 5.3 TB/s of 541 MB (78 % of the measured copy rate), with the
// special-function unit (4 a value) and the issue slots (31 instructions a value) each busy more than half
// of the time; 1 x 131072 x 1024 f32: 355 us, 6.1 TB/s (89 %).
// ------------------------------------------------------------------------------------------------
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowBytes = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTiny = 1e-36f;   // well above the smallest normal number (the approximations flush what is below)

// Special functions by approximation: 1/x is good to 2^-23, 2^x and 1/sqrt x to 2^-22, and v log2 e adds |v| 2^-23
// to e^v, so a sigmoid s is good to about 2^-21 + (1 - s) |v| 2^-23.  The exact functions are several
// instructions each, of which the kernels issue 31 and 62 a value in all.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsqrt_approx(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
// 1 + e^-v, the reciprocal of sigmoid(v); inf where e^-v is
__device__ __forceinline__ float2 one_plus_exp2(float2 v) {
  const float2 t = fp::mul2(v, dup(-kLog2e));
  return fp::add2(make_float2(fp::ex2_approx(t.x), fp::ex2_approx(t.y)), dup(1.f));
}
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }
__device__ __forceinline__ float2 rcp2(float2 d) { return make_float2(rcp_approx(d.x), rcp_approx(d.y)); }
// l = rate r, and in the mixed form a little less: there c = 0 is a decay of zero, not of one.
template <bool kFar>
__device__ __forceinline__ float2 log_decay(float2 rate, float2 r) {
  return kFar ? fp::fma2(rate, r, dup(-kTiny)) : fp::mul2(rate, r);
}
// c of a decay e^l.  Above -1/4 expm1 by the Taylor polynomial of degree 6, whose remainder l^6 / 5040 is 5e-8
// of the value; below, 2^x, whose error is 2^-22 and the argument's |l| 2^-23.  kFar = false where no
// channel of the warp can leave the polynomial's range (l >= -rate).
constexpr float kNear = 0.25f;
template <bool kFar>
__device__ __forceinline__ float2 decay(float2 l) {
  float2 q = fp::fma2(l, dup(1.f / 720), dup(1.f / 120));
  q = fp::fma2(q, l, dup(1.f / 24));
  q = fp::fma2(q, l, dup(1.f / 6));
  q = fp::fma2(q, l, dup(0.5f));
  float2 c = fp::fma2(fp::mul2(q, l), l, l);
  if (kFar) {
    const float2 a = make_float2(fp::ex2_approx(l.x * kLog2e), fp::ex2_approx(l.y * kLog2e));
    c.x = l.x < -kNear ? a.x : c.x;
    c.y = l.y < -kNear ? a.y : c.y;
  }
  return c;
}
// 1 - a^2, without cancellation next to one: -c (2 + c), plus a number too small to matter that keeps it from
// being zero.
template <bool kFar>
__device__ __forceinline__ float2 one_minus_a2(float2 c) {
  float2 v = fp::fma2(c, fp::fma2(c, dup(-1.f), dup(-2.f)), dup(kTiny));
  if (kFar) {
    v.x = c.x < 0.f ? v.x : fmaf(-c.x, c.x, 1.f);
    v.y = c.y < 0.f ? v.y : fmaf(-c.y, c.y, 1.f);
  }
  return v;
}

// Copy of 8 bytes, of which the first n are read and the others zeros.
__device__ __forceinline__ void cp_async8(void* dst, const void* src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(tc::smem_u32(dst)), "l"(src), "r"(n) : "memory");
}

// Rows of one array for the calling warp: ROWS rows from `src` (the warp's first row, the tile's first
// channel) on, kRowBytes each; `rows` and `bytes` are how many rows and bytes of a row lie inside the
// array, the rest becomes zeros.  ALIGN is what every row start is known to be aligned to: 16, 8 or
// 4 (one copy per so many bytes), or 2 (odd bf16 rows, through registers).
template <int ROWS, int ALIGN>
__device__ __forceinline__ void load_rows(unsigned char* dst, const unsigned char* src, int64_t pitch, int rows,
                                          int bytes, int lane) {
  constexpr int kPer = ALIGN == 2 ? 4 : ALIGN;   // bytes a lane moves at a time
  constexpr int kLanes = kRowBytes / kPer;       // lanes a row takes: 8, 16 or 32
  constexpr int kAtOnce = 32 / kLanes;
  static_assert(ROWS % kAtOnce == 0, "whole groups of rows");
  const int r = lane / kLanes, at = lane % kLanes * kPer;
  const unsigned char* s = src + r * pitch + at;
  unsigned char* d = dst + r * kRowBytes + at;
  if (ALIGN == 16 && rows >= ROWS && bytes >= kRowBytes) {
#pragma unroll
    for (int k = 0; k < ROWS / kAtOnce; ++k) cp_async16(d + k * kAtOnce * kRowBytes, s + k * kAtOnce * pitch, 16);
    return;
  }
#pragma unroll
  for (int k = 0; k < ROWS / kAtOnce; ++k) {
    const int n = r + k * kAtOnce < rows ? min(max(bytes - at, 0), kPer) : 0;
    const unsigned char* sk = n > 0 ? s + k * kAtOnce * pitch : src;
    unsigned char* dk = d + k * kAtOnce * kRowBytes;
    if constexpr (ALIGN == 16) {
      cp_async16(dk, sk, n);
    } else if constexpr (ALIGN == 8) {
      cp_async8(dk, sk, n);
    } else if constexpr (ALIGN == 4) {
      if (n == 4) cp_async4(dk, sk);
      else *reinterpret_cast<uint32_t*>(dk) = 0u;   // the width is a multiple of 4 bytes
    } else {
      uint32_t v = 0;
      if (n >= 2) v = *reinterpret_cast<const uint16_t*>(sk);
      if (n >= 4) v |= (uint32_t)*reinterpret_cast<const uint16_t*>(sk + 2) << 16;
      *reinterpret_cast<uint32_t*>(dk) = v;
    }
  }
}

template <typename T>
struct Tile {
  static constexpr int kCh = kRowBytes / (int)sizeof(T);   // channels of a tile
  static constexpr int kCpl = kCh / 32;                    // channels of a lane
};

// The pair k of a lane's values in its warp's rows: for bf16 the lane's two channels of row k, for
// f32 its one channel of rows 2k and 2k + 1.
__device__ __forceinline__ float2 pair_at(const unsigned char* rows, int k, int lane, __nv_bfloat16) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(rows + k * kRowBytes + lane * 4);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_at(const unsigned char* rows, int k, int lane, float) {
  const float* f = reinterpret_cast<const float*>(rows + 2 * k * kRowBytes) + lane;
  return make_float2(f[0], f[kRowBytes / 4]);
}

// Writes a lane's channels of one row; `n` >= 1 of them lie inside the array.
template <int ALIGN>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&v)[2], int n) {
  if (ALIGN >= 4) {   // the width is even: both lie inside
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
  } else {
    p[0] = __float2bfloat16_rn(v[0]);
    if (n > 1) p[1] = __float2bfloat16_rn(v[1]);
  }
}
template <int ALIGN>
__device__ __forceinline__ void store_row(float* p, const float (&v)[2], int n) {
  p[0] = v[0];
}

// Where a tile lies.  Tickets run over all columns of a time before the next time.
struct Place {
  int64_t b, t0, word;   // word: index of the tile's first look-back word
  int32_t c0, ti, left;  // left: channels inside the array
  uint32_t tile;
};
template <typename T, int STEPS, bool kReverse>
__device__ __forceinline__ Place place(const RecParams& p, uint32_t tile) {
  constexpr int kCh = Tile<T>::kCh;
  const uint32_t all = p.cols * (uint32_t)p.batch, k = tile / all, col = tile % all;
  Place q;
  q.tile = tile;
  q.ti = (int32_t)(kReverse ? p.ntile - 1 - k : k);
  q.b = col / p.cols;
  q.c0 = (int32_t)(col % p.cols) * kCh;
  q.left = (int32_t)min((int64_t)kCh, p.D - q.c0);
  q.t0 = (int64_t)q.ti * STEPS;
  q.word = ((int64_t)col * p.ntile + q.ti) * kCh;
  return q;
}

// The look-back words are cleared by a kernel of their own, whose end only the first look-back of a block
// waits for: the first tiles are loaded and worked on meanwhile.
__global__ void __launch_bounds__(256) rec_clear_kernel(uint4* words, int64_t n) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x; k < n; k += (int64_t)gridDim.x * 256)
    words[k] = make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void wait_for_words() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// At a kernel's end: the last block to get here leaves the tickets at zero for the next call.
__device__ __forceinline__ void finish_tickets(const RecParams& p) {
  __syncthreads();
  if (p.ticket && threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(p.ticket + 1, 1u) == gridDim.x - 1) {
      p.ticket[0] = 0;
      p.ticket[1] = 0;
    }
  }
}

// A lane's values over its warp's SPW steps, in pairs: for bf16 the two channels of a step, for f32 two
// steps of one channel.
template <typename T, int SPW>
struct Walk {
  static constexpr int kCpl = Tile<T>::kCpl, kPairs = SPW * kCpl / 2;
  // the state after pair k from the one before it (f32: in x; y is the state between its two steps)
  template <int F>
  static __device__ __forceinline__ float2 next(float2 c, float2 b, float2 h) {
    if constexpr (kCpl == 2) return step<F>(c, b, h);
    h.y = step<F>(c.x, b.x, h.x);
    h.x = step<F>(c.y, b.y, h.y);
    return h;
  }
  // the gradient that pair k hands to the step before it, from the one that is handed to it (f32: in x)
  template <int F>
  static __device__ __forceinline__ float2 before(float2 c, float2 dy, float2 Q) {
    if constexpr (kCpl == 2) return decayed<F>(c, fp::add2(dy, Q));
    Q.x = decayed<F>(c.x, dy.x + decayed<F>(c.y, dy.y + Q.x));
    return Q;
  }
  // sets the pairs of steps from `steps` on
  static __device__ __forceinline__ void cut(float2 (&v)[kPairs], int steps, float to) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      if constexpr (kCpl == 2) {
        if (k >= steps) v[k] = dup(to);
      } else {
        if (2 * k >= steps) v[k].x = to;
        if (2 * k + 1 >= steps) v[k].y = to;
      }
    }
  }
};

// By one warp: the maps of a block's warps as one (in time order, or backwards), and the states before each of
// them from the one before the first, which becomes the one behind the last.
template <int NW, int N, bool kBack, typename M, typename L>
__device__ __forceinline__ void block_map(const M& maps, const L& logs, int cl, float (&A)[N], float (&H)[N]) {
  float l[N];
#pragma unroll
  for (int c = 0; c < N; ++c) {
    H[c] = l[c] = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const float2 m = maps[kBack ? NW - 1 - k : k][cl + c];
      H[c] = lookback::apply(m.x, m.y, H[c]);
      l[c] += logs[k][cl + c];
    }
  }
  const float2 a = decay<true>(make_float2(l[0], l[N - 1]));
  A[0] = a.x;
  A[N - 1] = N == 2 ? a.y : a.x;
}
template <int NW, int N, bool kBack, typename M, typename B>
__device__ __forceinline__ void block_states(const M& maps, B& before, int cl, float (&h)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c) {
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const int k = kBack ? NW - 1 - j : j;
      before[k][cl + c] = h[c];
      const float2 m = maps[k][cl + c];
      h[c] = lookback::apply(m.x, m.y, h[c]);
    }
  }
}

// The same in the third form: the state before the `count`-th warp from the one before the first.
template <int NW, int N, bool kBack, typename M>
__device__ __forceinline__ float2 safe_state(const M& maps, int cl, int count, float2 h) {
#pragma unroll 1
  for (int j = 0; j < count; ++j) {
    const int k = kBack ? NW - 1 - j : j;
    const float2 m0 = maps[k][cl], m1 = maps[k][cl + N - 1];
    h = step<kSafe>(make_float2(m0.x, m1.x), make_float2(m0.y, m1.y), h);
  }
  return h;
}

// Whether a lane's rows hold an input gate so closed that its 1 / i overflows when squared, but not so that i is 0
// (-inf in every 16th step, as a mask, takes 8 x 4096 x 2048 bf16 from 103 to 119 us).
template <typename T, int ROWS>
__device__ __forceinline__ bool hardly_open(const unsigned char* rows, int lane) {
  bool any = false;
#pragma unroll 1
  for (int k = 0; k < ROWS; ++k) {
    const unsigned char* row = rows + k * kRowBytes;
    const float2 g = Tile<T>::kCpl == 2 ? pair_at(row, 0, lane, __nv_bfloat16()) : dup(reinterpret_cast<const float*>(row)[lane]);
    any = any || (g.x < -44.f && g.x > -89.f) || (g.y < -44.f && g.y > -89.f);   // 2^64 = e^44.4, 2^128 = e^88.7
  }
  return any;
}

// A step formed from its row in shared memory (of x, gate_a, gate_x and, in the backward, dy), in the third form.
struct Step {
  float2 x, dy, c, mi, xi, io, r;
};
template <typename T, bool kBackward>
__device__ __forceinline__ Step step_at(const unsigned char* row, int array, int lane, float2 rate) {
  auto at = [&](int a) {
    const unsigned char* v = row + a * array;
    return Tile<T>::kCpl == 2 ? pair_at(v, 0, lane, __nv_bfloat16()) : dup(reinterpret_cast<const float*>(v)[lane]);
  };
  Step v;
  v.x = at(0);
  v.r = rcp2(one_plus_exp2(at(1)));
  const float2 d = one_plus_exp2(at(2)), i = rcp2(d);
  v.c = decay<true>(log_decay<true>(rate, v.r));
  const float2 u = one_minus_a2<true>(v.c), over = make_float2(rsqrt_approx(u.x), rsqrt_approx(u.y));
  const float2 m = fp::mul2(u, over);
  v.mi = fp::mul2(m, i);
  if (!kBackward) {   // as in the forward's other forms, while that is good
    const float2 d2 = fp::mul2(fp::mul2(u, d), d);
    const float2 mi = fp::mul2(u, make_float2(rsqrt_approx(d2.x), rsqrt_approx(d2.y)));
    v.mi = make_float2(d2.x < kInf ? mi.x : v.mi.x, d2.y < kInf ? mi.y : v.mi.y);
  } else {
    const float2 ix = fp::mul2(i, v.x);
    v.dy = at(3);
    v.xi = fp::mul2(fp::mul2(m, ix), fp::fma2(i, dup(-1.f), dup(1.f)));
    v.io = decayed<kSafe>(v.c, fp::mul2(ix, fp::mul2(over, v.r)));
  }
  return v;
}

// NW warps of 16 steps.  Half as many blocks of 8 warps wait for the look-back together, so bf16,
// bound by issue slots, takes four blocks of 4 warps an SM (8 x 4096 x 2048: 103 us, 107 us with two of
// 8); f32, whose rows are half as many channels, takes the longer tiles and with them half the look-back's
// chain (1 x 131072 x 1024: 355 us, 381 us with 4 warps).
template <typename T>
struct Forward {
  static constexpr int kNw = sizeof(T) == 2 ? 4 : 8, kSpw = 16, kSteps = kNw * kSpw, kBlocks = 16 / kNw;
};

// How a tile's rows get to shared memory: as one TMA box an array, or by every warp for its own rows in
// copies of 16 bytes (arrays that TMA does not take: broadcast axes), 8, 4 or 2.  A box costs its
// block a few instructions, the copies a tenth of all (8 x 4096 x 2048 bf16: forward 103 us, 111 us by
// copies of 16; backward 215 and 253 us); 29 x 12456 x 332 bf16, whose rows start on 8 bytes, takes
// 355 us by copies of 8 and 392 by copies of 4.
constexpr int kTma = 32;

__device__ __forceinline__ void tma_tile(void* dst, const CUtensorMap* map, uint64_t* bar, const Place& q) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          tc::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(tc::smem_u32(bar)), "r"(q.c0), "r"((int32_t)q.t0), "r"((int32_t)q.b)
      : "memory");
}
// By one thread: N arrays' boxes of `bytes` each into a stage.
template <int N>
__device__ __forceinline__ void tma_load(unsigned char* stage, const RecParams& p, uint64_t* bar, const Place& q,
                                         int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc::smem_u32(bar)), "r"(N * bytes)
               : "memory");
#pragma unroll
  for (int a = 0; a < N; ++a) tma_tile(stage + a * bytes, p.map + a, bar, q);
}
// A stage's boxes are there (bounded: 1 s, then SSD_ERR_TIMEOUT is latched).
__device__ __forceinline__ void tma_wait(uint64_t* bar, uint32_t phase, WsHeader* hdr) {
  if (!tc::mbar_wait_bounded(bar, phase, 1000000000ull) && threadIdx.x == 0) latch_error(hdr, SSD_ERR_TIMEOUT, 402);
}

template <typename T>
struct ForwardShared {
  static constexpr int NW = Forward<T>::kNw, kCh = Tile<T>::kCh;
  float2 maps[NW][kCh];    // (c, H) of every warp's steps
  float logs[NW][kCh];     // their log decays together
  float before[NW][kCh];   // the state before every warp's steps
  float rates[3][kCh];     // -c softplus(decay) of the tile's channels
  Place places[3];         // of the tile in hand, the one being loaded and the one after it
  uint64_t full[2];        // TMA: a stage's boxes have landed
};
// By one warp: a tile's place and its channels' rates.
template <typename T>
__device__ __forceinline__ void fetch_forward(const RecParams& p, ForwardShared<T>& s, uint32_t last, int turn) {
  constexpr int kCpl = Tile<T>::kCpl;
  const int lane = threadIdx.x % 32, cl = lane * kCpl;
  uint32_t tile = last + gridDim.x;
  if (p.ticket) {
    if (lane == 0) tile = atomicAdd(p.ticket, 1u);
    tile = __shfl_sync(0xffffffffu, tile, 0);
  }
  const Place q = place<T, Forward<T>::kSteps, false>(p, tile);
  if (lane == 0) s.places[turn] = q;
  if (tile < p.tiles) {
#pragma unroll
    for (int c = 0; c < kCpl; ++c)
      s.rates[turn][cl + c] = cl + c < q.left ? -p.c * softplus(p.decay[q.c0 + cl + c]) : 0.f;
  }
}

// The rest of a tile with huge values: from its maps on (behind barrier A), or from the states before the warps'
// steps (behind barrier B).  `stage`: the tile's rows; `turn`: where it lies in `places`.
template <typename T, int ALIGN>
__device__ __noinline__ void odd_forward(const RecParams& p, ForwardShared<T>& s, const unsigned char* stage, int turn,
                                         bool maps, bool first) {
  constexpr int NW = Forward<T>::kNw, SPW = Forward<T>::kSpw, kCh = Tile<T>::kCh, kCpl = Tile<T>::kCpl;
  constexpr int kWarpBytes = SPW * kRowBytes, kArray = NW * kWarpBytes;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, cl = lane * kCpl;
  const Place q = s.places[turn];
  const float2 rate = make_float2(s.rates[turn][cl], s.rates[turn][cl + kCpl - 1]);
  const int steps = (int)p.T - (int)q.t0 - warp * SPW, inside = min(SPW, max(0, steps));
  const unsigned char* rows = stage + warp * kWarpBytes;
  if (maps) {
    float2 H = make_float2(0.f, 0.f);
#pragma unroll 1
    for (int k = 0; k < inside; ++k) {
      const Step v = step_at<T, false>(rows + k * kRowBytes, kArray, lane, rate);
      H = step<kSafe>(v.c, fp::mul2(v.mi, v.x), H);
    }
    s.maps[warp][cl].y = H.x;
    if (kCpl == 2) s.maps[warp][cl + kCpl - 1].y = H.y;
    __syncthreads();
    if (warp == 0) {
      float A[kCpl], H[kCpl], h[kCpl];
      block_map<NW, kCpl, false>(s.maps, s.logs, cl, A, H);
      const float2 all = safe_state<NW, kCpl, false>(s.maps, cl, NW, make_float2(0.f, 0.f));
      H[0] = all.x;
      H[kCpl - 1] = kCpl == 2 ? all.y : all.x;
      if (first) wait_for_words();
      uint64_t* words = p.words + q.word + cl;
      const bool last = q.ti == p.ntile - 1;
      uint64_t v[kCpl];
      if (q.ti == 0) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) h[c] = p.init && cl + c < q.left ? p.init[q.b * p.D + q.c0 + cl + c] : 0.f;
      } else {
        if (!last) {
#pragma unroll
          for (int c = 0; c < kCpl; ++c) v[c] = lookback::map(A[c], H[c]);
          lookback::publish(words, v);
        }
        lookback::state_before<1>(words - kCh, -kCh, q.ti, h, p.hdr, 400);
      }
      if (!last) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) v[c] = lookback::inclusive(lookback::apply_safe(A[c], H[c], h[c]));
        lookback::publish(words, v);
      }
      s.before[0][cl] = h[0];
      if (kCpl == 2) s.before[0][cl + kCpl - 1] = h[kCpl - 1];
    } else if (warp == 1) {
      const int next = turn == 2 ? 0 : turn + 1;
      fetch_forward(p, s, s.places[next].tile, next == 2 ? 0 : next + 1);
    }
    __syncthreads();
  }
  float2 h = safe_state<NW, kCpl, false>(s.maps, cl, warp, make_float2(s.before[0][cl], s.before[0][cl + kCpl - 1]));
  const int n = min(kCpl, max(0, q.left - cl));
  if (n > 0 && steps > 0) {
    const int64_t states = (q.b * p.nch + (q.t0 + warp * SPW) / kChunk) * p.D + q.c0 + cl;
    if (p.states_out && warp * SPW % kChunk == 0 && SSD_INDEX_OK(p.hdr, states + n - 1, p.batch * p.nch * p.D, 60)) {
      p.states_out[states] = h.x;
      if (n == 2) p.states_out[states + 1] = h.y;
    }
    const int64_t row0 = (q.b * p.T + q.t0 + warp * SPW) * p.D + q.c0 + cl;
#pragma unroll 1
    for (int k = 0; k < inside; ++k) {
      const Step v = step_at<T, false>(rows + k * kRowBytes, kArray, lane, rate);
      h = step<kSafe>(v.c, fp::mul2(v.mi, v.x), h);
      const float o[2] = {h.x, h.y};
      if (p.y && SSD_INDEX_OK(p.hdr, row0 + k * p.D + n - 1, p.batch * p.T * p.D, 61))
        store_row<ALIGN>(static_cast<T*>(p.y) + row0 + k * p.D, o, n);
    }
    const int64_t at = q.b * p.D + q.c0 + cl;
    if (p.final_state && steps <= SPW && SSD_INDEX_OK(p.hdr, at + n - 1, p.batch * p.D, 62)) {
      p.final_state[at] = h.x;
      if (n == 2) p.final_state[at + 1] = h.y;
    }
  }
  __syncthreads();   // the rows and maps are read no more
}

template <typename T, int ALIGN>
__global__ void __launch_bounds__(32 * Forward<T>::kNw, Forward<T>::kBlocks) rec_forward_kernel(const __grid_constant__ RecParams p) {
  constexpr int NW = Forward<T>::kNw, SPW = Forward<T>::kSpw, kCh = Tile<T>::kCh, kCpl = Tile<T>::kCpl;
  constexpr int kPairs = Walk<T, SPW>::kPairs, kWarpBytes = SPW * kRowBytes, kArray = NW * kWarpBytes;
  constexpr int kStage = 3 * kArray;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ ForwardShared<T> s;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int cl = lane * kCpl;

  auto load = [&](const Place& q, int stage) {
    if constexpr (ALIGN == kTma) {
      if (threadIdx.x == 0 && q.tile < p.tiles) tma_load<3>(smem + stage * kStage, p, s.full + stage, q, kArray);
      return;
    }
    if (q.tile < p.tiles) {
      const int64_t t = q.t0 + warp * SPW;
      const int rows = (int)min((int64_t)SPW, max((int64_t)0, p.T - t)), bytes = q.left * (int)sizeof(T);
      unsigned char* d = smem + stage * kStage + warp * kWarpBytes;
      // a warp whose rows all lie past the end reads nothing: its pointers are the array's start
      auto at = [&](const void* base, const int64_t (&stride)[2]) {
        return static_cast<const unsigned char*>(base) +
               (rows > 0 ? (q.b * stride[0] + t * stride[1] + q.c0) * (int64_t)sizeof(T) : 0);
      };
      load_rows<SPW, ALIGN>(d, at(p.x, p.xs), p.xs[1] * sizeof(T), rows, bytes, lane);
      load_rows<SPW, ALIGN>(d + kArray, at(p.ga, p.as), p.as[1] * sizeof(T), rows, bytes, lane);
      load_rows<SPW, ALIGN>(d + 2 * kArray, at(p.gx, p.gs), p.gs[1] * sizeof(T), rows, bytes, lane);
    }
    cp_async_commit();
  };
  if (ALIGN == kTma && threadIdx.x == 0) {
    tc::mbar_init(s.full, 1);
    tc::mbar_init(s.full + 1, 1);
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    fetch_forward(p, s, blockIdx.x - gridDim.x, 0);
    __syncwarp();
    fetch_forward(p, s, blockIdx.x, 1);
  }
  __syncthreads();
  load(s.places[0], 0);
  for (int it = 0, turn = 0;; ++it) {
    const int slot = it & 1, here = turn, next = here == 2 ? 0 : here + 1;
    turn = next;
    const Place& q = s.places[here];
    if (q.tile >= p.tiles) break;
    load(s.places[next], slot ^ 1);
    if constexpr (ALIGN == kTma) {
      tma_wait(s.full + slot, (it >> 1) & 1, p.hdr);
    } else {
      cp_async_wait<1>();
      __syncwarp();
    }
    const float2 rate = make_float2(s.rates[here][cl], s.rates[here][cl + kCpl - 1]);
    // whether a channel of the tile can decay faster than e^-1/4 a step: the same for all warps
    const bool far = __any_sync(0xffffffffu, fminf(rate.x, rate.y) < -kNear);
    const int steps = (int)p.T - (int)q.t0 - warp * SPW;   // of this warp's that lie inside; SPW or more: all
    const int inside = min(SPW, max(0, steps));

    const unsigned char* rows = smem + slot * kStage + warp * kWarpBytes;
    float2 dec[kPairs], b[kPairs];
    bool large = false;   // a huge value, or NaN
    auto first = [&](auto form) {   // the steps and their map
      constexpr int F = decltype(form)::value;
      constexpr bool kFar = F == kMixed;
      float2 l = make_float2(0.f, 0.f), most = l;   // their log decays together; infinite where a d^2 is
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        const float2 lk = log_decay<kFar>(rate, rcp2(one_plus_exp2(pair_at(rows + kArray, k, lane, T()))));
        l = fp::add2(l, lk);
        dec[k] = decay<kFar>(lk);
        // m i = sqrt(u) / d = u / sqrt(u d^2), u = 1 - a^2, d = 1 / i: one special function, not two.  Where d^2
        // overflows, i < 2^-64, that is 0: such tiles are odd too.
        const float2 d = one_plus_exp2(pair_at(rows + 2 * kArray, k, lane, T()));
        const float2 u = one_minus_a2<kFar>(dec[k]);
        const float2 v = fp::mul2(fp::mul2(u, d), d);       // never 0, nor 0 * inf
        most = fp::add2(most, v);
        const float2 mi = fp::mul2(u, make_float2(rsqrt_approx(v.x), rsqrt_approx(v.y)));
        b[k] = fp::mul2(mi, pair_at(rows, k, lane, T()));
      }
      if (steps < SPW) {   // steps past the end change nothing; nobody needs the maps of such warps
        Walk<T, SPW>::cut(dec, steps, -kTiny);
        Walk<T, SPW>::cut(b, steps, 0.f);
      }
      if constexpr (kCpl == 1) l = dup(l.x + l.y);
      l = fp::add2(l, dup(-kTiny));   // maps are of the mixed form
      const float2 all = decay<true>(l);
      float2 H = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) H = Walk<T, SPW>::template next<F>(dec[k], b[k], H);
      s.maps[warp][cl] = make_float2(all.x, H.x);
      s.logs[warp][cl] = l.x;
      if (kCpl == 2) {
        s.maps[warp][cl + kCpl - 1] = make_float2(all.y, H.y);
        s.logs[warp][cl + kCpl - 1] = l.y;
      }
      large = huge2(kCpl == 2 ? H : dup(H.x));
      if (rarely(!(most.x + most.y < kInf))) large = large || hardly_open<T, SPW>(rows + 2 * kArray, lane);
    };
    if (far) first(std::integral_constant<int, kMixed>());
    else first(std::integral_constant<int, kSlow>());
    // A: the warps' maps are there; everyone is done with this stage's rows
    if (rarely(__syncthreads_or(large))) {
      odd_forward<T, ALIGN>(p, s, smem + slot * kStage, here, true, it == 0);
      continue;
    }
    if (warp == 0) {
      float A[kCpl], H[kCpl], h[kCpl];
      block_map<NW, kCpl, false>(s.maps, s.logs, cl, A, H);
      if (it == 0) wait_for_words();
      uint64_t* words = p.words + q.word + cl;
      const bool last = q.ti == p.ntile - 1;
      uint64_t v[kCpl];
      if (q.ti == 0) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) h[c] = p.init && cl + c < q.left ? p.init[q.b * p.D + q.c0 + cl + c] : 0.f;
      } else {
        if (!last) {
#pragma unroll
          for (int c = 0; c < kCpl; ++c) v[c] = lookback::map(A[c], H[c]);
          lookback::publish(words, v);
        }
        // 8 words at a time save 4 % of a lone long sequence's chain (1 x 109272 x 576 bf16: 201 us, 210 with 7, 240
        // with 5) and cost the registers 2 % of the others' (8 x 4096 x 2048: 104.4, 102.7 and 102.7)
        lookback::state_before<7>(words - kCh, -kCh, q.ti, h, p.hdr, 400);
      }
      if (!last) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) v[c] = lookback::inclusive(lookback::apply_safe(A[c], H[c], h[c]));
        lookback::publish(words, v);
      }
      large = huge2(make_float2(h[0], h[kCpl - 1]));
      block_states<NW, kCpl, false>(s.maps, s.before, cl, h);
    } else if (warp == 1) {
      fetch_forward(p, s, s.places[next].tile, next == 2 ? 0 : next + 1);
    }
    // B: the states before the warps' steps are there, and the tile after the next
    if (rarely(__syncthreads_or(large))) {
      odd_forward<T, ALIGN>(p, s, smem + slot * kStage, here, false, false);
      continue;
    }
    float2 h = make_float2(s.before[warp][cl], s.before[warp][cl + kCpl - 1]);
    const int n = min(kCpl, max(0, q.left - cl));   // this lane's channels that lie inside
    if (p.states_out && warp * SPW % kChunk == 0 && steps > 0) {
      const int64_t at = (q.b * p.nch + (q.t0 + warp * SPW) / kChunk) * p.D + q.c0 + cl;
      if (n > 0 && SSD_INDEX_OK(p.hdr, at + n - 1, p.batch * p.nch * p.D, 60)) {
        p.states_out[at] = h.x;
        if (n == 2) p.states_out[at + 1] = h.y;
      }
    }
    const int64_t row0 = (q.b * p.T + q.t0 + warp * SPW) * p.D + q.c0 + cl;
    const int live = p.y && n > 0 ? inside : 0;   // steps to write
    const bool ends = p.final_state && n > 0 && steps > 0 && steps <= SPW;   // the last step is this warp's
    auto walk = [&](auto whole, auto form) {
      T* y = static_cast<T*>(p.y) + row0;
      auto store = [&](int t, float v0, float v1) {
        const float v[2] = {v0, v1};
        if ((decltype(whole)::value || t < live) &&
            SSD_INDEX_OK(p.hdr, row0 + t * p.D + n - 1, p.batch * p.T * p.D, 61))
          store_row<ALIGN>(y, v, n);
        y += p.D;
      };
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        h = Walk<T, SPW>::template next<decltype(form)::value>(dec[k], b[k], h);
        if constexpr (kCpl == 2) {
          store(k, h.x, h.y);
        } else {
          store(2 * k, h.y, 0.f);
          store(2 * k + 1, h.x, 0.f);
        }
      }
    };
    auto second = [&](auto form) {
      if (live == SPW) walk(std::true_type(), form);
      else if (live > 0 || ends) walk(std::false_type(), form);
    };
    if (far) second(std::integral_constant<int, kMixed>());
    else second(std::integral_constant<int, kSlow>());
    if (ends) {
      const int64_t at = q.b * p.D + q.c0 + cl;
      if (SSD_INDEX_OK(p.hdr, at + n - 1, p.batch * p.D, 62)) {
        p.final_state[at] = h.x;
        if (n == 2) p.final_state[at + 1] = h.y;
      }
    }
  }
  cp_async_wait_all();
  finish_tickets(p);
}

// ------------------------------------------------------------------------------------------------
// Backward.
//
// The same tiles, from the last to the first; a tile's state comes from the states that the forward
// kept (one a tile), so only dL/dh is carried by look-back: C = a G, the gradient that a tile hands
// to the step before it, maps to a C + Q over a tile with the same decay a as the forward's.  A warp
// forms the forward maps of its steps, takes the state before them, walks them forward for
//   mi = m i,  xi = mi x (1 - i),  kr = a (h_{t-1} - a i x / m) r,  r   (kept in registers)
// and composes the reverse map; with C known a walk backwards gives G and writes
//   dx = G mi, dgate_x = G xi, dgate_a = rate G kr (1 - r)   and sums G kr for ddecay.
// ddecay: one partial row per tile, added in tile order by rec_ddecay_kernel.
//
// 8 x 4096 x 2048 bf16: 215 us, 4.4 TB/s of 944 MB (65 % of the measured copy rate): five values are kept
// for every step and channel, so 128 registers a thread (none spilled) and two blocks an SM, which issue 62
// instructions a value half of the time and wait for their block's barriers and look-back otherwise.
// ------------------------------------------------------------------------------------------------
constexpr int kSpwBwd = 8;
static_assert(kWarps * kSpwBwd == kChunk, "a backward tile starts from one kept state");

// The tile after `last`, for one warp.
__device__ __forceinline__ uint32_t take_ticket(const RecParams& p, uint32_t last) {
  uint32_t tile = last + gridDim.x;
  if (p.ticket) {
    if (threadIdx.x % 32 == 0) tile = atomicAdd(p.ticket, 1u);
    tile = __shfl_sync(0xffffffffu, tile, 0);
  }
  return tile;
}
template <typename T>
struct BackwardShared {
  static constexpr int kCh = Tile<T>::kCh;
  float2 maps[kWarps][kCh];   // forward (c, H) of every warp's steps
  float2 back[kWarps][kCh];   // reverse (c, Q)
  float logs[kWarps][kCh];    // their log decays together
  float after[kWarps][kCh];   // C from the step after every warp's steps
  float sums[kWarps][kCh];    // G kr over every warp's steps
  float rates[3][kCh];        // -c softplus(decay)
  float start[3][kCh];        // the kept state
  int64_t partial_at;         // where the tile before has its row of ddecay partials,
  int partial_left;           // and how many of its channels lie inside (warp 2's)
  Place places[3];            // of the tile in hand, the one being loaded and the one after it
  uint64_t full[2];           // TMA: a stage's boxes have landed
};
// By one warp: a tile's place, its channels' rates and the state before it.
template <typename T>
__device__ __forceinline__ void fetch_backward(const RecParams& p, BackwardShared<T>& s, uint32_t tile, int turn) {
  constexpr int kCpl = Tile<T>::kCpl;
  const int lane = threadIdx.x % 32, cl = lane * kCpl;
  const Place q = place<T, kChunk, true>(p, tile);
  if (lane == 0) s.places[turn] = q;
  if (tile < p.tiles) {
    const float* kept = p.states_in + (q.b * p.nch + q.ti) * p.D + q.c0;
#pragma unroll
    for (int c = 0; c < kCpl; ++c) {
      const bool in = cl + c < q.left;
      s.rates[turn][cl + c] = in ? -p.c * softplus(p.decay[q.c0 + cl + c]) : 0.f;
      s.start[turn][cl + c] = in ? kept[cl + c] : 0.f;
    }
  }
}
// By warp 2, once everyone's sums of a tile are there: its row of ddecay partials.
template <typename T>
__device__ __forceinline__ void write_partial(const RecParams& p, const BackwardShared<T>& s) {
  constexpr int kCpl = Tile<T>::kCpl;
  const int cl = threadIdx.x % 32 * kCpl;
  const int64_t at = s.partial_at + cl;
#pragma unroll
  for (int c = 0; c < kCpl; ++c) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += s.sums[k][cl + c];
    if (cl + c < s.partial_left && SSD_INDEX_OK(p.hdr, at + c, p.batch * p.nch * p.D, 65)) p.partial[at + c] = v;
  }
}

// The rest of a tile with huge values, as odd_forward.  Returns the warp's sum of G kr.
template <typename T, int ALIGN>
__device__ __noinline__ float2 odd_backward(const RecParams& p, BackwardShared<T>& s, const unsigned char* stage,
                                            int turn, uint32_t after, bool maps, bool first) {
  constexpr int SPW = kSpwBwd, kCh = Tile<T>::kCh, kCpl = Tile<T>::kCpl;
  constexpr int kWarpBytes = SPW * kRowBytes, kArray = kWarps * kWarpBytes;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, cl = lane * kCpl;
  const Place q = s.places[turn];
  const float2 rate = make_float2(s.rates[turn][cl], s.rates[turn][cl + kCpl - 1]);
  const int steps = (int)p.T - (int)q.t0 - warp * SPW, inside = min(SPW, max(0, steps));
  const unsigned char* rows = stage + warp * kWarpBytes;
  if (maps) {
    float2 H = make_float2(0.f, 0.f), Q = H;
#pragma unroll 1
    for (int k = 0; k < inside; ++k) {
      const Step v = step_at<T, true>(rows + k * kRowBytes, kArray, lane, rate);
      H = step<kSafe>(v.c, fp::mul2(v.mi, v.x), H);
    }
#pragma unroll 1
    for (int k = inside - 1; k >= 0; --k) {
      const Step v = step_at<T, true>(rows + k * kRowBytes, kArray, lane, rate);
      Q = decayed<kSafe>(v.c, fp::add2(v.dy, Q));
    }
    s.maps[warp][cl].y = H.x;
    s.back[warp][cl].y = Q.x;
    if (kCpl == 2) {
      s.maps[warp][cl + kCpl - 1].y = H.y;
      s.back[warp][cl + kCpl - 1].y = Q.y;
    }
    __syncthreads();
    if (warp == 0) {
      float A[kCpl], R[kCpl], C[kCpl];
      block_map<kWarps, kCpl, true>(s.back, s.logs, cl, A, R);
      const float2 all = safe_state<kWarps, kCpl, true>(s.back, cl, kWarps, make_float2(0.f, 0.f));
      R[0] = all.x;
      R[kCpl - 1] = kCpl == 2 ? all.y : all.x;
      if (first) wait_for_words();
      uint64_t* words = p.words + q.word + cl;
      uint64_t v[kCpl];
      if (q.ti == p.ntile - 1) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c)
          C[c] = p.dfinal && cl + c < q.left ? p.dfinal[q.b * p.D + q.c0 + cl + c] : 0.f;
      } else {
        if (q.ti > 0) {
#pragma unroll
          for (int c = 0; c < kCpl; ++c) v[c] = lookback::map(A[c], R[c]);
          lookback::publish(words, v);
        }
        lookback::state_before<1>(words + kCh, kCh, p.ntile - 1 - q.ti, C, p.hdr, 401);
      }
      if (q.ti > 0) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) v[c] = lookback::inclusive(lookback::apply_safe(A[c], R[c], C[c]));
        lookback::publish(words, v);
      }
      s.after[kWarps - 1][cl] = C[0];
      if (kCpl == 2) s.after[kWarps - 1][cl + kCpl - 1] = C[kCpl - 1];
    } else if (warp == 1) {
      const int next = turn == 2 ? 0 : turn + 1;
      fetch_backward(p, s, __shfl_sync(0xffffffffu, after, 0), next == 2 ? 0 : next + 1);
    } else if (warp == 2 && !first) {
      write_partial(p, s);
    }
    __syncthreads();
  }
  float2 prev[SPW], sum = make_float2(0.f, 0.f);
  float2 h = safe_state<kWarps, kCpl, false>(s.maps, cl, warp, make_float2(s.start[turn][cl], s.start[turn][cl + kCpl - 1]));
  float2 C = safe_state<kWarps, kCpl, true>(s.back, cl, kWarps - 1 - warp,
                                            make_float2(s.after[kWarps - 1][cl], s.after[kWarps - 1][cl + kCpl - 1]));
  const int n = min(kCpl, max(0, q.left - cl)), live = n > 0 ? inside : 0;
  const int64_t row0 = (q.b * p.T + q.t0 + warp * SPW) * p.D + q.c0 + cl;
#pragma unroll 1
  for (int k = 0; k < live; ++k) {
    const Step v = step_at<T, true>(rows + k * kRowBytes, kArray, lane, rate);
    prev[k] = h;
    h = step<kSafe>(v.c, fp::mul2(v.mi, v.x), h);
  }
#pragma unroll 1
  for (int k = live - 1; k >= 0; --k) {
    const Step v = step_at<T, true>(rows + k * kRowBytes, kArray, lane, rate);
    const float2 G = fp::add2(v.dy, C);
    C = decayed<kSafe>(v.c, G);
    const float2 kr = decayed<kSafe>(v.c, fp::fma2(prev[k], v.r, neg2(v.io)));
    const float2 vx = fp::mul2(G, v.mi), vg = fp::mul2(G, v.xi);
    const float2 va = fp::mul2(G, fp::mul2(fp::mul2(rate, kr), fp::fma2(v.r, dup(-1.f), dup(1.f))));
    if (kCpl == 2 || k % 2 == 0) sum.x = fmaf(G.x, kr.x, sum.x);   // in the order of the other forms
    if (kCpl == 2 || k % 2 == 1) sum.y = fmaf(G.y, kr.y, sum.y);
    const int64_t at = row0 + k * p.D;
    if (SSD_INDEX_OK(p.hdr, at + n - 1, p.batch * p.T * p.D, 63)) {
      const float x2[2] = {vx.x, vx.y}, a2[2] = {va.x, va.y}, g2[2] = {vg.x, vg.y};
      store_row<ALIGN>(static_cast<T*>(p.dx) + at, x2, n);
      store_row<ALIGN>(static_cast<T*>(p.dga) + at, a2, n);
      store_row<ALIGN>(static_cast<T*>(p.dgx) + at, g2, n);
    }
  }
  if (warp == 0 && p.dinit && q.ti == 0 && n > 0) {
    const int64_t at = q.b * p.D + q.c0 + cl;
    if (SSD_INDEX_OK(p.hdr, at + n - 1, p.batch * p.D, 64)) {
      p.dinit[at] = C.x;
      if (n == 2) p.dinit[at + 1] = C.y;
    }
  }
  __syncthreads();   // the rows and maps are read no more
  return sum;
}

template <typename T, int ALIGN, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) rec_backward_kernel(const __grid_constant__ RecParams p) {
  constexpr int SPW = kSpwBwd, kCh = Tile<T>::kCh, kCpl = Tile<T>::kCpl;
  constexpr int kPairs = Walk<T, SPW>::kPairs, kWarpBytes = SPW * kRowBytes, kArray = kWarps * kWarpBytes;
  constexpr int kStage = 4 * kArray;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ BackwardShared<T> s;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int cl = lane * kCpl;

  auto load = [&](const Place& q, int stage) {
    if constexpr (ALIGN == kTma) {
      if (threadIdx.x == 0 && q.tile < p.tiles) tma_load<4>(smem + stage * kStage, p, s.full + stage, q, kArray);
      return;
    }
    if (q.tile < p.tiles) {
      const int64_t t = q.t0 + warp * SPW;
      const int rows = (int)min((int64_t)SPW, max((int64_t)0, p.T - t)), bytes = q.left * (int)sizeof(T);
      unsigned char* d = smem + stage * kStage + warp * kWarpBytes;
      auto at = [&](const void* base, const int64_t (&stride)[2]) {
        return static_cast<const unsigned char*>(base) +
               (rows > 0 ? (q.b * stride[0] + t * stride[1] + q.c0) * (int64_t)sizeof(T) : 0);
      };
      load_rows<SPW, ALIGN>(d, at(p.x, p.xs), p.xs[1] * sizeof(T), rows, bytes, lane);
      load_rows<SPW, ALIGN>(d + kArray, at(p.ga, p.as), p.as[1] * sizeof(T), rows, bytes, lane);
      load_rows<SPW, ALIGN>(d + 2 * kArray, at(p.gx, p.gs), p.gs[1] * sizeof(T), rows, bytes, lane);
      load_rows<SPW, ALIGN>(d + 3 * kArray, at(p.dy, p.ds), p.ds[1] * sizeof(T), rows, bytes, lane);
    }
    cp_async_commit();
  };
  if (ALIGN == kTma && threadIdx.x == 0) {
    tc::mbar_init(s.full, 1);
    tc::mbar_init(s.full + 1, 1);
    tc::fence_mbar_init();
  }
  if (warp == 0) {
    const uint32_t one = take_ticket(p, blockIdx.x - gridDim.x), two = take_ticket(p, blockIdx.x);
    fetch_backward(p, s, one, 0);
    fetch_backward(p, s, two, 1);
  }
  __syncthreads();
  load(s.places[0], 0);
  if (threadIdx.x == 64) s.partial_left = 0;
  for (int it = 0, turn = 0;; ++it) {
    const int slot = it & 1, here = turn, next = here == 2 ? 0 : here + 1;
    turn = next;
    const Place& q = s.places[here];
    if (q.tile >= p.tiles) break;
    if constexpr (ALIGN == kTma) {
      tma_wait(s.full + slot, (it >> 1) & 1, p.hdr);
    } else {
      // The stage that is filled now held the tile before, whose dy the walk at its end read: a lane's
      // copies cover rows that other lanes read, so every lane of the warp has to be through.
      __syncwarp();
      load(s.places[next], slot ^ 1);
      cp_async_wait<1>();
      __syncwarp();
    }
    const float2 rate = make_float2(s.rates[here][cl], s.rates[here][cl + kCpl - 1]);
    uint32_t after = s.places[next].tile + gridDim.x;   // of warp 1's lane 0: the tile after the next, asked for early
    if (warp == 1 && lane == 0 && p.ticket) after = atomicAdd(p.ticket, 1u);
    const bool far = __any_sync(0xffffffffu, fminf(rate.x, rate.y) < -kNear);   // as in the forward
    const float2 h0 = make_float2(s.start[here][cl], s.start[here][cl + kCpl - 1]);
    const int steps = (int)p.T - (int)q.t0 - warp * SPW, inside = min(SPW, max(0, steps));

    const unsigned char* rows = smem + slot * kStage + warp * kWarpBytes;
    // kr holds a i x r / m, what h_{t-1} r is compared with, until the state is known (r / m does not overflow)
    float2 dec[kPairs], mi[kPairs], xi[kPairs], kr[kPairs], r[kPairs];
    bool large = false;   // a huge value, or NaN
    auto first = [&](auto form) {   // the steps and their maps
      constexpr int F = decltype(form)::value;
      constexpr bool kFar = F == kMixed;
      float2 l = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        r[k] = rcp2(one_plus_exp2(pair_at(rows + kArray, k, lane, T())));
        const float2 lk = log_decay<kFar>(rate, r[k]);
        l = fp::add2(l, lk);
        dec[k] = decay<kFar>(lk);
        const float2 i = rcp2(one_plus_exp2(pair_at(rows + 2 * kArray, k, lane, T())));
        const float2 u = one_minus_a2<kFar>(dec[k]);
        const float2 over = make_float2(rsqrt_approx(u.x), rsqrt_approx(u.y));   // 1 / m, at most 1e18
        const float2 ix = fp::mul2(i, pair_at(rows, k, lane, T()));
        const float2 m = fp::mul2(u, over);
        mi[k] = fp::mul2(m, i);
        xi[k] = fp::mul2(fp::mul2(m, ix), fp::fma2(i, dup(-1.f), dup(1.f)));
        kr[k] = decayed<F>(dec[k], fp::mul2(ix, fp::mul2(over, r[k])));
      }
      if (steps < SPW) {   // steps past the end change nothing (their x and dy are zeros)
        Walk<T, SPW>::cut(dec, steps, -kTiny);
        Walk<T, SPW>::cut(mi, steps, 0.f);
        Walk<T, SPW>::cut(r, steps, 0.f);
        l = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kPairs; ++k) l = fp::add2(l, fp::mul2(rate, r[k]));
      }
      if constexpr (kCpl == 1) l = dup(l.x + l.y);
      l = fp::add2(l, dup(-kTiny));   // maps are of the mixed form
      const float2 all = decay<true>(l);
      float2 H = make_float2(0.f, 0.f), Q = H;
#pragma unroll
      for (int k = 0; k < kPairs; ++k)
        H = Walk<T, SPW>::template next<F>(dec[k], fp::mul2(mi[k], pair_at(rows, k, lane, T())), H);
      // the reverse map: dy + C enters a step, a (dy + C) leaves it
#pragma unroll
      for (int k = kPairs - 1; k >= 0; --k)
        Q = Walk<T, SPW>::template before<F>(dec[k], pair_at(rows + 3 * kArray, k, lane, T()), Q);
      s.maps[warp][cl] = make_float2(all.x, H.x);
      s.back[warp][cl] = make_float2(all.x, Q.x);
      s.logs[warp][cl] = l.x;
      if (kCpl == 2) {
        s.maps[warp][cl + kCpl - 1] = make_float2(all.y, H.y);
        s.back[warp][cl + kCpl - 1] = make_float2(all.y, Q.y);
        s.logs[warp][cl + kCpl - 1] = l.y;
      }
      large = huge2(kCpl == 2 ? H : dup(H.x)) || huge2(kCpl == 2 ? Q : dup(Q.x));
    };
    if (far) first(std::integral_constant<int, kMixed>());
    else first(std::integral_constant<int, kSlow>());
    // A: the warps' maps are there, and the sums of the tile before
    const bool odd_maps = __syncthreads_or(large);
    // A box replaces a tile that every warp has left only now (its rows are read to the tile's end; a third
    // stage, asked for a tile earlier, took the L1 cache's room: 285 us instead of 215).
    if constexpr (ALIGN == kTma) load(s.places[next], slot ^ 1);
    auto put_sum = [&](float2 sum) {
      s.sums[warp][cl] = sum.x;
      if (kCpl == 2) s.sums[warp][cl + kCpl - 1] = sum.y;
      else s.sums[warp][cl] += sum.y;
      if (threadIdx.x == 64) {
        s.partial_at = (q.b * p.nch + q.ti) * p.D + q.c0;
        s.partial_left = q.left;
      }
    };
    if (rarely(odd_maps)) {
      put_sum(odd_backward<T, ALIGN>(p, s, smem + slot * kStage, here, after, true, it == 0));
      continue;
    }
    if (warp == 0) {
      float A[kCpl], Q[kCpl], C[kCpl];
      block_map<kWarps, kCpl, true>(s.back, s.logs, cl, A, Q);
      if (it == 0) wait_for_words();
      uint64_t* words = p.words + q.word + cl;
      uint64_t v[kCpl];
      if (q.ti == p.ntile - 1) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c)
          C[c] = p.dfinal && cl + c < q.left ? p.dfinal[q.b * p.D + q.c0 + cl + c] : 0.f;
      } else {
        if (q.ti > 0) {
#pragma unroll
          for (int c = 0; c < kCpl; ++c) v[c] = lookback::map(A[c], Q[c]);
          lookback::publish(words, v);
        }
        lookback::state_before<8 / kCpl>(words + kCh, kCh, p.ntile - 1 - q.ti, C, p.hdr, 401);
      }
      if (q.ti > 0) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) v[c] = lookback::inclusive(lookback::apply_safe(A[c], Q[c], C[c]));
        lookback::publish(words, v);
      }
      large = huge2(make_float2(C[0], C[kCpl - 1]));
      block_states<kWarps, kCpl, true>(s.back, s.after, cl, C);
#pragma unroll
      for (int c = 0; c < kCpl; ++c) {
        if (p.dinit && q.ti == 0 && cl + c < q.left) {
          const int64_t at = q.b * p.D + q.c0 + cl + c;
          if (SSD_INDEX_OK(p.hdr, at, p.batch * p.D, 64)) p.dinit[at] = C[c];
        }
      }
    } else if (warp == 1) {
      fetch_backward(p, s, __shfl_sync(0xffffffffu, after, 0), next == 2 ? 0 : next + 1);
    } else if (warp == 2 && it > 0) {
      write_partial(p, s);
    }
    {   // the state before the warp's steps, and kr of every step
      float2 h = h0;
      for (int k = 0; k < warp; ++k) {
        const float2 m0 = s.maps[k][cl], m1 = s.maps[k][cl + kCpl - 1];
        h = step<kMixed>(make_float2(m0.x, m1.x), make_float2(m0.y, m1.y), h);
      }
      large = large || huge2(h);
      auto states = [&](auto form) {
        constexpr int F = decltype(form)::value;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          const float2 b = fp::mul2(mi[k], pair_at(rows, k, lane, T()));
          float2 prev = h;
          if constexpr (kCpl == 2) {
            h = step<F>(dec[k], b, h);
          } else {
            prev.y = step<F>(dec[k].x, b.x, prev.x);
            h.x = step<F>(dec[k].y, b.y, prev.y);
          }
          kr[k] = decayed<F>(dec[k], fp::fma2(prev, r[k], neg2(kr[k])));
          r[k] = fp::mul2(fp::mul2(rate, kr[k]), fp::fma2(r[k], dup(-1.f), dup(1.f)));   // of dgate_a
        }
      };
      if (far) states(std::integral_constant<int, kMixed>());
      else states(std::integral_constant<int, kSlow>());
    }
    // B: C from the step after every warp's steps
    if (rarely(__syncthreads_or(large))) {
      put_sum(odd_backward<T, ALIGN>(p, s, smem + slot * kStage, here, after, false, false));
      continue;
    }
    float2 C = make_float2(s.after[warp][cl], s.after[warp][cl + kCpl - 1]), sum = make_float2(0.f, 0.f);
    const int n = min(kCpl, max(0, q.left - cl));
    const int live = n > 0 ? inside : 0;
    const int64_t row0 = (q.b * p.T + q.t0 + warp * SPW) * p.D + q.c0 + cl;
    auto walk = [&](auto whole, auto form) {
      constexpr int F = decltype(form)::value;
      const int64_t last = row0 + (SPW - 1) * p.D;
      T *px = static_cast<T*>(p.dx) + last, *pa = static_cast<T*>(p.dga) + last, *pg = static_cast<T*>(p.dgx) + last;
      auto store = [&](int t, float x0, float x1, float a0, float a1, float g0, float g1) {
        if ((decltype(whole)::value || t < live) &&
            SSD_INDEX_OK(p.hdr, row0 + t * p.D + n - 1, p.batch * p.T * p.D, 63)) {
          const float x2[2] = {x0, x1}, a2[2] = {a0, a1}, g2[2] = {g0, g1};
          store_row<ALIGN>(px, x2, n);
          store_row<ALIGN>(pa, a2, n);
          store_row<ALIGN>(pg, g2, n);
        }
        px -= p.D, pa -= p.D, pg -= p.D;
      };
#pragma unroll
      for (int k = kPairs - 1; k >= 0; --k) {
        const float2 dy = pair_at(rows + 3 * kArray, k, lane, T());
        float2 G;
        if constexpr (kCpl == 2) {
          G = fp::add2(dy, C);
          C = decayed<F>(dec[k], G);
        } else {
          G.y = dy.y + C.x;
          G.x = dy.x + decayed<F>(dec[k].y, G.y);
          C.x = decayed<F>(dec[k].x, G.x);
        }
        sum = fp::fma2(G, kr[k], sum);
        const float2 vx = fp::mul2(G, mi[k]), vg = fp::mul2(G, xi[k]), va = fp::mul2(G, r[k]);
        if constexpr (kCpl == 2) {
          store(k, vx.x, vx.y, va.x, va.y, vg.x, vg.y);
        } else {
          store(2 * k + 1, vx.y, 0.f, va.y, 0.f, vg.y, 0.f);
          store(2 * k, vx.x, 0.f, va.x, 0.f, vg.x, 0.f);
        }
      }
    };
    auto second = [&](auto form) {
      if (live == SPW) walk(std::true_type(), form);
      else walk(std::false_type(), form);
    };
    if (far) second(std::integral_constant<int, kMixed>());
    else second(std::integral_constant<int, kSlow>());
    put_sum(sum);
  }
  cp_async_wait_all();
  __syncthreads();
  if (warp == 2 && s.partial_left > 0) write_partial(p, s);
  finish_tickets(p);
}

// ddecay[d] = -c sigmoid(decay) * sum of the partial rows: a block takes 32 channels, its warps every
// 32nd row each, joined in warp order.
__global__ void __launch_bounds__(1024) rec_ddecay_kernel(RecParams p) {
  __shared__ float part[32][33];
  follow();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t d = (int64_t)blockIdx.x * 32 + lane, rows = p.batch * p.nch;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (d < p.D) {
    int64_t r = warp;
    for (; r + 96 < rows; r += 128) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += p.partial[(r + 32 * k) * p.D + d];
    }
    for (; r < rows; r += 32) s[0] += p.partial[r * p.D + d];
  }
  part[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  if (warp == 0 && d < p.D) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += part[k][lane];
    p.ddecay[d] = -p.c * v / (1.f + expf(-p.decay[d]));
  }
}

// ------------------------------------------------------------------------------------------------
// One step (serving): a thread takes V neighbouring channels of U sequences, so that the channels' rates
// are formed once for them.  Bound by memory for many sequences (512 x 2560 f32: 6.2 us, 5.1 TB/s),
// by the launch and one trip to memory for few.
// ------------------------------------------------------------------------------------------------
template <typename T, int V>
struct alignas(sizeof(T) * V) Vals {
  T v[V];
};

template <typename T, int V, int U>
__global__ void __launch_bounds__(128) rec_step_kernel(RecParams p) {
  constexpr int P = (V + 1) / 2;
  const int64_t d = ((int64_t)blockIdx.x * 128 + threadIdx.x) * V;
  if (d >= p.D) return;
  Vals<T, V> x[U], ga[U], gx[U];
  Vals<float, V> h[U];
  const int64_t b0 = (int64_t)blockIdx.y * U;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t b = b0 + u < p.batch ? b0 + u : b0;
    x[u] = *reinterpret_cast<const Vals<T, V>*>(static_cast<const T*>(p.x) + b * p.xs[0] + d);
    ga[u] = *reinterpret_cast<const Vals<T, V>*>(static_cast<const T*>(p.ga) + b * p.as[0] + d);
    gx[u] = *reinterpret_cast<const Vals<T, V>*>(static_cast<const T*>(p.gx) + b * p.gs[0] + d);
    if (p.init) h[u] = *reinterpret_cast<const Vals<float, V>*>(p.init + b * p.D + d);
  }
  float2 rate[P];
#pragma unroll
  for (int k = 0; k < P; ++k)
    rate[k] = make_float2(-p.c * softplus(p.decay[d + 2 * k]), V > 1 ? -p.c * softplus(p.decay[d + 2 * k + (V > 1)]) : 0.f);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    Vals<T, V> y;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      auto pair = [&](const Vals<T, V>& v) { return make_float2((float)v.v[2 * k], V > 1 ? (float)v.v[2 * k + (V > 1)] : 0.f); };
      const float2 c = decay<true>(log_decay<true>(rate[k], rcp2(one_plus_exp2(pair(ga[u])))));
      const float2 q = one_minus_a2<true>(c), i = rcp2(one_plus_exp2(pair(gx[u])));
      const float2 m = fp::mul2(q, make_float2(rsqrt_approx(q.x), rsqrt_approx(q.y)));
      float2 s = make_float2(0.f, 0.f);
      if (p.init) s = make_float2(h[u].v[2 * k], V > 1 ? h[u].v[2 * k + (V > 1)] : 0.f);
      s = step<kSafe>(c, fp::mul2(fp::mul2(m, i), pair(x[u])), s);
      h[u].v[2 * k] = s.x;
      st_from_f32(&y.v[2 * k], s.x);
      if (V > 1) {
        h[u].v[2 * k + (V > 1)] = s.y;
        st_from_f32(&y.v[2 * k + (V > 1)], s.y);
      }
    }
    const int64_t at = (b0 + u) * p.D + d;
    if (b0 + u < p.batch) {
      *reinterpret_cast<Vals<float, V>*>(p.final_state + at) = h[u];
      *reinterpret_cast<Vals<T, V>*>(static_cast<T*>(p.y) + at) = y;
    }
  }
}

constexpr int64_t kMinTileSteps = 64;   // no kernel's tile is shorter
constexpr int64_t kMaxElems = (int64_t)1 << 40;

ssd_status check_shape(const gated_recurrence_shape* s, bool backward) {
  if (!s || s->batch < 0 || s->seqlen < 0 || s->d_model < 1) return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_F32 && s->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (!(s->c > 0.f) || !isfinite(s->c)) return SSD_ERR_INVALID_ARG;
  for (int k = 0; k < 2; ++k)
    if (s->x_stride[k] < 0 || s->gate_a_stride[k] < 0 || s->gate_x_stride[k] < 0 ||
        (backward && s->dy_stride[k] < 0))
      return SSD_ERR_INVALID_ARG;
  if (s->d_model > 0x7fffff00LL || s->batch > 0x7fffffffLL || s->seqlen > 0x7fffffffLL || s->batch > kMaxElems / s->d_model ||
      (s->batch > 0 && s->seqlen > kMaxElems / s->d_model / s->batch))
    return SSD_ERR_UNSUPPORTED;
  // blocks of the per-channel kernels, and tiles (tickets are 32 bits)
  if ((s->batch * s->d_model + 127) / 128 > 0x7fffffffLL ||
      s->batch * ((s->d_model + 31) / 32) * ((s->seqlen + kMinTileSteps - 1) / kMinTileSteps) > 0x7f000000LL)
    return SSD_ERR_UNSUPPORTED;
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
  size_t scan = 0, states = 0, partial = 0, total = 0;   // scan: look-back words
};
RecLayout rec_layout(const gated_recurrence_shape* s, bool backward) {
  RecLayout L;
  size_t off = sizeof(WsHeader);
  L.scan = off;
  const int64_t ntile = (s->seqlen + kMinTileSteps - 1) / kMinTileSteps;
  if (ntile > 1)
    off = align_up(off + sizeof(uint64_t) * (size_t)(s->batch * ntile * align_up(s->d_model, 64)),
                   kWsAlign);
  if (backward) {
    L.states = off;
    const int64_t nch = (s->seqlen + kChunk - 1) / kChunk;
    off = align_up(off + sizeof(float) * (size_t)(s->batch * nch * s->d_model), kWsAlign);
    L.partial = off;
    off = align_up(off + sizeof(float) * (size_t)(s->batch * nch * s->d_model), kWsAlign);
  }
  L.total = off;
  return L;
}

cudaError_t set_rows(float* dst, const float* src, int64_t n, cudaStream_t st) {
  if (!dst || n == 0) return cudaSuccess;
  return src ? cudaMemcpyAsync(dst, src, sizeof(float) * (size_t)n, cudaMemcpyDeviceToDevice, st)
             : cudaMemsetAsync(dst, 0, sizeof(float) * (size_t)n, st);
}

// Alignment that every row of the arrays is known to have: 16, 8, 4 or (bf16) 2 bytes.
int row_align(size_t e, std::initializer_list<std::pair<const void*, const int64_t*>> in,
              std::initializer_list<const void*> out, int64_t D) {
  uint64_t bits = 0;
  for (const auto& a : in)
    bits |= reinterpret_cast<uintptr_t>(a.first) | (uint64_t)(a.second[0] | a.second[1]) * e;
  // an output row only needs its stores' 4 bytes
  uint64_t obits = (uint64_t)D * e;
  for (const void* o : out) obits |= reinterpret_cast<uintptr_t>(o);
  if (obits % 4 != 0) return 2;
  return bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
}

// A tile kernel: behind the clearing of its look-back words, or by itself where it has one tile in time.
template <typename T>
cudaError_t launch_tiles(void (*kernel)(RecParams), RecParams p, int blocks, unsigned threads, size_t smem,
                         cudaStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(blocks, p.tiles);
  if (p.ntile == 1) {
    p.ticket = nullptr;
    kernel<<<grid, threads, smem, st>>>(p);
    return cudaGetLastError();
  }
  const int64_t n = (int64_t)p.tiles * Tile<T>::kCh * (int64_t)sizeof(uint64_t) / 16;
  rec_clear_kernel<<<(unsigned)std::min<int64_t>((n + 255) / 256, 152 * 4), 256, 0, st>>>(
      reinterpret_cast<uint4*>(p.words), n);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? launch_next(kernel, grid, threads, smem, st, p) : e;
}

template <typename T, int ALIGN>
cudaError_t launch_forward_as(RecParams p, cudaStream_t st) {
  using F = Forward<T>;
  auto* kernel = rec_forward_kernel<T, ALIGN>;
  constexpr int kSmem = 2 * 3 * F::kSteps * kRowBytes;
  static_assert(F::kSteps >= kMinTileSteps, "the workspace is sized for tiles of kMinTileSteps");
  p.ntile = (p.T + F::kSteps - 1) / F::kSteps;
  p.cols = (uint32_t)((p.D + Tile<T>::kCh - 1) / Tile<T>::kCh);
  p.tiles = (uint32_t)(p.batch * p.cols * p.ntile);
  int blocks = 0;
  cudaError_t e = resident_blocks(kernel, 32 * F::kNw, kSmem, &blocks);
  if (e != cudaSuccess) return e;
  return launch_tiles<T>(kernel, p, blocks, 32 * F::kNw, kSmem, st);
}

// Tensor maps of the first n of x, gate_a, gate_x and dy in tiles of `steps`.
bool make_maps(RecParams& p, bool bf16, int steps, int n) {
  const void* base[4] = {p.x, p.ga, p.gx, p.dy};
  const int64_t* stride[4] = {p.xs, p.as, p.gs, p.ds};
  const int ch = bf16 ? Tile<__nv_bfloat16>::kCh : Tile<float>::kCh;
  for (int a = 0; a < n; ++a)
    if (!make_tensor_map(&p.map[a], bf16, base[a], p.batch, p.T, p.D, stride[a][0], stride[a][1], steps, ch))
      return false;
  return true;
}

cudaError_t launch_forward(RecParams p, bool bf16, cudaStream_t st) {
  const int align = row_align(bf16 ? 2 : 4, {{p.x, p.xs}, {p.ga, p.as}, {p.gx, p.gs}}, {p.y}, p.D);
  if (align == 16 && make_maps(p, bf16, bf16 ? Forward<__nv_bfloat16>::kSteps : Forward<float>::kSteps, 3))
    return bf16 ? launch_forward_as<__nv_bfloat16, kTma>(p, st) : launch_forward_as<float, kTma>(p, st);
  if (bf16)
    return align == 16 ? launch_forward_as<__nv_bfloat16, 16>(p, st)
         : align == 8 ? launch_forward_as<__nv_bfloat16, 8>(p, st)
         : align == 4 ? launch_forward_as<__nv_bfloat16, 4>(p, st)
                      : launch_forward_as<__nv_bfloat16, 2>(p, st);
  return align == 16 ? launch_forward_as<float, 16>(p, st)
       : align == 8 ? launch_forward_as<float, 8>(p, st)
                    : launch_forward_as<float, 4>(p, st);
}

template <typename T, int ALIGN>
cudaError_t launch_backward_as(RecParams p, cudaStream_t st) {
  auto* kernel = rec_backward_kernel<T, ALIGN, 2>;
  constexpr int kSmem = 2 * 4 * kWarps * kSpwBwd * kRowBytes;
  int blocks = 0;
  cudaError_t e = resident_blocks(kernel, kThreads, kSmem, &blocks);
  if (e != cudaSuccess) return e;
  if ((e = launch_tiles<T>(kernel, p, blocks, kThreads, kSmem, st)) != cudaSuccess) return e;
  return launch_next(rec_ddecay_kernel, (unsigned)((p.D + 31) / 32), 1024, 0, st, p);
}

cudaError_t launch_backward(RecParams p, bool bf16, cudaStream_t st) {
  p.ntile = p.nch;
  const int64_t ch = bf16 ? Tile<__nv_bfloat16>::kCh : Tile<float>::kCh;
  p.cols = (uint32_t)((p.D + ch - 1) / ch);
  p.tiles = (uint32_t)(p.batch * p.cols * p.ntile);
  const int align = row_align(bf16 ? 2 : 4, {{p.x, p.xs}, {p.ga, p.as}, {p.gx, p.gs}, {p.dy, p.ds}},
                              {p.dx, p.dga, p.dgx}, p.D);
  if (align == 16 && make_maps(p, bf16, kChunk, 4))
    return bf16 ? launch_backward_as<__nv_bfloat16, kTma>(p, st) : launch_backward_as<float, kTma>(p, st);
  if (bf16)
    return align == 16 ? launch_backward_as<__nv_bfloat16, 16>(p, st)
         : align == 8 ? launch_backward_as<__nv_bfloat16, 8>(p, st)
         : align == 4 ? launch_backward_as<__nv_bfloat16, 4>(p, st)
                      : launch_backward_as<__nv_bfloat16, 2>(p, st);
  return align == 16 ? launch_backward_as<float, 16>(p, st)
       : align == 8 ? launch_backward_as<float, 8>(p, st)
                    : launch_backward_as<float, 4>(p, st);
}

template <typename T, int V, int U>
cudaError_t launch_step_as(const RecParams& p, cudaStream_t st) {
  const int64_t cols = (p.D + 128 * V - 1) / (128 * V), rows = (p.batch + U - 1) / U;
  for (int64_t r0 = 0; r0 < rows; r0 += 65535) {   // gridDim.y
    RecParams q = p;
    const int64_t b0 = r0 * U;
    q.batch = p.batch - b0;
    q.x = static_cast<const T*>(p.x) + b0 * p.xs[0];
    q.ga = static_cast<const T*>(p.ga) + b0 * p.as[0];
    q.gx = static_cast<const T*>(p.gx) + b0 * p.gs[0];
    q.init = p.init ? p.init + b0 * p.D : nullptr;
    q.final_state = p.final_state + b0 * p.D;
    q.y = static_cast<T*>(p.y) + b0 * p.D;
    rec_step_kernel<T, V, U><<<dim3((unsigned)cols, (unsigned)std::min<int64_t>(65535, rows - r0)), 128, 0, st>>>(q);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t launch_step(const RecParams& p, cudaStream_t st) {
  const uint64_t bits = (reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.ga) |
                         reinterpret_cast<uintptr_t>(p.gx) | reinterpret_cast<uintptr_t>(p.y) |
                         (uint64_t)(p.xs[0] | p.as[0] | p.gs[0] | p.D) * sizeof(T));
  const uint64_t sbits = reinterpret_cast<uintptr_t>(p.init) | reinterpret_cast<uintptr_t>(p.final_state);
  if (bits % (4 * sizeof(T)) != 0 || sbits % 16 != 0) return launch_step_as<T, 1, 1>(p, st);
  // few sequences: every one to threads of its own, for the machine's sake
  return p.batch * p.D < (int64_t)152 * 1024 * 4 ? launch_step_as<T, 4, 1>(p, st) : launch_step_as<T, 4, 2>(p, st);
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
  char* ws = static_cast<char*>(workspace);
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.ticket = p.hdr->counters;
  p.words = reinterpret_cast<uint64_t*>(ws + rec_layout(shape, false).scan);
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
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.ticket = p.hdr->counters;
  p.words = reinterpret_cast<uint64_t*>(ws + L.scan);
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
  return done(launch_backward(p, bf16, st));
}

ssd_status gated_recurrence_step(const gated_recurrence_shape* shape, const void* x,
                                 const void* gate_a, const void* gate_x, const float* decay,
                                 const float* state, void* y, float* state_out, void* stream) {
  if (!shape) return SSD_ERR_INVALID_ARG;
  gated_recurrence_shape one = *shape;   // the step strides are ignored
  one.x_stride[1] = one.gate_a_stride[1] = one.gate_x_stride[1] = 0;
  const ssd_status bad = check_shape(&one, false);
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
  return done(bf16 ? launch_step<__nv_bfloat16>(p, st) : launch_step<float>(p, st));
}

}  // extern "C"
