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
#include <map>
#include <mutex>
#include <utility>

#include "common.cuh"
#include "fp_helpers.cuh"
#include "lookback.cuh"

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
  int64_t ntile;     // tiles in time
  uint32_t tiles;    // tiles in all
  uint32_t* ticket;  // NULL where the order of the tiles does not matter
  uint64_t* words;
  WsHeader* hdr;
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

// ------------------------------------------------------------------------------------------------
// Forward.
//
// The work is cut into tiles of kSteps steps by one 128-byte row of channels.  A block takes tiles
// by ticket, time-major, so a tile only ever waits for tiles with smaller tickets, which blocks
// hold that are running: every wait ends.  A warp owns SPW consecutive steps of the tile and loads
// them for itself (cp.async, the next tile's rows in flight while this one is computed), forms w and
// b = m i x once, in registers, and composes its steps into one map; the maps of the block's
// warps and, by look-back, of earlier tiles give the state before the warp's first step, and a
// second walk over the registers writes y.  Every input byte is read once.
// ------------------------------------------------------------------------------------------------
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowBytes = 128;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 dup(float v) { return make_float2(v, v); }
// 1 / (1 + e^-v); e^-v = inf gives 0
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 t = fp::mul2(v, dup(-kLog2e));
  const float2 d = make_float2(1.f + fp::ex2_approx(t.x), 1.f + fp::ex2_approx(t.y));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
// expm1(l) for l <= 0.  Above -1/4 the Taylor polynomial of degree 6, whose remainder l^6 / 5040 is
// 5e-8 of the value; below, 2^x - 1, whose error 2^-22 is at most 1e-6 of the value.  `far` is false
// where no channel of the warp can leave the polynomial's range (l >= -rate).
constexpr float kNear = 0.25f;
__device__ __forceinline__ float2 expm1_neg2(float2 l, bool far) {
  float2 q = fp::fma2(l, dup(1.f / 720), dup(1.f / 120));
  q = fp::fma2(q, l, dup(1.f / 24));
  q = fp::fma2(q, l, dup(1.f / 6));
  q = fp::fma2(q, l, dup(0.5f));
  float2 w = fp::fma2(fp::mul2(q, l), l, l);
  if (far) {
    if (l.x < -kNear) w.x = fp::ex2_approx(l.x * kLog2e) - 1.f;
    if (l.y < -kNear) w.y = fp::ex2_approx(l.y * kLog2e) - 1.f;
  }
  return w;
}
struct Gates2 {
  float2 r, i, w, m;
};
__device__ __forceinline__ Gates2 gates2(float2 ga, float2 gx, float2 rate, bool far) {
  Gates2 g;
  g.r = sigmoid2(ga);
  g.i = sigmoid2(gx);
  g.w = expm1_neg2(fp::mul2(fp::mul2(rate, g.r), dup(-1.f)), far);
  const float2 s = fp::fma2(g.w, dup(-1.f), dup(-2.f));   // -(2 + w)
  const float2 u = fp::mul2(g.w, s);                      // 1 - a^2
  g.m = make_float2(sqrt_approx(u.x), sqrt_approx(u.y));
  return g;
}

// Rows of one array for the calling warp: `rows` rows from step t0 on (rows at or past T become
// zeros, as do channels at or past D), kRowBytes each.  ALIGN is what every row start is known to be
// aligned to: 16 (one copy per 16 bytes), 4, or 2 (odd bf16 rows, through registers).
template <typename T, int ROWS, int ALIGN>
__device__ __forceinline__ void load_rows(unsigned char* dst, const T* src, int64_t row_stride, int64_t t0,
                                          int64_t Tlen, int64_t ch_left, int lane) {
  constexpr int kPer = ALIGN == 2 ? 4 : ALIGN;         // bytes a lane moves at a time
  constexpr int kLanes = kRowBytes / kPer;             // lanes a row takes
  constexpr int kRowsAtOnce = 32 / kLanes < 1 ? 1 : 32 / kLanes;
  const int64_t bytes_left = ch_left * (int64_t)sizeof(T);
#pragma unroll
  for (int r0 = 0; r0 < ROWS; r0 += kRowsAtOnce) {
    const int r = r0 + lane / kLanes, at = lane % kLanes * kPer;
    if (ROWS % kRowsAtOnce != 0 && r >= ROWS) continue;
    int64_t n = t0 + r < Tlen ? bytes_left - at : 0;
    n = n < 0 ? 0 : n > kPer ? kPer : n;
    const unsigned char* s =
        reinterpret_cast<const unsigned char*>(n > 0 ? src + (t0 + r) * row_stride : src) + (n > 0 ? at : 0);
    unsigned char* d = dst + r * kRowBytes + at;
    if constexpr (ALIGN == 16) {
      cp_async16(d, s, (int)n);
    } else if constexpr (ALIGN == 4) {
      if (n >= 4) cp_async4(d, s);
      else if (n == 2) *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint16_t*>(s);
      else *reinterpret_cast<uint32_t*>(d) = 0u;
    } else {
      uint32_t v = 0;
      if (n >= 2) v = *reinterpret_cast<const uint16_t*>(s);
      if (n >= 4) v |= (uint32_t)*reinterpret_cast<const uint16_t*>(s + 2) << 16;
      *reinterpret_cast<uint32_t*>(d) = v;
    }
  }
}

template <typename T>
struct Tile {
  static constexpr int kCh = kRowBytes / (int)sizeof(T);   // channels of a tile
  static constexpr int kCpl = kCh / 32;                    // channels of a lane
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

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

// Channel c of a lane in row s.
template <typename T>
__device__ __forceinline__ float dy_at(const unsigned char* rows, int s, int lane, int c) {
  return to_f32(*(reinterpret_cast<const T*>(rows + s * kRowBytes) + lane * Tile<T>::kCpl + c));
}

// Writes a lane's channels of one row; `n` of them are inside the array.
template <int ALIGN>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&v)[2], int n) {
  if (ALIGN >= 4 && n == 2) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
  } else {
    if (n > 0) p[0] = __float2bfloat16_rn(v[0]);
    if (n > 1) p[1] = __float2bfloat16_rn(v[1]);
  }
}
template <int ALIGN>
__device__ __forceinline__ void store_row(float* p, const float (&v)[1], int n) {
  if (n > 0) p[0] = v[0];
}

// Where a tile lies.  Tickets run over all columns of a time before the next time.
struct Place {
  int64_t b, c0, t0, ti, word;   // word: index of the tile's first look-back word
};
template <typename T, int STEPS, bool kReverse>
__device__ __forceinline__ Place place(const RecParams& p, uint32_t ticket) {
  constexpr int kCh = Tile<T>::kCh;
  const uint32_t cols = (uint32_t)((p.D + kCh - 1) / kCh), all = cols * (uint32_t)p.batch;
  const uint32_t k = ticket / all, col = ticket % all;
  Place q;
  q.ti = kReverse ? p.ntile - 1 - k : k;
  q.b = col / cols;
  q.c0 = (int64_t)(col % cols) * kCh;
  q.t0 = q.ti * STEPS;
  q.word = ((int64_t)col * p.ntile + q.ti) * kCh;
  return q;
}

template <typename T, int SPW, int ALIGN, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) rec_forward_kernel(RecParams p) {
  constexpr int kSteps = kWarps * SPW, kCh = Tile<T>::kCh, kCpl = Tile<T>::kCpl;
  constexpr int kVals = SPW * kCpl, kWarpBytes = SPW * kRowBytes, kStage = 3 * kWarps * kWarpBytes;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 maps[2][kWarps][kCh];   // (W, H) of every warp's steps
  __shared__ float before[2][kCh];          // the state before the tile
  __shared__ float rates[2][kCh];           // c softplus(decay) of the tile's channels
  __shared__ uint32_t s_ticket;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int cl = lane * kCpl;
  const T* src[3] = {static_cast<const T*>(p.x), static_cast<const T*>(p.ga), static_cast<const T*>(p.gx)};

  auto load = [&](uint32_t ticket, int stage) {
    if (ticket < p.tiles) {
      const Place q = place<T, kSteps, false>(p, ticket);
      const int64_t bs[3] = {p.xs[0], p.as[0], p.gs[0]}, ts[3] = {p.xs[1], p.as[1], p.gs[1]};
#pragma unroll
      for (int a = 0; a < 3; ++a)
        load_rows<T, SPW, ALIGN>(smem + stage * kStage + (a * kWarps + warp) * kWarpBytes,
                                 src[a] + q.b * bs[a] + q.c0, ts[a], q.t0 + warp * SPW, p.T, p.D - q.c0, lane);
    }
    cp_async_commit();
  };
  auto take = [&]() { return atomicAdd(p.ticket, 1u); };
  auto set_rates = [&](uint32_t ticket, int slot) {   // by one warp
    if (ticket >= p.tiles) return;
    const Place q = place<T, kSteps, false>(p, ticket);
#pragma unroll
    for (int c = 0; c < kCpl; ++c)
      rates[slot][cl + c] = q.c0 + cl + c < p.D ? p.c * softplus(p.decay[q.c0 + cl + c]) : 0.f;
  };

  uint32_t cur, nxt;
  if (p.ticket) {
    if (threadIdx.x == 0) s_ticket = take();
    __syncthreads();
    cur = s_ticket;
    __syncthreads();
    if (threadIdx.x == 0) s_ticket = take();
    __syncthreads();
    nxt = s_ticket;
  } else {   // one tile in time: no order to keep
    cur = blockIdx.x;
    nxt = cur + gridDim.x;
  }
  load(cur, 0);
  if (warp == 2) set_rates(cur, 0);
  __syncthreads();
  for (int it = 0; cur < p.tiles; ++it) {
    load(nxt, (it + 1) & 1);
    cp_async_wait<1>();
    __syncwarp();
    const Place q = place<T, kSteps, false>(p, cur);
    const int nch = (int)min((int64_t)kCpl, max((int64_t)0, p.D - q.c0 - cl));
    const float2 rate2 = make_float2(rates[it & 1][cl], rates[it & 1][cl + kCpl - 1]);
    const bool far = __any_sync(0xffffffffu, fmaxf(rate2.x, rate2.y) > kNear);

    const unsigned char* rows = smem + (it & 1) * kStage + warp * kWarpBytes;
    float w[kVals], b[kVals];   // value s * kCpl + c: step s, channel c
#pragma unroll
    for (int k = 0; k < kVals / 2; ++k) {
      const float2 x = pair_at(rows, k, lane, T());
      const Gates2 g = gates2(pair_at(rows + kWarps * kWarpBytes, k, lane, T()),
                              pair_at(rows + 2 * kWarps * kWarpBytes, k, lane, T()), rate2, far);
      const float2 bv = fp::mul2(fp::mul2(g.m, g.i), x);
      w[2 * k] = g.w.x, w[2 * k + 1] = g.w.y;
      b[2 * k] = bv.x, b[2 * k + 1] = bv.y;
    }
    const int64_t steps_left = p.T - q.t0 - warp * SPW;
    if (steps_left < SPW) {   // steps past the end change nothing
#pragma unroll
      for (int s = 0; s < SPW; ++s)
        if (s >= steps_left) {
#pragma unroll
          for (int c = 0; c < kCpl; ++c) w[s * kCpl + c] = b[s * kCpl + c] = 0.f;
        }
    }
#pragma unroll
    for (int c = 0; c < kCpl; ++c) {
      float W = 0.f, H = 0.f;
#pragma unroll
      for (int s = 0; s < SPW; ++s) {
        H = lookback::apply(w[s * kCpl + c], b[s * kCpl + c], H);
        W = lookback::apply(w[s * kCpl + c], w[s * kCpl + c], W);
      }
      maps[it & 1][warp][cl + c] = make_float2(W, H);
    }
    __syncthreads();
    uint32_t later = nxt + gridDim.x;
    if (warp == 0) {
      float W[kCpl], H[kCpl], h[kCpl];
#pragma unroll
      for (int c = 0; c < kCpl; ++c) {
        W[c] = H[c] = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float2 m = maps[it & 1][k][cl + c];
          H[c] = lookback::apply(m.x, m.y, H[c]);
          W[c] = lookback::apply(m.x, m.x, W[c]);
        }
      }
      uint64_t* words = p.words + q.word + cl;
      const bool last = q.ti == p.ntile - 1;
      uint64_t v[kCpl];
      if (q.ti == 0) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) h[c] = p.init && c < nch ? p.init[q.b * p.D + q.c0 + cl + c] : 0.f;
      } else {
        if (!last) {
#pragma unroll
          for (int c = 0; c < kCpl; ++c) v[c] = lookback::word(W[c], H[c], lookback::kMap);
          lookback::publish(words, v);
        }
        lookback::state_before<8>(words - kCh, -kCh, q.ti, h, p.hdr, 400);
      }
      if (!last) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c)
          v[c] = lookback::word(0.f, lookback::apply(W[c], H[c], h[c]), lookback::kInclusive);
        lookback::publish(words, v);
      }
#pragma unroll
      for (int c = 0; c < kCpl; ++c) before[it & 1][cl + c] = h[c];
    } else if (warp == 1) {
      if (p.ticket && lane == 0) s_ticket = take();
    } else if (warp == 2) {
      set_rates(nxt, (it + 1) & 1);
    }
    __syncthreads();
    if (p.ticket) later = s_ticket;
    float h[kCpl];
#pragma unroll
    for (int c = 0; c < kCpl; ++c) h[c] = before[it & 1][cl + c];
    for (int k = 0; k < warp; ++k) {
#pragma unroll
      for (int c = 0; c < kCpl; ++c) {
        const float2 m = maps[it & 1][k][cl + c];
        h[c] = lookback::apply(m.x, m.y, h[c]);
      }
    }
    if (p.states_out && warp * SPW % kChunk == 0 && steps_left > 0) {
      const int64_t at = (q.b * p.nch + (q.t0 + warp * SPW) / kChunk) * p.D + q.c0 + cl;
#pragma unroll
      for (int c = 0; c < kCpl; ++c)
        if (c < nch && SSD_INDEX_OK(p.hdr, at + c, p.batch * p.nch * p.D, 60)) p.states_out[at + c] = h[c];
    }
    const int64_t row0 = (q.b * p.T + q.t0 + warp * SPW) * p.D + q.c0 + cl;
    T* y = static_cast<T*>(p.y);
#pragma unroll
    for (int s = 0; s < SPW; ++s) {
#pragma unroll
      for (int c = 0; c < kCpl; ++c) h[c] = lookback::apply(w[s * kCpl + c], b[s * kCpl + c], h[c]);
      if (y && nch > 0 && s < steps_left &&
          SSD_INDEX_OK(p.hdr, row0 + s * p.D + nch - 1, p.batch * p.T * p.D, 61))
        store_row<ALIGN>(y + row0 + s * p.D, h, nch);
    }
    if (p.final_state && q.ti == p.ntile - 1 && warp == kWarps - 1) {
      const int64_t at = q.b * p.D + q.c0 + cl;
#pragma unroll
      for (int c = 0; c < kCpl; ++c)
        if (c < nch && SSD_INDEX_OK(p.hdr, at + c, p.batch * p.D, 62)) p.final_state[at + c] = h[c];
    }
    cur = nxt;
    nxt = later;
  }
  cp_async_wait_all();
}

// ------------------------------------------------------------------------------------------------
// Backward.
//
// The same tiles, from the last to the first; a tile's state comes from the states that the forward
// kept (one a tile), so only dL/dh is carried by look-back: C = a G, the gradient that a tile hands
// to the step before it, maps to C + W C + Q over a tile with the same W as the forward's.  A warp
// forms the forward maps of its steps, takes the state before them, walks them forward for
//   mi = m i,  xi = mi x (1 - i),  kr = a (h_{t-1} - a i x / m) r,  r   (kept in registers)
// and composes the reverse map; with C known a walk backwards gives G and writes
//   dx = G mi, dgate_x = G xi, dgate_a = -rate G kr (1 - r)   and sums G kr for ddecay.
// ddecay: one partial row per tile, added in tile order by rec_ddecay_kernel.
// ------------------------------------------------------------------------------------------------
constexpr int kSpwBwd = 8;
static_assert(kWarps * kSpwBwd == kChunk, "a backward tile starts from one kept state");

template <typename T, int ALIGN, int MINB, int STAGES>
__global__ void __launch_bounds__(kThreads, MINB) rec_backward_kernel(RecParams p) {
  constexpr int SPW = kSpwBwd, kSteps = kWarps * SPW, kCh = Tile<T>::kCh, kCpl = Tile<T>::kCpl;
  constexpr int kVals = SPW * kCpl, kWarpBytes = SPW * kRowBytes, kArray = kWarps * kWarpBytes;
  constexpr int kStage = 4 * kArray;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float2 maps[2][kWarps][kCh];   // forward (W, H) of every warp's steps
  __shared__ float2 back[2][kWarps][kCh];   // reverse (W, Q)
  __shared__ float after[2][kCh];           // C from the tile after
  __shared__ float sums[2][kWarps][kCh];    // G kr over every warp's steps
  __shared__ float rates[2][kCh], start[2][kCh];
  __shared__ uint32_t s_ticket;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int cl = lane * kCpl;
  const T* src[4] = {static_cast<const T*>(p.x), static_cast<const T*>(p.ga), static_cast<const T*>(p.gx),
                     static_cast<const T*>(p.dy)};

  auto load = [&](uint32_t ticket, int stage) {
    if (ticket < p.tiles) {
      const Place q = place<T, kSteps, true>(p, ticket);
      const int64_t bs[4] = {p.xs[0], p.as[0], p.gs[0], p.ds[0]}, ts[4] = {p.xs[1], p.as[1], p.gs[1], p.ds[1]};
#pragma unroll
      for (int a = 0; a < 4; ++a)
        load_rows<T, SPW, ALIGN>(smem + stage * kStage + a * kArray + warp * kWarpBytes,
                                 src[a] + q.b * bs[a] + q.c0, ts[a], q.t0 + warp * SPW, p.T, p.D - q.c0, lane);
    }
    cp_async_commit();
  };
  auto take = [&]() { return atomicAdd(p.ticket, 1u); };
  auto set_channels = [&](uint32_t ticket, int slot) {   // by one warp: rates and the kept state
    if (ticket >= p.tiles) return;
    const Place q = place<T, kSteps, true>(p, ticket);
#pragma unroll
    for (int c = 0; c < kCpl; ++c) {
      const int64_t d = q.c0 + cl + c;
      rates[slot][cl + c] = d < p.D ? p.c * softplus(p.decay[d]) : 0.f;
      start[slot][cl + c] = d < p.D ? p.states_in[(q.b * p.nch + q.ti) * p.D + d] : 0.f;
    }
  };

  uint32_t cur, nxt;
  if (p.ticket) {
    if (threadIdx.x == 0) s_ticket = take();
    __syncthreads();
    cur = s_ticket;
    __syncthreads();
    if (threadIdx.x == 0) s_ticket = take();
    __syncthreads();
    nxt = s_ticket;
  } else {
    cur = blockIdx.x;
    nxt = cur + gridDim.x;
  }
  load(cur, 0);
  if (warp == 2) set_channels(cur, 0);
  __syncthreads();
  for (int it = 0; cur < p.tiles; ++it) {
    const int slot = it & 1;
    load(nxt, (it + 1) % STAGES);
    cp_async_wait<1>();
    __syncwarp();
    const Place q = place<T, kSteps, true>(p, cur);
    const int nch = (int)min((int64_t)kCpl, max((int64_t)0, p.D - q.c0 - cl));
    const float2 rate2 = make_float2(rates[slot][cl], rates[slot][cl + kCpl - 1]);
    const bool far = __any_sync(0xffffffffu, fmaxf(rate2.x, rate2.y) > kNear);
    const int64_t steps_left = p.T - q.t0 - warp * SPW;

    const unsigned char* rows = smem + (it % STAGES) * kStage + warp * kWarpBytes;
    float w[kVals], mi[kVals], xi[kVals], kr[kVals], r[kVals];   // value s * kCpl + c
    float b[kVals];
#pragma unroll
    for (int k = 0; k < kVals / 2; ++k) {
      const float2 x = pair_at(rows, k, lane, T());
      const Gates2 g = gates2(pair_at(rows + kArray, k, lane, T()), pair_at(rows + 2 * kArray, k, lane, T()),
                              rate2, far);
      const float2 m = fp::mul2(g.m, g.i), bv = fp::mul2(m, x);
      const float2 ic = fp::fma2(g.i, dup(-1.f), dup(1.f));
      const float2 xv = fp::mul2(bv, ic);
      // a i x / m (0 where m is): what kr subtracts from h_{t-1}
      const float2 ix = fp::mul2(g.i, x);
      const float2 over = make_float2(g.m.x > 0.f ? rcp_approx(g.m.x) : 0.f, g.m.y > 0.f ? rcp_approx(g.m.y) : 0.f);
      const float2 a = fp::fma2(g.w, dup(1.f), dup(1.f));
      const float2 sub = fp::mul2(fp::mul2(a, ix), over);
      w[2 * k] = g.w.x, w[2 * k + 1] = g.w.y;
      b[2 * k] = bv.x, b[2 * k + 1] = bv.y;
      mi[2 * k] = m.x, mi[2 * k + 1] = m.y;
      xi[2 * k] = xv.x, xi[2 * k + 1] = xv.y;
      kr[2 * k] = sub.x, kr[2 * k + 1] = sub.y;
      r[2 * k] = g.r.x, r[2 * k + 1] = g.r.y;
    }
    if (steps_left < SPW) {   // steps past the end change nothing and hand nothing on
#pragma unroll
      for (int s = 0; s < SPW; ++s)
        if (s >= steps_left) {
#pragma unroll
          for (int c = 0; c < kCpl; ++c) {
            const int k = s * kCpl + c;
            w[k] = b[k] = mi[k] = xi[k] = kr[k] = 0.f;
          }
        }
    }
#pragma unroll
    for (int c = 0; c < kCpl; ++c) {
      float W = 0.f, H = 0.f;
#pragma unroll
      for (int s = 0; s < SPW; ++s) {
        H = lookback::apply(w[s * kCpl + c], b[s * kCpl + c], H);
        W = lookback::apply(w[s * kCpl + c], w[s * kCpl + c], W);
      }
      maps[slot][warp][cl + c] = make_float2(W, H);
    }
    // reverse map of the warp's steps: dy + C enters a step, a (dy + C) leaves it
    float Wq[kCpl], Q[kCpl];
#pragma unroll
    for (int c = 0; c < kCpl; ++c) Q[c] = 0.f;
#pragma unroll
    for (int s = SPW - 1; s >= 0; --s) {
#pragma unroll
      for (int c = 0; c < kCpl; ++c) {
        const float G = dy_at<T>(rows + 3 * kArray, s, lane, c) + Q[c];
        Q[c] = lookback::apply(w[s * kCpl + c], 0.f, G);
      }
    }
#pragma unroll
    for (int c = 0; c < kCpl; ++c) {
      Wq[c] = maps[slot][warp][cl + c].x;
      back[slot][warp][cl + c] = make_float2(Wq[c], Q[c]);
    }
    __syncthreads();
    uint32_t later = nxt + gridDim.x;
    if (warp == 0) {
      float W[kCpl], H[kCpl], C[kCpl];
#pragma unroll
      for (int c = 0; c < kCpl; ++c) {
        W[c] = H[c] = 0.f;
#pragma unroll
        for (int k = kWarps - 1; k >= 0; --k) {
          const float2 m = back[slot][k][cl + c];
          H[c] = lookback::apply(m.x, m.y, H[c]);
          W[c] = lookback::apply(m.x, m.x, W[c]);
        }
      }
      uint64_t* words = p.words + q.word + cl;
      uint64_t v[kCpl];
      if (q.ti == p.ntile - 1) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) C[c] = p.dfinal && c < nch ? p.dfinal[q.b * p.D + q.c0 + cl + c] : 0.f;
      } else {
        if (q.ti > 0) {
#pragma unroll
          for (int c = 0; c < kCpl; ++c) v[c] = lookback::word(W[c], H[c], lookback::kMap);
          lookback::publish(words, v);
        }
        lookback::state_before<8>(words + kCh, kCh, p.ntile - 1 - q.ti, C, p.hdr, 401);
      }
      if (q.ti > 0) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c)
          v[c] = lookback::word(0.f, lookback::apply(W[c], H[c], C[c]), lookback::kInclusive);
        lookback::publish(words, v);
      }
#pragma unroll
      for (int c = 0; c < kCpl; ++c) after[slot][cl + c] = C[c];
    } else if (warp == 1) {
      if (p.ticket && lane == 0) s_ticket = take();
    } else if (warp == 2) {
      set_channels(nxt, slot ^ 1);
    }
    // the state before the warp's steps, and kr of every step (before C is needed)
    {
      float h[kCpl];
#pragma unroll
      for (int c = 0; c < kCpl; ++c) h[c] = start[slot][cl + c];
      for (int k = 0; k < warp; ++k) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) {
          const float2 m = maps[slot][k][cl + c];
          h[c] = lookback::apply(m.x, m.y, h[c]);
        }
      }
#pragma unroll
      for (int s = 0; s < SPW; ++s) {
#pragma unroll
        for (int c = 0; c < kCpl; ++c) {
          const int k = s * kCpl + c;
          const float a = 1.f + w[k];
          const float prev = h[c];
          h[c] = lookback::apply(w[k], b[k], prev);
          kr[k] = s < steps_left ? a * (prev - kr[k]) * r[k] : 0.f;
        }
      }
    }
    __syncthreads();
    if (p.ticket) later = s_ticket;
    float C[kCpl], sum[kCpl];
#pragma unroll
    for (int c = 0; c < kCpl; ++c) {
      C[c] = after[slot][cl + c];
      sum[c] = 0.f;
    }
    for (int k = kWarps - 1; k > warp; --k) {
#pragma unroll
      for (int c = 0; c < kCpl; ++c) {
        const float2 m = back[slot][k][cl + c];
        C[c] = lookback::apply(m.x, m.y, C[c]);
      }
    }
    const int64_t row0 = (q.b * p.T + q.t0 + warp * SPW) * p.D + q.c0 + cl;
#pragma unroll
    for (int s = SPW - 1; s >= 0; --s) {
      float vx[kCpl], va[kCpl], vg[kCpl];
#pragma unroll
      for (int c = 0; c < kCpl; ++c) {
        const int k = s * kCpl + c;
        const float G = dy_at<T>(rows + 3 * kArray, s, lane, c) + C[c];
        const float e = G * kr[k];
        vx[c] = G * mi[k];
        vg[c] = G * xi[k];
        va[c] = -(c ? rate2.y : rate2.x) * e * (1.f - r[k]);
        sum[c] += e;
        C[c] = lookback::apply(w[k], 0.f, G);
      }
      if (nch > 0 && s < steps_left && SSD_INDEX_OK(p.hdr, row0 + s * p.D + nch - 1, p.batch * p.T * p.D, 63)) {
        store_row<ALIGN>(static_cast<T*>(p.dx) + row0 + s * p.D, vx, nch);
        store_row<ALIGN>(static_cast<T*>(p.dga) + row0 + s * p.D, va, nch);
        store_row<ALIGN>(static_cast<T*>(p.dgx) + row0 + s * p.D, vg, nch);
      }
    }
#pragma unroll
    for (int c = 0; c < kCpl; ++c) sums[slot][warp][cl + c] = sum[c];
    if (p.dinit && q.ti == 0 && warp == 0) {
      const int64_t at = q.b * p.D + q.c0 + cl;
#pragma unroll
      for (int c = 0; c < kCpl; ++c)
        if (c < nch && SSD_INDEX_OK(p.hdr, at + c, p.batch * p.D, 64)) p.dinit[at + c] = C[c];
    }
    __syncthreads();
    if (warp == 3) {   // the tile's row of ddecay partials
      const int64_t at = (q.b * p.nch + q.ti) * p.D + q.c0 + cl;
#pragma unroll
      for (int c = 0; c < kCpl; ++c) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) v += sums[slot][k][cl + c];
        if (c < nch && SSD_INDEX_OK(p.hdr, at + c, p.batch * p.nch * p.D, 65)) p.partial[at + c] = v;
      }
    }
    cur = nxt;
    nxt = later;
  }
  cp_async_wait_all();
}

// ddecay[d] = -c sigmoid(decay) * sum of the partial rows: a block takes 32 channels, its warps every
// 32nd row each, joined in warp order.
__global__ void __launch_bounds__(1024) rec_ddecay_kernel(RecParams p) {
  __shared__ float part[32][33];
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
  if (s->d_model > kMaxElems || s->batch > kMaxElems / s->d_model ||
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
  size_t scan = 0, states = 0, partial = 0, total = 0;   // scan: ticket, then look-back words
};
RecLayout rec_layout(const gated_recurrence_shape* s, bool backward) {
  RecLayout L;
  size_t off = sizeof(WsHeader);
  L.scan = off;
  const int64_t ntile = (s->seqlen + kMinTileSteps - 1) / kMinTileSteps;
  if (ntile > 1)
    off = align_up(off + kWsAlign + sizeof(uint64_t) * (size_t)(s->batch * ntile * align_up(s->d_model, 64)),
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

constexpr int kSpwFwd = 8;   // steps a warp takes of a forward tile
constexpr int64_t kTileSteps = kWarps * kSpwFwd;

// Alignment that every row of the arrays is known to have: 16, 4 or (bf16) 2 bytes.
int row_align(size_t e, std::initializer_list<std::pair<const void*, const int64_t*>> in,
              std::initializer_list<const void*> out, int64_t D) {
  uint64_t bits = 0;
  for (const auto& a : in)
    bits |= reinterpret_cast<uintptr_t>(a.first) | (uint64_t)(a.second[0] | a.second[1]) * e;
  // an output row only needs its stores' 4 bytes
  uint64_t obits = (uint64_t)D * e;
  for (const void* o : out) obits |= reinterpret_cast<uintptr_t>(o);
  if (obits % 4 != 0) return 2;
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 2;
}

// Blocks of `kernel` that the device holds at once (looked up once per kernel and device).
template <typename K>
cudaError_t resident_blocks(K* kernel, int threads, int smem, int* out) {
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, int> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_pair(reinterpret_cast<const void*>(kernel), dev);
  const auto it = known.find(key);
  if (it != known.end()) {
    *out = it->second;
    return cudaSuccess;
  }
  int sms = 0, per = 0;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  *out = known[key] = sms * std::max(per, 1);
  return cudaSuccess;
}

template <typename T, int ALIGN>
cudaError_t launch_forward_as(RecParams p, cudaStream_t st) {
  auto* kernel = rec_forward_kernel<T, kSpwFwd, ALIGN, 3>;
  constexpr int kSmem = 2 * 3 * kWarps * kSpwFwd * kRowBytes;
  int blocks = 0;
  cudaError_t e = resident_blocks(kernel, kThreads, kSmem, &blocks);
  if (e != cudaSuccess) return e;
  if (p.ntile > 1) {   // tickets and look-back words start at zero
    const size_t n = kWsAlign + sizeof(uint64_t) * (size_t)p.tiles * Tile<T>::kCh;
    if ((e = cudaMemsetAsync(p.ticket, 0, n, st)) != cudaSuccess) return e;
  } else {
    p.ticket = nullptr;
  }
  kernel<<<(unsigned)std::min<int64_t>(blocks, p.tiles), kThreads, kSmem, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_forward(RecParams p, bool bf16, cudaStream_t st) {
  p.ntile = (p.T + kTileSteps - 1) / kTileSteps;
  const int64_t ch = bf16 ? Tile<__nv_bfloat16>::kCh : Tile<float>::kCh;
  p.tiles = (uint32_t)(p.batch * ((p.D + ch - 1) / ch) * p.ntile);
  const int align = row_align(bf16 ? 2 : 4, {{p.x, p.xs}, {p.ga, p.as}, {p.gx, p.gs}}, {p.y}, p.D);
  if (bf16)
    return align == 16 ? launch_forward_as<__nv_bfloat16, 16>(p, st)
         : align == 4 ? launch_forward_as<__nv_bfloat16, 4>(p, st)
                      : launch_forward_as<__nv_bfloat16, 2>(p, st);
  return align == 16 ? launch_forward_as<float, 16>(p, st) : launch_forward_as<float, 4>(p, st);
}

template <typename T, int ALIGN>
cudaError_t launch_backward_as(RecParams p, cudaStream_t st) {
  auto* kernel = rec_backward_kernel<T, ALIGN, 2, 2>;
  constexpr int kSmem = 2 * 4 * kWarps * kSpwBwd * kRowBytes;
  int blocks = 0;
  cudaError_t e = resident_blocks(kernel, kThreads, kSmem, &blocks);
  if (e != cudaSuccess) return e;
  if (p.ntile > 1) {
    const size_t n = kWsAlign + sizeof(uint64_t) * (size_t)p.tiles * Tile<T>::kCh;
    if ((e = cudaMemsetAsync(p.ticket, 0, n, st)) != cudaSuccess) return e;
  } else {
    p.ticket = nullptr;
  }
  kernel<<<(unsigned)std::min<int64_t>(blocks, p.tiles), kThreads, kSmem, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  rec_ddecay_kernel<<<(unsigned)((p.D + 31) / 32), 1024, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_backward(RecParams p, bool bf16, cudaStream_t st) {
  p.ntile = p.nch;
  const int64_t ch = bf16 ? Tile<__nv_bfloat16>::kCh : Tile<float>::kCh;
  p.tiles = (uint32_t)(p.batch * ((p.D + ch - 1) / ch) * p.ntile);
  const int align = row_align(bf16 ? 2 : 4, {{p.x, p.xs}, {p.ga, p.as}, {p.gx, p.gs}, {p.dy, p.ds}},
                              {p.dx, p.dga, p.dgx}, p.D);
  if (bf16)
    return align == 16 ? launch_backward_as<__nv_bfloat16, 16>(p, st)
         : align == 4 ? launch_backward_as<__nv_bfloat16, 4>(p, st)
                      : launch_backward_as<__nv_bfloat16, 2>(p, st);
  return align == 16 ? launch_backward_as<float, 16>(p, st) : launch_backward_as<float, 4>(p, st);
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
  p.ticket = reinterpret_cast<uint32_t*>(ws + rec_layout(shape, false).scan);
  p.words = reinterpret_cast<uint64_t*>(reinterpret_cast<char*>(p.ticket) + kWsAlign);
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
  p.ticket = reinterpret_cast<uint32_t*>(ws + L.scan);
  p.words = reinterpret_cast<uint64_t*>(ws + L.scan + kWsAlign);
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
