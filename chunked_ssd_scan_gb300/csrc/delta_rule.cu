// Gated delta rule (declarations in include/ssdscan.h), step by step on the CUDA cores:
//   S_t = a_t S_{t-1} + u_t k_t^T,  u_t = beta_t e_t,  e_t = v_t - a_t S_{t-1} k_t,  a = exp(g),  y_t = scale S_t q_t
// and its reverse mode with G_t the gradient of S_t:
//   G_t += scale dy_t q_t^T;  du_t = G_t k_t;  dv_t = beta_t du_t;  dbeta_t = du_t . e_t
//   G_{t-1} = a_t (G_t - dv_t k_t^T)
// G does not depend on S, so a walk backwards gives du and the G before every chunk; all else follows chunk by
// chunk, in parallel, from the states and gradients at the chunks' borders (D_i = decay up to step i of the
// chunk, E_i = behind it, M_ij = between):
//   dq_i = scale (D_i S^T dy_i + sum_j<=i M_ij (dy_i . u_j) k_j)
//   dk_i = E_i G^T u_i - D_i S^T dv_i + scale sum_j>=i M_ji (dy_j . u_i) q_j
//          - sum_j<i M_ij (dv_i . u_j) k_j - sum_j>i M_ji (dv_j . u_i) k_j
//   dg_i = D_last <G, S> + sum_{a >= i} D_a (scale q_a . S^T dy_a - k_a . S^T dv_a) + sum_{b < i} E_b k_b . G^T u_b
//          + sum_{a >= i > b} M_ab (scale (dy_a . u_b) (q_a . k_b) - (dv_a . u_b) (k_a . k_b))
// that is, every product that the decay of step i is a factor of.  (The shorter <dS, S> before the chunk less the sum of
// q . dq - dv . v over the steps before i cancels: behind a reset of a state of size 1000 dg was off by 1e-3.)
#include <string.h>

#include <algorithm>
#include <initializer_list>

#include "delta_tc.cuh"
#include "launch.h"
#include "pack.cuh"

namespace ssd {
namespace {

using namespace delta;

// Steps whose rows are in shared memory at once, with the next ones on their way: 16 steps take longer than a load from
// DRAM; with 256 keys their registers only do for 8.
template <int KE>
constexpr int kTileOf = KE > 16 ? 8 : 16;
constexpr int kThreads = 128;

// Where lane l of a row's eight keeps element e of its KE: four neighbours, then 32 further.
__device__ __forceinline__ int key_of(int e, int l) { return (e >> 2) * 32 + l * 4 + (e & 3); }

__device__ __forceinline__ float sum8(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  v += __shfl_xor_sync(0xffffffffu, v, 2);
  return v + __shfl_xor_sync(0xffffffffu, v, 4);
}

// A warp's eight lanes hold a row's K values, R rows each; the rows do not meet, so a block is a slice of 16 R of V.
template <int KE, int R>
struct Walk {
  float s[R][KE];
  int l, row[R];   // row within the slice
  __device__ __forceinline__ Walk() {
    l = threadIdx.x & 7;
#pragma unroll
    for (int r = 0; r < R; ++r) row[r] = (threadIdx.x >> 3) + 16 * r;
  }
  __device__ __forceinline__ void load(const float* base, int64_t v0, int64_t V, int64_t K) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < KE; ++e)
        s[r][e] = base && v0 + row[r] < V && key_of(e, l) < K ? base[(v0 + row[r]) * K + key_of(e, l)] : 0.f;
  }
  // Over the state `cell` of `cells` in `base`.
  __device__ __forceinline__ void store(const Params& p, float* base, int64_t cell, int64_t cells, int site, int64_t v0) const {
    float* to = base + cell * p.K * p.V;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < KE; ++e) {
        const int64_t at = (v0 + row[r]) * p.K + key_of(e, l);
        if (v0 + row[r] < p.V && key_of(e, l) < p.K &&
            SSD_INDEX_OK(p.hdr, cell * p.K * p.V + at, cells * p.K * p.V, site))
          to[at] = s[r][e];
      }
  }
};

template <int KE>
__device__ __forceinline__ void row_of(float (&f)[KE], const float* sm, int l) {
#pragma unroll
  for (int e = 0; e < KE; e += 4) {
    const float4 v = *reinterpret_cast<const float4*>(sm + key_of(e, l));
    f[e] = v.x;
    f[e + 1] = v.y;
    f[e + 2] = v.z;
    f[e + 3] = v.w;
  }
}

// Steps [t, t + kTile) of q, k, a slice of v (or dy) and the gates, one tile ahead in registers.
template <typename T, int KE, int R>
struct TileLoad {
  static constexpr int kRows = 16 * R;
  static constexpr int kTile = kTileOf<KE>;
  static constexpr int kKeys = KE * 8, kPer = kTile * kKeys / kThreads;
  static constexpr int kVals = kTile * kRows / kThreads;
  float q[kPer], k[kPer], v[kVals], gate;
  __device__ __forceinline__ void fetch(const Params& p, const T* vbase, int64_t vstep, int64_t b, int64_t h,
                                        int64_t v0, int64_t t, int64_t end) {
    const int64_t hk = h / (p.H / p.Hk);
    const T* qb = static_cast<const T*>(p.q) + b * p.qs[0] + hk * p.qs[2];
    const T* kb = static_cast<const T*>(p.k) + b * p.ks[0] + hk * p.ks[2];
#pragma unroll
    for (int n = 0; n < kPer; ++n) {
      const int at = n * kThreads + threadIdx.x, i = at / kKeys, c = at % kKeys;
      const bool in = t + i < end && c < p.K;
      q[n] = in ? ld_f32(qb + (t + i) * p.qs[1] + c) : 0.f;
      k[n] = in ? ld_f32(kb + (t + i) * p.ks[1] + c) : 0.f;
    }
#pragma unroll
    for (int n = 0; n < kVals; ++n) {
      const int at = n * kThreads + threadIdx.x, i = at / kRows, c = at % kRows;
      v[n] = t + i < end && v0 + c < p.V ? ld_f32(vbase + (t + i) * vstep + v0 + c) : 0.f;
    }
    gate = threadIdx.x < kTile ? 1.f : 0.f;   // past the end: a decay of one and no write, so no step needs a branch
    if (threadIdx.x < 2 * kTile) {
      const int64_t at = t + (threadIdx.x & (kTile - 1));
      if (at < end)
        gate = threadIdx.x < kTile ? expf(decay_log(p, b, at, h)) : __ldg(p.beta + b * p.bs[0] + at * p.bs[1] + h);
    }
  }
};
template <int KE, int R>
struct Tile {
  static constexpr int kRows = 16 * R;
  static constexpr int kTile = kTileOf<KE>;
  float q[kTile][KE * 8], k[kTile][KE * 8], v[kTile][kRows], out[kTile][kRows], err[kTile][kRows];
  float gate[2 * kTile];   // decays, betas
  template <typename T>
  __device__ __forceinline__ void put(const TileLoad<T, KE, R>& r) {
#pragma unroll
    for (int n = 0; n < TileLoad<T, KE, R>::kPer; ++n) {
      const int at = n * kThreads + threadIdx.x;
      (&q[0][0])[at] = r.q[n];
      (&k[0][0])[at] = r.k[n];
    }
#pragma unroll
    for (int n = 0; n < TileLoad<T, KE, R>::kVals; ++n) (&v[0][0])[n * kThreads + threadIdx.x] = r.v[n];
    if (threadIdx.x < 2 * kTile) gate[threadIdx.x] = r.gate;
  }
};

// Forward.  One chunk a block where the states before the chunks are known (backward: only err is wanted then).
template <typename T, int KE, int R>
__global__ void __launch_bounds__(kThreads) delta_walk_kernel(const __grid_constant__ Params p, bool by_chunk) {
  constexpr int kTile = kTileOf<KE>, kRows = 16 * R;
  __shared__ __align__(16) Tile<KE, R> sm;
  int64_t id = blockIdx.x;
  const int64_t slice = id % p.slices;
  id /= p.slices;
  const int64_t h = id % p.H;
  id /= p.H;
  const int64_t chunk = by_chunk ? id % p.nch : 0, b = by_chunk ? id / p.nch : id;
  const int64_t v0 = slice * kRows, begin = chunk * kChunk, end = by_chunk ? min(begin + kChunk, p.T) : p.T;
  const int64_t KV = p.K * p.V;
  Walk<KE, R> w;
  w.load(by_chunk ? p.states_in + ((b * p.nch + chunk) * p.H + h) * KV
                  : p.init ? p.init + (b * p.H + h) * KV : nullptr, v0, p.V, p.K);
  const T* vbase = static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[2];
  TileLoad<T, KE, R> next;
  next.fetch(p, vbase, p.vs[1], b, h, v0, begin, end);
  for (int64_t t = begin; t < end; t += kTile) {
    __syncthreads();
    sm.put(next);
    __syncthreads();
    if (t + kTile < end) next.fetch(p, vbase, p.vs[1], b, h, v0, t + kTile, end);
    if (p.states_out && t % kChunk == 0)
      w.store(p, p.states_out, (b * p.nch + t / kChunk) * p.H + h, p.batch * p.nch * p.H, 2004, v0);
    const int n = (int)min((int64_t)kTile, end - t);
    // The outputs' sums over a row's lanes wait until all steps of the tile are through: on the way from one step to the
    // next lies only the product with k.  (With them in between a step took 660 cycles.)
    float part[R][kTile];
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      float kk[KE];
      row_of(kk, sm.k[i], w.l);
      const float a = sm.gate[i], beta = sm.gate[kTile + i];
      float u[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
#pragma unroll
        for (int e = 0; e < KE; e += 4) {
          d0 = fmaf(w.s[r][e], kk[e], d0);
          d1 = fmaf(w.s[r][e + 1], kk[e + 1], d1);
          d2 = fmaf(w.s[r][e + 2], kk[e + 2], d2);
          d3 = fmaf(w.s[r][e + 3], kk[e + 3], d3);
        }
        const float err = fmaf(-a, sum8((d0 + d1) + (d2 + d3)), sm.v[i][w.row[r]]);
        u[r] = i < n ? beta * err : 0.f;   // past the end a state of infinities would give NaN
        if (w.l == 0 && p.err) sm.err[i][w.row[r]] = err;
      }
      float qq[KE];
      row_of(qq, sm.q[i], w.l);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int e = 0; e < KE; e += 2) {
          w.s[r][e] = fmaf(a, w.s[r][e], u[r] * kk[e]);
          w.s[r][e + 1] = fmaf(a, w.s[r][e + 1], u[r] * kk[e + 1]);
          o0 = fmaf(w.s[r][e], qq[e], o0);
          o1 = fmaf(w.s[r][e + 1], qq[e + 1], o1);
        }
        part[r][i] = o0 + o1;
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i0 = 0; i0 < kTile; i0 += 8) {   // lane l of a row's eight gets the sum of step l
#pragma unroll
        for (int o = 4; o; o >>= 1)
#pragma unroll
          for (int j = i0; j < i0 + o; ++j) {
            const bool upper = w.l & o;
            const float keep = upper ? part[r][j + o] : part[r][j], give = upper ? part[r][j] : part[r][j + o];
            part[r][j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        sm.out[i0 + w.l][w.row[r]] = part[r][i0] * p.scale;
      }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kTile * kRows / kThreads; ++m) {
      const int at = m * kThreads + threadIdx.x, i = at / kRows, c = at % kRows;
      if (i < n && v0 + c < p.V) {
        const int64_t to = ((b * p.T + t + i) * p.H + h) * p.V + v0 + c;
        if (!SSD_INDEX_OK(p.hdr, to, p.batch * p.T * p.H * p.V, 2001)) continue;
        if (p.y) st_from_f32(static_cast<T*>(p.y) + to, sm.out[i][c]);
        if (p.err) p.err[to] = sm.err[i][c];
      }
    }
  }
  if (p.final_state) w.store(p, p.final_state, b * p.H + h, p.batch * p.H, 2005, v0);
}

// Backward: G along time, last step first.
template <typename T, int KE, int R>
__global__ void __launch_bounds__(kThreads) delta_walk_back_kernel(const __grid_constant__ Params p) {
  constexpr int kTile = kTileOf<KE>, kRows = 16 * R;
  __shared__ __align__(16) Tile<KE, R> sm;
  int64_t id = blockIdx.x;
  const int64_t slice = id % p.slices;
  id /= p.slices;
  const int64_t h = id % p.H, b = id / p.H, v0 = slice * kRows, KV = p.K * p.V;
  Walk<KE, R> w;
  w.load(p.dfinal ? p.dfinal + (b * p.H + h) * KV : nullptr, v0, p.V, p.K);
  const T* dyb = static_cast<const T*>(p.dy) + b * p.ds[0] + h * p.ds[2];
  TileLoad<T, KE, R> next;
  const int64_t first = (p.T - 1) / kTile * kTile;
  next.fetch(p, dyb, p.ds[1], b, h, v0, first, p.T);
  for (int64_t t = first; t >= 0; t -= kTile) {
    __syncthreads();
    sm.put(next);
    __syncthreads();
    if (t >= kTile) next.fetch(p, dyb, p.ds[1], b, h, v0, t - kTile, p.T);
    const int n = (int)min((int64_t)kTile, p.T - t);
#pragma unroll
    for (int i = kTile - 1; i >= 0; --i) {
      float kk[KE], qq[KE];
      row_of(kk, sm.k[i], w.l);
      row_of(qq, sm.q[i], w.l);
      const float a = sm.gate[i], beta = sm.gate[kTile + i];
      float dv[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float dy = sm.v[i][w.row[r]] * p.scale;
        float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
#pragma unroll
        for (int e = 0; e < KE; e += 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w.s[r][e + j] = fmaf(dy, qq[e + j], w.s[r][e + j]);
          d0 = fmaf(w.s[r][e], kk[e], d0);
          d1 = fmaf(w.s[r][e + 1], kk[e + 1], d1);
          d2 = fmaf(w.s[r][e + 2], kk[e + 2], d2);
          d3 = fmaf(w.s[r][e + 3], kk[e + 3], d3);
        }
        const float du = sum8((d0 + d1) + (d2 + d3));
        dv[r] = i < n ? beta * du : 0.f;
        if (w.l == 0) {
          sm.err[i][w.row[r]] = du;
          sm.out[i][w.row[r]] = dv[r];
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < KE; ++e) w.s[r][e] = a * fmaf(-dv[r], kk[e], w.s[r][e]);
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < kTile * kRows / kThreads; ++m) {
      const int at = m * kThreads + threadIdx.x, i = at / kRows, c = at % kRows;
      if (i < n && v0 + c < p.V) {
        const int64_t to = ((b * p.T + t + i) * p.H + h) * p.V + v0 + c;
        if (!SSD_INDEX_OK(p.hdr, to, p.batch * p.T * p.H * p.V, 2002)) continue;
        p.du[to] = sm.err[i][c];
        st_from_f32(static_cast<T*>(p.dv) + to, sm.out[i][c]);
      }
    }
    if (t % kChunk == 0) w.store(p, p.dstates, (b * p.nch + t / kChunk) * p.H + h, p.batch * p.nch * p.H, 2006, v0);
  }
  if (p.dinit) w.store(p, p.dinit, b * p.H + h, p.batch * p.H, 2007, v0);
}

// dq, dk and the part of dg of one chunk and key head, 64 of its keys a block: five products over V in slabs of 16
// values, then the four of the chunk's steps with each other.  (4 x 4096 x 16 heads of 128 x 128 f32:
// 2.7 of the backward call's 5.6 ms; 255 registers, one block an SM.)
constexpr int kGradThreads = 256, kSlab = 16, kPitch = 68;
struct GradSmem {
  float dy[kSlab][kPitch], u[kSlab][kPitch], dv[kSlab][kPitch];   // [value][step]
  float s[kSlab][kPitch], g[kSlab][kPitch];                       // [value][key]
  float b[kChunk][kPitch], n[kChunk][kPitch];                     // [step][step]
  float q[kChunk][kPitch], k[kChunk][kPitch];                     // [step][key]
  float qk[kChunk][kPitch], kk[kChunk][kPitch];                   // [step][step]: products of these keys
  float sum[kGradThreads / 32];
  float read[kChunk], wrote[kChunk];                              // of dg: what step a reads of S; what step b writes to G
  ChunkDecay c;
};

__device__ __forceinline__ void outer(float (&acc)[4][4], const float4& x, const float4& y) {
  const float a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
}
__device__ __forceinline__ float4 four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float sum) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, sum))));
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kGradThreads) delta_chunk_grad_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) unsigned char raw[];
  GradSmem& sm = *reinterpret_cast<GradSmem*>(raw);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  int64_t id = blockIdx.x;
  const int64_t hk = id % p.Hk;
  id /= p.Hk;
  const int64_t chunk = id % p.nch, b = id / p.nch, t0 = chunk * kChunk, k0 = (int64_t)blockIdx.y * 64;
  const int n = (int)min((int64_t)kChunk, p.T - t0);
  const int64_t group = p.H / p.Hk, KV = p.K * p.V;
  for (int at = tid; at < kChunk * 64; at += kGradThreads) {
    const int i = at >> 6, c = at & 63;
    const bool in = i < n && k0 + c < p.K;
    sm.q[i][c] = in ? ld_f32(static_cast<const T*>(p.q) + b * p.qs[0] + (t0 + i) * p.qs[1] + hk * p.qs[2] + k0 + c) : 0.f;
    sm.k[i][c] = in ? ld_f32(static_cast<const T*>(p.k) + b * p.ks[0] + (t0 + i) * p.ks[1] + hk * p.ks[2] + k0 + c) : 0.f;
  }
  __syncthreads();
  {   // columns 16 apart: neighbouring lanes' rows on different banks
    float qk[4][4] = {}, kk[4][4] = {};
#pragma unroll 2
    for (int m = 0; m < 64; m += 4) {
      float4 col[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) col[j] = four(&sm.k[tx + 16 * j][m]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 q = four(&sm.q[ty * 4 + i][m]), k = four(&sm.k[ty * 4 + i][m]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qk[i][j] = dot4(q, col[j], qk[i][j]);
          kk[i][j] = dot4(k, col[j], kk[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sm.qk[ty * 4 + i][tx + 16 * j] = qk[i][j];
        sm.kk[ty * 4 + i][tx + 16 * j] = kk[i][j];
      }
  }
  float dq[4][4] = {}, dk[4][4] = {};
  for (int64_t h = hk * group; h < (hk + 1) * group; ++h) {
    __syncthreads();
    if (tid < 32) chunk_decay_warp(p, sm.c, b, t0, n, h, tid);
    __syncthreads();
    const float* S = p.states_in + ((b * p.nch + chunk) * p.H + h) * KV;
    const float* G = chunk + 1 < p.nch ? p.dstates + ((b * p.nch + chunk + 1) * p.H + h) * KV : p.dfinal ? p.dfinal + (b * p.H + h) * KV : nullptr;
    float x1[4][4] = {}, x2[4][4] = {}, x3[4][4] = {}, bb[4][4] = {}, nn[4][4] = {};
    float inner = 0.f;
    for (int64_t v0 = 0; v0 < p.V; v0 += kSlab) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int at = m * kGradThreads + tid, i = at >> 4, c = at & 15;
        const bool in = i < n && v0 + c < p.V;
        const int64_t to = ((b * p.T + t0 + i) * p.H + h) * p.V + v0 + c;
        const float beta = sm.c.beta[i];
        sm.dy[c][i] = in ? ld_f32(static_cast<const T*>(p.dy) + b * p.ds[0] + (t0 + i) * p.ds[1] + h * p.ds[2] + v0 + c) : 0.f;
        sm.u[c][i] = in ? beta * p.err[to] : 0.f;
        sm.dv[c][i] = in ? beta * p.du[to] : 0.f;
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int at = m * kGradThreads + tid, r = at >> 6, c = at & 63;
        const bool in = v0 + r < p.V && k0 + c < p.K;
        const int64_t to = (v0 + r) * p.K + k0 + c;
        const float s = in ? S[to] : 0.f, g = in && G ? G[to] : 0.f;
        sm.s[r][c] = s;
        sm.g[r][c] = g;
        inner = fmaf(s, g, inner);
      }
      __syncthreads();
#pragma unroll 4
      for (int r = 0; r < kSlab; ++r) {
        const float4 dy = four(&sm.dy[r][ty * 4]), u = four(&sm.u[r][ty * 4]), dv = four(&sm.dv[r][ty * 4]);
        const float4 uj = four(&sm.u[r][tx * 4]), s = four(&sm.s[r][tx * 4]), g = four(&sm.g[r][tx * 4]);
        outer(x1, dy, s);
        outer(x2, u, g);
        outer(x3, dv, s);
        outer(bb, dy, uj);
        outer(nn, dv, uj);
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = ty * 4 + i, c = tx * 4 + j;
        const float m = c <= r ? decay_between(sm.c, r, c) : 0.f;
        sm.b[r][c] = c <= r ? p.scale * m * bb[i][j] : 0.f;   // a bad value of a later step stays out
        if (c <= r) {   // symmetric: both steps' k gradients take it
          const float v = c < r ? -m * nn[i][j] : 0.f;
          sm.n[r][c] = v;
          sm.n[c][r] = v;
        }
      }
    __syncthreads();
    float dqh[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      const float from = sm.c.from[r], to = sm.c.to[r];
      float read = 0.f, wrote = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float q1 = p.scale * from * x1[i][j], wr = to * x2[i][j], r1 = from * x3[i][j];
        const float q = sm.q[r][tx * 4 + j], k = sm.k[r][tx * 4 + j];
        dqh[i][j] = q1;
        dk[i][j] += wr - r1;
        read += q * q1 - k * r1;
        wrote = fmaf(k, wr, wrote);
      }
      read = sum16(read);
      wrote = sum16(wrote);
      if (tx == 0) {
        sm.read[r] = read;
        sm.wrote[r] = wrote;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
    if ((tid & 31) == 0) sm.sum[tid >> 5] = inner;
#pragma unroll 4
    for (int m = 0; m < kChunk; ++m) {
      const float4 q = four(&sm.q[m][tx * 4]), k = four(&sm.k[m][tx * 4]);
      outer(dqh, make_float4(sm.b[ty * 4][m], sm.b[ty * 4 + 1][m], sm.b[ty * 4 + 2][m], sm.b[ty * 4 + 3][m]), k);
      outer(dk, four(&sm.b[m][ty * 4]), q);
      outer(dk, four(&sm.n[m][ty * 4]), k);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) dq[i][j] += dqh[i][j];
    __syncthreads();
    // dg over these keys.  The pairs a > b, summed along a's row before every step, in b's place (four threads a row), ...
    const int row = tid >> 2, part = tid & 3;
    {
      float w[16], ahead = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int c = part * 16 + j;
        w[j] = c < row ? fmaf(sm.b[row][c], sm.qk[row][c], sm.n[row][c] * sm.kk[row][c]) : 0.f;
        ahead += w[j];
      }
      float upto = ahead;
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        const float v = __shfl_up_sync(0xffffffffu, upto, o, 4);
        if (part >= o) upto += v;
      }
      float sum = __shfl_up_sync(0xffffffffu, upto, 1, 4);
      if (part == 0) sum = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        sm.b[row][part * 16 + j] = sum;
        sum += w[j];
      }
    }
    __syncthreads();
    {   // ... then over the rows from the step on, with what these read and the steps before have written
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int a = part * 16 + j;
        sum += a >= row ? sm.b[a][row] + sm.read[a] : sm.wrote[a];
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      float all = 0.f;
#pragma unroll
      for (int w = 0; w < kGradThreads / 32; ++w) all += sm.sum[w];
      const int64_t to = (((int64_t)blockIdx.y * p.batch * p.nch + b * p.nch + chunk) * p.H + h) * kChunk + row;
      if (part == 0 && SSD_INDEX_OK(p.hdr, to, gridDim.y * p.batch * p.nch * p.H * kChunk, 2008))
        p.partial[to] = fmaf(all, sm.c.from[kChunk - 1], sum);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = ty * 4 + i;
      const int64_t c = k0 + tx * 4 + j;
      if (r < n && c < p.K) {
        const int64_t to = ((b * p.T + t0 + r) * p.Hk + hk) * p.K + c;
        if (SSD_INDEX_OK(p.hdr, to, p.batch * p.T * p.Hk * p.K, 2003)) {
          st_from_f32(static_cast<T*>(p.dq) + to, dq[i][j]);
          st_from_f32(static_cast<T*>(p.dk) + to, dk[i][j]);
        }
      }
    }
}

// dbeta of one chunk and head, a warp takes eight steps' products over V, and dg, summed over the blocks of keys.
__global__ void __launch_bounds__(256) delta_gate_grad_kernel(const __grid_constant__ Params p, int key_blocks) {
  int64_t id = blockIdx.x;
  const int64_t h = id % p.H;
  id /= p.H;
  const int64_t chunk = id % p.nch, b = id / p.nch, t0 = chunk * kChunk;
  const int n = (int)min((int64_t)kChunk, p.T - t0), lane = threadIdx.x & 31;
  for (int i = threadIdx.x >> 5; i < n; i += 8) {
    const int64_t at = ((b * p.T + t0 + i) * p.H + h) * p.V;
    float de = 0.f;
    for (int64_t c = lane; c < p.V; c += 32) de = fmaf(p.du[at + c], p.err[at + c], de);
#pragma unroll
    for (int o = 16; o; o >>= 1) de += __shfl_xor_sync(0xffffffffu, de, o);
    const int64_t to = (b * p.T + t0 + i) * p.H + h;
    if (lane == 0 && SSD_INDEX_OK(p.hdr, to, p.batch * p.T * p.H, 2009)) p.dbeta[to] = de;
  }
  if (p.dg && threadIdx.x < n) {
    const int64_t per = p.batch * p.nch * p.H * kChunk;
    const float* part = p.partial + blockIdx.x * (int64_t)kChunk + threadIdx.x;
    float sum = 0.f;
    for (int kb = 0; kb < key_blocks; ++kb) sum += part[kb * per];
    const int64_t to = (b * p.T + t0 + threadIdx.x) * p.H + h;
    if (SSD_INDEX_OK(p.hdr, to, p.batch * p.T * p.H, 2010)) p.dg[to] = sum;
  }
}

// One step of every sequence.  A row of the state is in eight lanes; a thread takes N rows.
template <typename T, int KE, int N, bool kWide>
__global__ void __launch_bounds__(128) delta_step_kernel(const __grid_constant__ Params p) {
  const int l = threadIdx.x & 7;
  int64_t id = blockIdx.x;
  const int64_t slice = id % p.slices;
  id /= p.slices;
  const int64_t h = id % p.H, b = id / p.H, hk = h / (p.H / p.Hk);
  const int64_t v0 = slice * (16 * N) + (threadIdx.x >> 3);
  const float* S = p.init ? p.init + (b * p.H + h) * p.V * p.K : nullptr;
  float* out = p.final_state + (b * p.H + h) * p.V * p.K;
  const T* qp = static_cast<const T*>(p.q) + b * p.qs[0] + hk * p.qs[2];
  const T* kp = static_cast<const T*>(p.k) + b * p.ks[0] + hk * p.ks[2];
  float s[N][KE], k[KE], q[KE], v[N];
#pragma unroll
  for (int r = 0; r < N; ++r)
#pragma unroll
    for (int e = 0; e < KE; e += 4) {
      const int c = key_of(e, l);
      const int64_t row = v0 + r * 16;
      if constexpr (kWide) {
        const float4 f = S && row < p.V && c < p.K ? *reinterpret_cast<const float4*>(S + row * p.K + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        s[r][e] = f.x;
        s[r][e + 1] = f.y;
        s[r][e + 2] = f.z;
        s[r][e + 3] = f.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[r][e + j] = S && row < p.V && c + j < p.K ? S[row * p.K + c + j] : 0.f;
      }
    }
#pragma unroll
  for (int e = 0; e < KE; e += 4) {
    const int c = key_of(e, l);
    if constexpr (kWide) {
      using K4 = Pack<T, 4>;
      float2 a[2], b[2];
      K4::unpack(c < p.K ? K4::raw(kp + c) : K4::none(), a);
      K4::unpack(c < p.K ? K4::raw(qp + c) : K4::none(), b);
      k[e] = a[0].x, k[e + 1] = a[0].y, k[e + 2] = a[1].x, k[e + 3] = a[1].y;
      q[e] = b[0].x, q[e + 1] = b[0].y, q[e + 2] = b[1].x, q[e + 3] = b[1].y;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        k[e + j] = c + j < p.K ? ld_f32(kp + c + j) : 0.f;
        q[e + j] = c + j < p.K ? ld_f32(qp + c + j) : 0.f;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < N; ++r)
    v[r] = v0 + r * 16 < p.V ? ld_f32(static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[2] + v0 + r * 16) : 0.f;
  const float a = expf(decay_log(p, b, 0, h)), beta = __ldg(p.beta + b * p.bs[0] + h);
#pragma unroll
  for (int r = 0; r < N; ++r) {
    float d0 = 0.f, d1 = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
    for (int e = 0; e < KE; e += 2) {
      d0 = fmaf(s[r][e], k[e], d0);
      d1 = fmaf(s[r][e + 1], k[e + 1], d1);
    }
    const float u = beta * fmaf(-a, sum8(d0 + d1), v[r]);
#pragma unroll
    for (int e = 0; e < KE; e += 2) {
      s[r][e] = fmaf(a, s[r][e], u * k[e]);
      s[r][e + 1] = fmaf(a, s[r][e + 1], u * k[e + 1]);
      o0 = fmaf(s[r][e], q[e], o0);
      o1 = fmaf(s[r][e + 1], q[e + 1], o1);
    }
    const float o = sum8(o0 + o1);
    const int64_t row = v0 + r * 16;
    if (row >= p.V) continue;
    if (l == 0) st_from_f32(static_cast<T*>(p.y) + (b * p.H + h) * p.V + row, o * p.scale);
#pragma unroll
    for (int e = 0; e < KE; e += 4) {
      const int c = key_of(e, l);
      if constexpr (kWide) {
        if (c < p.K) *reinterpret_cast<float4*>(out + row * p.K + c) = make_float4(s[r][e], s[r][e + 1], s[r][e + 2], s[r][e + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < p.K) out[row * p.K + c + j] = s[r][e + j];
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------ host
bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
ssd_status done(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

bool mul_fits(std::initializer_list<int64_t> v, int64_t most) {
  int64_t all = 1;
  for (int64_t x : v) {
    if (x == 0) return true;
    if (all > most / x) return false;
    all *= x;
  }
  return true;
}

ssd_status check_shape(const gated_delta_rule_shape* s, bool back) {
  if (!s || s->batch < 0 || s->seqlen < 0 || s->key_heads < 1 || s->heads < 1 || s->key_dim < 1 || s->value_dim < 1)
    return SSD_ERR_INVALID_ARG;
  if (s->heads % s->key_heads != 0 || !isfinite(s->scale)) return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_F32 && s->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  for (int a = 0; a < 3; ++a)
    if (s->q_stride[a] < 0 || s->k_stride[a] < 0 || s->v_stride[a] < 0 || (back && s->dy_stride[a] < 0)) return SSD_ERR_INVALID_ARG;
  for (int a = 0; a < 2; ++a)
    if (s->g_stride[a] < 0 || s->beta_stride[a] < 0) return SSD_ERR_INVALID_ARG;
  if (s->key_dim > 256) return SSD_ERR_UNSUPPORTED;
  const int64_t b = std::max<int64_t>(s->batch, 1), most = INT64_MAX / 64;
  const int64_t nch = s->seqlen / kChunk + 1, slices = s->value_dim / 16 + 1;
  // grids of blocks and sizes of arrays
  if (!mul_fits({b, s->heads, nch, slices}, INT32_MAX) || !mul_fits({b, nch, s->heads, s->value_dim, s->key_dim + kChunk}, most))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

struct Layout {
  size_t err, du, states, dstates, partial, chunks, total;
};
// Whether strides and pointers may let the tensor-core kernels take a call of this shape.
bool tc_shape(const gated_delta_rule_shape* s) {
  return s->io_dtype == SSD_BF16 && s->key_dim % 8 == 0 && s->key_dim <= 128 && s->value_dim % 8 == 0;
}
int key_blocks(int64_t K) { return (int)((K + 63) / 64); }
// A call takes the tensor cores or the walk on the CUDA cores: what only one of them uses lies in the same place.
Layout layout(const gated_delta_rule_shape* s, bool back) {
  Layout L = {};
  size_t at = sizeof(WsHeader);
  const size_t nch = (size_t)((s->seqlen + kChunk - 1) / kChunk);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = align_up(at + bytes, kWsAlign);
    return here;
  };
  if (back) {
    const size_t states = (size_t)s->batch * nch * (size_t)(s->heads * s->value_dim * s->key_dim) * 4;
    L.states = take(states);
    L.dstates = take(states);
  }
  const size_t shared = at;
  if (tc_shape(s)) L.chunks = take(tc_bytes(s->batch, (int64_t)nch, s->heads, s->value_dim, s->key_dim, back));
  L.total = at;
  if (back) {
    at = shared;
    const size_t steps = (size_t)(s->batch * s->seqlen * s->heads * s->value_dim) * 4;
    L.err = take(steps);
    L.du = take(steps);
    L.partial = take((size_t)key_blocks(s->key_dim) * (size_t)s->batch * nch * (size_t)s->heads * kChunk * 4);
    L.total = std::max(L.total, at);
  }
  return L;
}

Params make_params(const gated_delta_rule_shape* s) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.batch = s->batch;
  p.T = s->seqlen;
  p.Hk = s->key_heads;
  p.H = s->heads;
  p.K = s->key_dim;
  p.V = s->value_dim;
  p.nch = (s->seqlen + kChunk - 1) / kChunk;
  for (int a = 0; a < 3; ++a) {
    p.qs[a] = s->q_stride[a];
    p.ks[a] = s->k_stride[a];
    p.vs[a] = s->v_stride[a];
    p.ds[a] = s->dy_stride[a];
  }
  for (int a = 0; a < 2; ++a) {
    p.gs[a] = s->g_stride[a];
    p.bs[a] = s->beta_stride[a];
  }
  p.scale = s->scale;
  return p;
}

// Blocks of 16 rows while these fit the SMs in a round or so (a step is then shorter: 3 x 777 x 6 heads of 60 x 100 f32
// 128 us, with 32 rows 159), else of 32 (a step's loads of k and q serve twice as many).
constexpr int64_t kFewBlocks = 2 * 152;

template <typename T, int KE>
cudaError_t launch_walk_as(Params p, bool by_chunk, cudaStream_t st) {
  const int64_t walks = p.batch * (by_chunk ? p.nch : 1) * p.H;
  p.slices = (p.V + 15) / 16;
  if (walks * p.slices <= kFewBlocks) {
    delta_walk_kernel<T, KE, 1><<<(unsigned)(walks * p.slices), kThreads, 0, st>>>(p, by_chunk);
  } else {
    p.slices = (p.V + 31) / 32;
    delta_walk_kernel<T, KE, 2><<<(unsigned)(walks * p.slices), kThreads, 0, st>>>(p, by_chunk);
  }
  return cudaGetLastError();
}
template <typename T, int KE>
cudaError_t launch_walk_back_as(Params p, cudaStream_t st) {
  const int64_t walks = p.batch * p.H;
  p.slices = (p.V + 15) / 16;
  if (walks * p.slices <= kFewBlocks) {
    delta_walk_back_kernel<T, KE, 1><<<(unsigned)(walks * p.slices), kThreads, 0, st>>>(p);
  } else {
    p.slices = (p.V + 31) / 32;
    delta_walk_back_kernel<T, KE, 2><<<(unsigned)(walks * p.slices), kThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

// Keys a lane holds: 8, 16 or 32 of up to 64, 128 or 256.
template <typename T>
cudaError_t launch_walk(const Params& p, bool by_chunk, cudaStream_t st) {
  if (p.K <= 64) return launch_walk_as<T, 8>(p, by_chunk, st);
  if (p.K <= 128) return launch_walk_as<T, 16>(p, by_chunk, st);
  return launch_walk_as<T, 32>(p, by_chunk, st);
}

template <typename T>
cudaError_t launch_backward(const Params& p, cudaStream_t st) {
  cudaError_t e = p.K <= 64    ? launch_walk_back_as<T, 8>(p, st)
                  : p.K <= 128 ? launch_walk_back_as<T, 16>(p, st)
                               : launch_walk_back_as<T, 32>(p, st);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(delta_chunk_grad_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(GradSmem));
  if (e != cudaSuccess) return e;
  const dim3 cells((unsigned)(p.batch * p.nch * p.Hk), (unsigned)key_blocks(p.K));
  delta_chunk_grad_kernel<T><<<cells, kGradThreads, sizeof(GradSmem), st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  delta_gate_grad_kernel<<<(unsigned)(p.batch * p.nch * p.H), 256, 0, st>>>(p, key_blocks(p.K));
  return cudaGetLastError();
}

template <typename T, int KE, int N>
cudaError_t launch_step_as(Params p, bool wide, cudaStream_t st) {
  p.slices = (p.V + 16 * N - 1) / (16 * N);
  const unsigned grid = (unsigned)(p.batch * p.H * p.slices);
  if (wide) delta_step_kernel<T, KE, N, true><<<grid, 128, 0, st>>>(p);
  else delta_step_kernel<T, KE, N, false><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_step(const Params& p, cudaStream_t st) {
  const uint64_t keys = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                        (uint64_t)(p.qs[0] | p.qs[2] | p.ks[0] | p.ks[2]) * sizeof(T);
  const bool wide = p.K % 4 == 0 && !misaligned(p.init, 16) && !misaligned(p.final_state, 16) && keys % (4 * sizeof(T)) == 0;
  if (p.K <= 64) return launch_step_as<T, 8, 2>(p, wide, st);
  if (p.K <= 128) return launch_step_as<T, 16, 2>(p, wide, st);
  return launch_step_as<T, 32, 1>(p, wide, st);
}

cudaError_t set_rows(float* dst, const float* src, int64_t n, cudaStream_t st) {
  if (!dst || n == 0) return cudaSuccess;
  return src ? cudaMemcpyAsync(dst, src, sizeof(float) * (size_t)n, cudaMemcpyDeviceToDevice, st)
             : cudaMemsetAsync(dst, 0, sizeof(float) * (size_t)n, st);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

namespace ssd {
namespace {
bool overlap(const float* a, int64_t n, const float* b, int64_t m) {   // counts of values
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + 4 * (uintptr_t)m && y < x + 4 * (uintptr_t)n;
}
}  // namespace
}  // namespace ssd

extern "C" {

size_t gated_delta_rule_workspace_bytes(const gated_delta_rule_shape* shape, int32_t backward) {
  if (check_shape(shape, false) != SSD_OK) return 0;
  return layout(shape, backward != 0).total;
}

ssd_status gated_delta_rule_forward(const gated_delta_rule_shape* shape, const void* q, const void* k, const void* v,
                                    const float* g, const float* beta, const float* init_state, void* y,
                                    float* final_state, float* states, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  const ssd_status bad = check_shape(shape, false);
  if (bad != SSD_OK) return bad;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  const bool empty = shape->batch == 0 || shape->seqlen == 0;
  if (!empty && (!q || !k || !v || !beta)) return SSD_ERR_INVALID_ARG;
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(y, e) || misaligned(g, 4) ||
      misaligned(beta, 4) || misaligned(init_state, 4) || misaligned(final_state, 4) || misaligned(states, 4))
    return SSD_ERR_INVALID_ARG;
  const Layout L = layout(shape, false);
  if (!workspace || misaligned(workspace, kWsAlign) || workspace_bytes < L.total) return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Params p = make_params(shape);
  // A sequence in segments: the last one's block may have written final_state before the first one's reads init_state.
  const int64_t state = p.batch * p.H * p.K * p.V;
  if (overlap(init_state, state, final_state, state) || overlap(init_state, state, states, state * p.nch))
    return SSD_ERR_INVALID_ARG;
  if (empty) return done(set_rows(final_state, init_state, p.batch * p.H * p.K * p.V, st));
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.beta = beta;
  p.init = init_state;
  p.y = y;
  p.final_state = final_state;
  p.states_out = states;
  p.hdr = static_cast<WsHeader*>(workspace);
  if (tc_shape(shape) && tc_takes(p, false)) return done(tc_forward(p, static_cast<char*>(workspace) + L.chunks, st));
  return done(bf16 ? launch_walk<__nv_bfloat16>(p, false, st) : launch_walk<float>(p, false, st));
}

ssd_status gated_delta_rule_backward(const gated_delta_rule_shape* shape, const void* q, const void* k, const void* v,
                                     const float* g, const float* beta, const float* init_state, const float* states,
                                     const void* dy, const float* dfinal, void* dq, void* dk, void* dv, float* dg,
                                     float* dbeta, float* dinit, void* workspace, size_t workspace_bytes, void* stream) {
  const ssd_status bad = check_shape(shape, true);
  if (bad != SSD_OK) return bad;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  const bool empty = shape->batch == 0 || shape->seqlen == 0;
  if (!empty && (!q || !k || !v || !beta || !dy || !dq || !dk || !dv || !dbeta)) return SSD_ERR_INVALID_ARG;
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(dy, e) || misaligned(dq, e) ||
      misaligned(dk, e) || misaligned(dv, e) || misaligned(g, 4) || misaligned(beta, 4) || misaligned(init_state, 4) ||
      misaligned(states, 4) || misaligned(dfinal, 4) || misaligned(dg, 4) || misaligned(dbeta, 4) || misaligned(dinit, 4))
    return SSD_ERR_INVALID_ARG;
  const Layout L = layout(shape, true);
  if (!workspace || misaligned(workspace, kWsAlign) || workspace_bytes < L.total) return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Params p = make_params(shape);
  if (empty) return done(set_rows(dinit, dfinal, p.batch * p.H * p.K * p.V, st));
  char* ws = static_cast<char*>(workspace);
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.beta = beta;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.err = reinterpret_cast<float*>(ws + L.err);
  p.states_in = states ? states : reinterpret_cast<float*>(ws + L.states);
  p.dy = dy;
  p.dfinal = dfinal;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  p.dg = dg;
  p.dbeta = dbeta;
  p.dinit = dinit;
  p.du = reinterpret_cast<float*>(ws + L.du);
  p.dstates = reinterpret_cast<float*>(ws + L.dstates);
  p.partial = reinterpret_cast<float*>(ws + L.partial);
  if (!states) p.init = init_state;
  if (tc_shape(shape) && tc_takes(p, true)) return done(tc_backward(p, states != nullptr, ws + L.chunks, st));
  Params f = p;   // v - S k of every step, from the states before the chunks
  f.y = nullptr;
  f.states_out = states ? nullptr : const_cast<float*>(p.states_in);
  const cudaError_t ce = bf16 ? launch_walk<__nv_bfloat16>(f, states != nullptr, st) : launch_walk<float>(f, states != nullptr, st);
  if (ce != cudaSuccess) return SSD_ERR_CUDA;
  return done(bf16 ? launch_backward<__nv_bfloat16>(p, st) : launch_backward<float>(p, st));
}

ssd_status gated_delta_rule_step(const gated_delta_rule_shape* shape, const void* q, const void* k, const void* v,
                                 const float* g, const float* beta, const float* state, void* y, float* state_out,
                                 void* stream) {
  if (!shape) return SSD_ERR_INVALID_ARG;
  gated_delta_rule_shape one = *shape;   // the step strides are ignored
  one.q_stride[1] = one.k_stride[1] = one.v_stride[1] = one.g_stride[1] = one.beta_stride[1] = 0;
  const ssd_status bad = check_shape(&one, false);
  if (bad != SSD_OK) return bad;
  if (shape->seqlen != 1) return SSD_ERR_INVALID_ARG;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  if (shape->batch == 0) return SSD_OK;
  if (!q || !k || !v || !beta || !y || !state_out) return SSD_ERR_INVALID_ARG;
  if (misaligned(q, e) || misaligned(k, e) || misaligned(v, e) || misaligned(y, e) || misaligned(g, 4) ||
      misaligned(beta, 4) || misaligned(state, 4) || misaligned(state_out, 4))
    return SSD_ERR_INVALID_ARG;
  Params p = make_params(&one);
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.beta = beta;
  p.init = state;
  p.y = y;
  p.final_state = state_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return done(bf16 ? launch_step<__nv_bfloat16>(p, st) : launch_step<float>(p, st));
}

}  // extern "C"
