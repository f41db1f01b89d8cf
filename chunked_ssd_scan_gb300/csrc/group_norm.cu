// Group norm with an activation, channels last (declarations in include/ssdscan.h):
//   xhat = (x - mean) rstd, z = xhat w + b, y = act(z), statistics over the S * C/G values of a
//   sample's group; reverse mode, dz = dy act'(z), q = dz w:
//   dx = rstd (q - mean(q) - xhat mean(q xhat)), dw = sum dz xhat, db = sum dz.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>

#include "common.cuh"
#include "fp_helpers.cuh"

namespace ssd {
namespace {

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
  float *stats;         // map kernels: [N, chunks, G, 2], mean and M2 or the two gradient sums
  float *part_w, *part_b;   // rows of parameter gradient partials [part_rows, C]
  int64_t part_rows;
  WsHeader* hdr;
};

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + e^-z)
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + fp::ex2_approx(-z * kLog2e)); }
template <bool kSilu>
__device__ __forceinline__ float act_fwd(float z) {
  return kSilu ? z * sigmoid(z) : z;
}
// act'(z)
template <bool kSilu>
__device__ __forceinline__ float act_grad(float z) {
  if (!kSilu) return 1.f;
  const float s = sigmoid(z);
  return s * fmaf(z, 1.f - s, 1.f);
}

// V neighbouring values as one load or store of up to 16 bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
  const Vec<T, V> q = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] = (float)q.v[k];
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
  Vec<T, V> q;
#pragma unroll
  for (int k = 0; k < V; ++k) st_from_f32(&q.v[k], f[k]);
  *reinterpret_cast<Vec<T, V>*>(p) = q;
}
template <int V>
__device__ __forceinline__ void load_param(const float* p, int64_t at, float none, float (&f)[V]) {
#pragma unroll
  for (int k = 0; k < V; ++k) f[k] = p ? __ldg(p + at + k) : none;
}

// ------------------------------------------------------------------------------------------------
// One position a sample (the norm of every token): a group's values stay in the registers of `lanes`
// neighbouring lanes (or of a whole block), K vectors of V values each; the mean and then the
// squares around it are summed over them by shuffles.  A thread keeps its channels for all the
// samples that its block takes, so weight and bias are read once, and has U samples in flight.
// Bound by memory: x and y once each.
// ------------------------------------------------------------------------------------------------
template <bool kBlock>
__device__ __forceinline__ float group_sum(float v, int lanes, float (&part)[2][kWarps], int& phase) {
  if (!kBlock) {
    for (int o = lanes / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) part[phase][threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) s += part[phase][k];
  phase ^= 1;   // the next sum writes elsewhere, and its barrier ends the reads of this one
  return s;
}

// What a thread of a token kernel works on.
template <int V, int K, bool kBlock>
struct TokenSlot {
  int64_t g, row, rows;   // its group, its first sample within a block's step, samples of a step
  int64_t c;              // its first channel
  bool in[K];             // which of its vectors lie inside the group
  int step;               // channels from one of its vectors to the next
  __device__ __forceinline__ TokenSlot(const NormParams& p) {
    int l;
    if (kBlock) {
      g = blockIdx.y;
      l = threadIdx.x;
      row = 0;
      rows = 1;
      step = kThreads * V;
    } else {
      const int64_t slots = p.G * p.lanes;
      int64_t s;
      if (slots >= kThreads) {
        s = (int64_t)blockIdx.y * kThreads + threadIdx.x;
        row = 0;
        rows = 1;
      } else {
        rows = kThreads / (int)slots;
        row = threadIdx.x / (int)slots;
        s = threadIdx.x % (int)slots;
        if (row >= rows) s = slots;   // a thread too many
      }
      g = s / p.lanes;
      l = (int)(s % p.lanes);
      step = p.lanes * V;
    }
    c = g * p.cg + (int64_t)l * V;
#pragma unroll
    for (int k = 0; k < K; ++k) in[k] = g < p.G && (int64_t)l * V + (int64_t)k * step < p.cg;
  }
};

template <typename T, int V, int K, int U, bool kBlock, bool kSilu>
__global__ void __launch_bounds__(kThreads) norm_token_forward_kernel(NormParams p) {
  __shared__ float part[2][kWarps];
  int phase = 0;
  const TokenSlot<V, K, kBlock> t(p);
  const int lanes = p.lanes;
  float w[K][V], bias[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (t.in[k]) {
      load_param<V>(p.w, t.c + k * t.step, 1.f, w[k]);
      load_param<V>(p.bias, t.c + k * t.step, 0.f, bias[k]);
    }
  }
  const float inv = 1.f / (float)p.cg;
  const int64_t stride = (int64_t)gridDim.x * t.rows * U;
  for (int64_t n0 = (int64_t)blockIdx.x * t.rows * U; n0 < p.N; n0 += stride) {
    float x[U][K][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u * t.rows + t.row;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (t.in[k] && n < p.N) {
          load_vec<T, V>(static_cast<const T*>(p.x) + n * p.xs[0] + t.c + k * t.step, x[u][k]);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) x[u][k][e] = 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u * t.rows + t.row;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) s += x[u][k][e];
      const float mean = group_sum<kBlock>(s, lanes, part, phase) * inv;
      s = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t.in[k]) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            x[u][k][e] -= mean;
            s = fmaf(x[u][k][e], x[u][k][e], s);
          }
        }
      const float rstd = 1.f / sqrtf(group_sum<kBlock>(s, lanes, part, phase) * inv + p.eps);
      if (n >= p.N) continue;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int64_t at = n * p.C + t.c + k * t.step;
        if (!t.in[k] || !SSD_INDEX_OK(p.hdr, at + V - 1, p.N * p.C, 70)) continue;
#pragma unroll
        for (int e = 0; e < V; ++e)
          x[u][k][e] = act_fwd<kSilu>(fmaf(x[u][k][e] * rstd, w[k][e], bias[k][e]));
        store_vec<T, V>(static_cast<T*>(p.y) + at, x[u][k]);
      }
      if (p.mean && t.in[0] && t.c == t.g * p.cg && SSD_INDEX_OK(p.hdr, n * p.G + t.g, p.N * p.G, 71)) {
        p.mean[n * p.G + t.g] = mean;
        p.rstd[n * p.G + t.g] = rstd;
      }
    }
  }
}

template <typename T, int V, int K, int U, bool kBlock, bool kSilu>
__global__ void __launch_bounds__(kThreads) norm_token_backward_kernel(NormParams p) {
  __shared__ float part[2][kWarps];
  int phase = 0;
  const TokenSlot<V, K, kBlock> t(p);
  const int lanes = p.lanes;
  float w[K][V], bias[K][V], dw[K][V], db[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (t.in[k]) {
      load_param<V>(p.w, t.c + k * t.step, 1.f, w[k]);
      load_param<V>(p.bias, t.c + k * t.step, 0.f, bias[k]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) dw[k][e] = db[k][e] = 0.f;
  }
  const float inv = 1.f / (float)p.cg;
  const int64_t stride = (int64_t)gridDim.x * t.rows * U;
  for (int64_t n0 = (int64_t)blockIdx.x * t.rows * U; n0 < p.N; n0 += stride) {
    float x[U][K][V], q[U][K][V], rstd[U], mean[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u * t.rows + t.row;
      const bool live = t.g < p.G && n < p.N;
      mean[u] = live ? __ldg(p.mean_in + n * p.G + t.g) : 0.f;
      rstd[u] = live ? __ldg(p.rstd_in + n * p.G + t.g) : 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (t.in[k] && n < p.N) {
          load_vec<T, V>(static_cast<const T*>(p.x) + n * p.xs[0] + t.c + k * t.step, x[u][k]);
          load_vec<T, V>(static_cast<const T*>(p.dy) + n * p.ds[0] + t.c + k * t.step, q[u][k]);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) x[u][k][e] = q[u][k][e] = 0.f;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u * t.rows + t.row;
      float s = 0.f, sx = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t.in[k]) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float xh = (x[u][k][e] - mean[u]) * rstd[u];
            const float dz = q[u][k][e] * act_grad<kSilu>(fmaf(xh, w[k][e], bias[k][e]));
            db[k][e] += dz;
            dw[k][e] = fmaf(dz, xh, dw[k][e]);
            x[u][k][e] = xh;
            q[u][k][e] = dz * w[k][e];
            s += q[u][k][e];
            sx = fmaf(q[u][k][e], xh, sx);
          }
        }
      s = group_sum<kBlock>(s, lanes, part, phase) * inv;
      sx = group_sum<kBlock>(sx, lanes, part, phase) * inv;
      if (n >= p.N) continue;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int64_t at = n * p.C + t.c + k * t.step;
        if (!t.in[k] || !SSD_INDEX_OK(p.hdr, at + V - 1, p.N * p.C, 72)) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) x[u][k][e] = rstd[u] * (q[u][k][e] - s - x[u][k][e] * sx);
        store_vec<T, V>(static_cast<T*>(p.dx) + at, x[u][k]);
      }
    }
  }
  if (p.part_rows == 0) return;
  __shared__ float2 rows[kThreads][V];   // the block's rows of samples joined, one partial a block
  const int slots = (int)min((int64_t)kThreads, p.G * p.lanes);   // threads of one row
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (!kBlock && t.rows > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < V; ++e) rows[threadIdx.x][e] = make_float2(dw[k][e], db[k][e]);
      __syncthreads();
      if (t.row > 0) continue;
      for (int r = 1; r < t.rows; ++r) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 v = rows[threadIdx.x + r * slots][e];
          dw[k][e] += v.x;
          db[k][e] += v.y;
        }
      }
    }
    const int64_t at = (int64_t)blockIdx.x * p.C + t.c + k * t.step;
    if (!t.in[k] || !SSD_INDEX_OK(p.hdr, at + V - 1, p.part_rows * p.C, 73)) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      p.part_w[at + e] = dw[k][e];
      p.part_b[at + e] = db[k][e];
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Many positions a sample: a sample's positions are cut into chunks, a block takes one chunk of one
// sample by one column tile of whole groups.  Two passes over x: the chunks' statistics, then
// their join and the output; the second pass goes through the samples backwards, so that what the
// first read last is still in L2.
// ------------------------------------------------------------------------------------------------
// count, mean and sum of squares around the mean; joined pairwise (Chan, Golub and LeVeque), so no
// difference of large squares is formed
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments join(const Moments& a, const Moments& b) {
  const float n = a.n + b.n;
  if (b.n == 0.f) return a;
  const float f = b.n / n, d = b.mean - a.mean;
  return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}
__device__ __forceinline__ Moments join_lanes(Moments m) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const Moments b = {__shfl_down_sync(0xffffffffu, m.n, o), __shfl_down_sync(0xffffffffu, m.mean, o),
                       __shfl_down_sync(0xffffffffu, m.m2, o)};
    m = join(m, b);
  }
  return m;   // in lane 0
}

// What a thread of a map kernel works on: vector `col` (and every kThreads-th after it, for a group
// wider than the block) of its tile, positions row, row + rows, ... of its chunk.
template <int V>
struct MapSlot {
  int64_t n, chunk, g0, groups, s0, s1;   // sample, chunk, groups of the tile, positions [s0, s1)
  int vecs, cols, rows, row, col;         // vectors of the tile, thread columns and rows
  __device__ __forceinline__ MapSlot(const NormParams& p, int64_t block) {
    const int64_t tiles = (p.G + p.tile_groups - 1) / p.tile_groups;
    const int64_t tile = block % tiles;
    chunk = block / tiles % p.chunks;
    n = block / tiles / p.chunks;
    g0 = tile * p.tile_groups;
    groups = min((int64_t)p.tile_groups, p.G - g0);
    vecs = (int)(groups * (p.cg / V));
    cols = min(vecs, kThreads);
    rows = kThreads / cols;
    row = threadIdx.x / cols;
    col = threadIdx.x % cols;
    s0 = chunk * p.chunk_rows;
    s1 = min(p.S, s0 + p.chunk_rows);
  }
  __device__ __forceinline__ int64_t channel(const NormParams& p, int v) const { return g0 * p.cg + (int64_t)v * V; }
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) norm_map_stats_kernel(NormParams p) {
  constexpr int U = 8;   // positions in flight: their moments are formed directly, around their mean
  __shared__ Moments all[kThreads];
  const MapSlot<V> t(p, blockIdx.x);
  Moments m = {0.f, 0.f, 0.f};
  if (t.row < t.rows)
    for (int v = t.col; v < t.vecs; v += kThreads) {
      const T* x = static_cast<const T*>(p.x) + t.n * p.xs[0] + t.channel(p, v);
      for (int64_t s = t.s0 + t.row; s < t.s1; s += U * t.rows) {
        float f[U][V], sum = 0.f, sq = 0.f;
        int have = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool in = s + u * t.rows < t.s1;
          if (in) load_vec<T, V>(x + (s + u * t.rows) * p.xs[1], f[u]);
          have += in;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < have) {
#pragma unroll
            for (int e = 0; e < V; ++e) sum += f[u][e];
          }
        const float n = (float)(have * V), mean = sum / n;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (u < have) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float d = f[u][e] - mean;
              sq = fmaf(d, d, sq);
            }
          }
        m = m.n == 0.f ? Moments{n, mean, sq} : join(m, {n, mean, sq});
      }
    }
  all[threadIdx.x] = m;
  __syncthreads();
  // a warp a group: its threads are columns [k per, (k + 1) per) of every row
  const int lane = threadIdx.x % 32, per = (int)(p.cg / V) < t.cols ? (int)(p.cg / V) : t.cols;
  for (int k = threadIdx.x / 32; k < t.groups; k += kWarps) {
    Moments g = {0.f, 0.f, 0.f};
    for (int j = lane; j < per * t.rows; j += 32) {
      const Moments b = all[j / per * t.cols + k * per + j % per];
      if (b.n > 0.f) g = g.n == 0.f ? b : join(g, b);
    }
    // lanes without values hand theirs over unchanged
    g = join_lanes(g);
    const int64_t at = ((t.n * p.chunks + t.chunk) * p.G + t.g0 + k) * 2;
    if (lane == 0 && SSD_INDEX_OK(p.hdr, at + 1, p.N * p.chunks * p.G * 2, 74)) {
      p.stats[at] = g.mean;
      p.stats[at + 1] = g.m2;
    }
  }
}

template <typename T, int V, bool kSilu>
__global__ void __launch_bounds__(kThreads) norm_map_apply_kernel(NormParams p) {
  constexpr int U = 8;
  __shared__ float2 fin[kThreads];   // mean and rstd of the tile's groups (at most kThreads of them)
  const MapSlot<V> t(p, (int64_t)gridDim.x - 1 - blockIdx.x);
  const int lane = threadIdx.x % 32;
  for (int k = threadIdx.x / 32; k < t.groups; k += kWarps) {
    Moments m = {0.f, 0.f, 0.f};
    for (int c = lane; c < p.chunks; c += 32) {
      const float* s = p.stats + ((t.n * p.chunks + c) * p.G + t.g0 + k) * 2;
      const float n = (float)(min(p.S, (c + 1) * p.chunk_rows) - c * p.chunk_rows) * (float)p.cg;
      const Moments b = {n, __ldcg(s), __ldcg(s + 1)};
      m = m.n == 0.f ? b : join(m, b);
    }
    m = join_lanes(m);
    if (lane == 0) {
      const float rstd = 1.f / sqrtf(m.m2 / m.n + p.eps);
      fin[k] = make_float2(m.mean, rstd);
      const int64_t at = t.n * p.G + t.g0 + k;
      if (p.mean && t.chunk == 0 && SSD_INDEX_OK(p.hdr, at, p.N * p.G, 75)) {
        p.mean[at] = m.mean;
        p.rstd[at] = rstd;
      }
    }
  }
  __syncthreads();
  if (t.row >= t.rows) return;
  for (int v = t.col; v < t.vecs; v += kThreads) {
    const int64_t c = t.channel(p, v);
    const float2 st = fin[v / (int)(p.cg / V)];
    float a[V], b[V];   // z = x a + b would round around a large mean: (x - mean) a + bias instead
    load_param<V>(p.w, c, 1.f, a);
    load_param<V>(p.bias, c, 0.f, b);
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] *= st.y;
    const T* x = static_cast<const T*>(p.x) + t.n * p.xs[0] + c;
    T* y = static_cast<T*>(p.y) + t.n * p.S * p.C + c;
    for (int64_t s = t.s0 + t.row; s < t.s1; s += U * t.rows) {
      float f[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u * t.rows < t.s1) load_vec<T, V>(x + (s + u * t.rows) * p.xs[1], f[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = s + u * t.rows;
        if (r >= t.s1 || !SSD_INDEX_OK(p.hdr, (t.n * p.S + r) * p.C + c + V - 1, p.N * p.S * p.C, 76)) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) f[u][e] = act_fwd<kSilu>(fmaf(f[u][e] - st.x, a[e], b[e]));
        store_vec<T, V>(y + r * p.C, f[u]);
      }
    }
  }
}

// Per chunk and channel, sum dz and sum dz xhat (which are the parameters' gradients' partials), and per
// group their sums times w, which the gradient of x needs.
template <typename T, int V, bool kSilu>
__global__ void __launch_bounds__(kThreads) norm_map_grad_sums_kernel(NormParams p) {
  constexpr int U = 4;
  __shared__ float2 all[kThreads][V];
  const MapSlot<V> t(p, blockIdx.x);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int gv = (int)(p.cg / V);
  float2 wide = make_float2(0.f, 0.f);   // a group wider than the block: this thread's share of its sums
  for (int v0 = 0; v0 < t.vecs; v0 += kThreads) {
    const int v = v0 + t.col;
    float dw[V], db[V], w[V];
#pragma unroll
    for (int e = 0; e < V; ++e) dw[e] = db[e] = w[e] = 0.f;
    if (t.row < t.rows && v < t.vecs) {
      const int64_t c = t.channel(p, v), at = t.n * p.G + t.g0 + v / gv;
      const float mean = __ldg(p.mean_in + at), rstd = __ldg(p.rstd_in + at);
      float bias[V];
      load_param<V>(p.w, c, 1.f, w);
      load_param<V>(p.bias, c, 0.f, bias);
      const T* x = static_cast<const T*>(p.x) + t.n * p.xs[0] + c;
      const T* dy = static_cast<const T*>(p.dy) + t.n * p.ds[0] + c;
      for (int64_t s = t.s0 + t.row; s < t.s1; s += U * t.rows) {
        float f[U][V], d[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (s + u * t.rows < t.s1) {
            load_vec<T, V>(x + (s + u * t.rows) * p.xs[1], f[u]);
            load_vec<T, V>(dy + (s + u * t.rows) * p.ds[1], d[u]);
          }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (s + u * t.rows < t.s1) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const float xh = (f[u][e] - mean) * rstd;
              const float dz = d[u][e] * act_grad<kSilu>(fmaf(xh, w[e], bias[e]));
              db[e] += dz;
              dw[e] = fmaf(dz, xh, dw[e]);
            }
          }
      }
    }
    // over the block's rows, per channel
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) all[threadIdx.x][e] = make_float2(db[e], dw[e]);
    __syncthreads();
    if (t.row == 0 && v < t.vecs) {
      float2 q = make_float2(0.f, 0.f);
      const int64_t at = (t.n * p.chunks + t.chunk) * p.C + t.channel(p, v);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float2 s = all[t.col][e];
        for (int r = 1; r < t.rows; ++r) {
          s.x += all[r * t.cols + t.col][e].x;
          s.y += all[r * t.cols + t.col][e].y;
        }
        if (p.part_rows > 0 && SSD_INDEX_OK(p.hdr, at + e, p.part_rows * p.C, 77)) {
          p.part_b[at + e] = s.x;
          p.part_w[at + e] = s.y;
        }
        q.x = fmaf(s.x, w[e], q.x);
        q.y = fmaf(s.y, w[e], q.y);
      }
      wide.x += q.x;
      wide.y += q.y;
    }
  }
  __syncthreads();
  all[threadIdx.x][0] = wide;   // (the threads of the first row hold the sums)
  __syncthreads();
  const int per = gv < t.cols ? gv : t.cols;
  for (int k = warp; k < t.groups; k += kWarps) {
    float2 s = make_float2(0.f, 0.f);
    for (int j = lane; j < per; j += 32) {
      s.x += all[k * per + j][0].x;
      s.y += all[k * per + j][0].y;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
      s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
    }
    const int64_t at = ((t.n * p.chunks + t.chunk) * p.G + t.g0 + k) * 2;
    if (lane == 0 && SSD_INDEX_OK(p.hdr, at + 1, p.N * p.chunks * p.G * 2, 78)) {
      p.stats[at] = s.x;
      p.stats[at + 1] = s.y;
    }
  }
}

template <typename T, int V, bool kSilu>
__global__ void __launch_bounds__(kThreads) norm_map_grad_apply_kernel(NormParams p) {
  constexpr int U = 4;
  __shared__ float2 fin[kThreads];   // mean q and mean q xhat of the tile's groups
  const MapSlot<V> t(p, (int64_t)gridDim.x - 1 - blockIdx.x);
  const int lane = threadIdx.x % 32, gv = (int)(p.cg / V);
  const float inv = 1.f / ((float)p.S * (float)p.cg);
  for (int k = threadIdx.x / 32; k < t.groups; k += kWarps) {
    float2 m = make_float2(0.f, 0.f);
    for (int c = lane; c < p.chunks; c += 32) {
      const float* s = p.stats + ((t.n * p.chunks + c) * p.G + t.g0 + k) * 2;
      m.x += __ldcg(s);
      m.y += __ldcg(s + 1);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      m.x += __shfl_xor_sync(0xffffffffu, m.x, o);
      m.y += __shfl_xor_sync(0xffffffffu, m.y, o);
    }
    if (lane == 0) fin[k] = make_float2(m.x * inv, m.y * inv);
  }
  __syncthreads();
  if (t.row >= t.rows) return;
  for (int v = t.col; v < t.vecs; v += kThreads) {
    const int64_t c = t.channel(p, v), at = t.n * p.G + t.g0 + v / gv;
    const float mean = __ldg(p.mean_in + at), rstd = __ldg(p.rstd_in + at);
    const float2 m = fin[v / gv];
    float w[V], bias[V];
    load_param<V>(p.w, c, 1.f, w);
    load_param<V>(p.bias, c, 0.f, bias);
    const T* x = static_cast<const T*>(p.x) + t.n * p.xs[0] + c;
    const T* dy = static_cast<const T*>(p.dy) + t.n * p.ds[0] + c;
    T* dx = static_cast<T*>(p.dx) + t.n * p.S * p.C + c;
    for (int64_t s = t.s0 + t.row; s < t.s1; s += U * t.rows) {
      float f[U][V], d[U][V];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s + u * t.rows < t.s1) {
          load_vec<T, V>(x + (s + u * t.rows) * p.xs[1], f[u]);
          load_vec<T, V>(dy + (s + u * t.rows) * p.ds[1], d[u]);
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t r = s + u * t.rows;
        if (r >= t.s1 || !SSD_INDEX_OK(p.hdr, (t.n * p.S + r) * p.C + c + V - 1, p.N * p.S * p.C, 79)) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (f[u][e] - mean) * rstd;
          const float q = d[u][e] * act_grad<kSilu>(fmaf(xh, w[e], bias[e])) * w[e];
          f[u][e] = rstd * (q - m.x - xh * m.y);
        }
        store_vec<T, V>(dx + r * p.C, f[u]);
      }
    }
  }
}

// dweight and dbias: a block takes 32 channels and its share of the partial rows (blockIdx.y of
// gridDim.y), its warps every 32nd row each, joined in warp order into row blockIdx.y.
__global__ void __launch_bounds__(1024) norm_param_grad_kernel(NormParams p) {
  __shared__ float2 part[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  const int64_t share = (p.part_rows + gridDim.y - 1) / gridDim.y, r0 = blockIdx.y * share;
  const int64_t r1 = min(p.part_rows, r0 + share);
  float2 s = make_float2(0.f, 0.f);
  if (c < p.C) {
#pragma unroll 8
    for (int64_t r = r0 + warp; r < r1; r += 32) {
      s.x += p.part_w[r * p.C + c];
      s.y += p.part_b[r * p.C + c];
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < p.C) {
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      v.x += part[k][lane].x;
      v.y += part[k][lane].y;
    }
    if (p.dw) p.dw[blockIdx.y * p.C + c] = v.x;
    if (p.db) p.db[blockIdx.y * p.C + c] = v.y;
  }
}

constexpr int64_t kMaxElems = (int64_t)1 << 40;

ssd_status check_shape(const group_norm_shape* s, bool backward) {
  if (!s || s->batch < 0 || s->rows < 0 || s->channels < 1 || s->groups < 1 ||
      s->channels % s->groups != 0)
    return SSD_ERR_INVALID_ARG;
  if (s->io_dtype != SSD_F32 && s->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (s->activation != SSD_ACT_NONE && s->activation != SSD_ACT_SILU) return SSD_ERR_INVALID_ARG;
  if (!(s->eps >= 0.f) || !isfinite(s->eps)) return SSD_ERR_INVALID_ARG;
  for (int k = 0; k < 2; ++k)
    if (s->x_stride[k] < 0 || (backward && s->dy_stride[k] < 0)) return SSD_ERR_INVALID_ARG;
  if (s->channels > 0x7fffffffLL || s->rows > kMaxElems / s->channels ||
      (s->rows > 0 && s->batch > kMaxElems / s->channels / s->rows))
    return SSD_ERR_UNSUPPORTED;
  if (s->batch > 0x7fffffffLL / s->groups) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

NormParams norm_params(const group_norm_shape* s) {
  NormParams p;
  memset(&p, 0, sizeof(p));
  p.N = s->batch;
  p.S = s->rows;
  p.C = s->channels;
  p.G = s->groups;
  p.cg = s->channels / s->groups;
  p.eps = s->eps;
  p.act = s->activation;
  memcpy(p.xs, s->x_stride, sizeof(p.xs));
  memcpy(p.ds, s->dy_stride, sizeof(p.ds));
  return p;
}

ssd_status done(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

// How a shape runs, and where its scratch lies.  Only the sizes decide (not the pointers or the
// device), so the workspace's size is known beforehand.
constexpr int kGridBlocks = 152 * 8;    // blocks that a map kernel is cut into, at least
constexpr int kTokenBlocks = 152 * 4;   // blocks of the token backward, which writes a partial row each
constexpr int kFoldRows = 64;           // partial rows are first joined to so many where there are many
constexpr int kTokenWidth = 4 * kThreads;   // vectors of a group that a token kernel holds in registers
struct NormPlan {
  int64_t part_rows = 0;
  int32_t chunks = 1;
  int64_t chunk_rows = 1;
  size_t stats = 0, part_w = 0, part_b = 0, total = 0;
};

// Largest vector (in values) that divides a group.
int max_vec(const group_norm_shape* s) {
  const int64_t cg = s->channels / s->groups;
  int v = s->io_dtype == SSD_BF16 ? 8 : 4;
  while (cg % v != 0) v /= 2;
  return v;
}

// Groups of a map kernel's column tile: as many as fill a block.
int64_t tile_groups(int64_t G, int64_t gv) { return std::max<int64_t>(1, std::min<int64_t>(G, kThreads / gv)); }

bool runs_as_tokens(int64_t S, int64_t G, int64_t gv) { return S == 1 && G <= 65535 && gv <= kTokenWidth; }

NormPlan norm_plan(const group_norm_shape* s, bool backward) {
  NormPlan L;
  const int64_t cg = s->channels / s->groups, gv = cg / max_vec(s), N = s->batch, S = s->rows;
  const int64_t tg = tile_groups(s->groups, gv);
  const int64_t blocks = std::max<int64_t>(1, N * ((s->groups + tg - 1) / tg));
  // enough chunks for the grid, none shorter than 16 positions, at most 1024 of them
  L.chunks = (int32_t)std::max<int64_t>(
      1, std::min<int64_t>({(kGridBlocks + blocks - 1) / blocks, (S + 15) / 16, 1024}));
  L.chunk_rows = std::max<int64_t>(1, (S + L.chunks - 1) / L.chunks);
  L.chunks = (int32_t)std::max<int64_t>(1, (S + L.chunk_rows - 1) / L.chunk_rows);
  size_t off = sizeof(WsHeader);
  L.stats = off;
  off = align_up(off + sizeof(float) * 2 * (size_t)(N * L.chunks * s->groups), kWsAlign);
  if (backward) {
    // a narrower vector (rows that are not aligned) may send a token's group to the map kernels
    L.part_rows = runs_as_tokens(S, s->groups, cg) ? kTokenBlocks
                : runs_as_tokens(S, s->groups, gv) ? std::max<int64_t>(kTokenBlocks, N)
                                                   : N * L.chunks;
    L.part_w = off;
    off = align_up(off + sizeof(float) * (size_t)((L.part_rows + kFoldRows) * s->channels), kWsAlign);
    L.part_b = off;
    off = align_up(off + sizeof(float) * (size_t)((L.part_rows + kFoldRows) * s->channels), kWsAlign);
  }
  L.total = off;
  return L;
}

// Vector width of a call: max_vec, or less where the arrays' rows are not aligned to it.
int call_vec(const group_norm_shape* s, std::initializer_list<const void*> arrays,
             std::initializer_list<const int64_t*> strides) {
  const uint64_t e = s->io_dtype == SSD_BF16 ? 2 : 4;
  uint64_t bits = 0;
  for (const void* a : arrays) bits |= reinterpret_cast<uintptr_t>(a);
  for (const int64_t* st : strides) bits |= (uint64_t)(st[0] | st[1]) * e;
  int v = max_vec(s);
  while (v > 1 && bits % (v * e) != 0) v /= 2;
  return v;
}

// Joins the partial rows of the parameters' gradients: at once, or where there are many through
// kFoldRows of them behind the others.
cudaError_t launch_param_grad(NormParams p, cudaStream_t st) {
  if (p.part_rows == 0) return cudaSuccess;
  const unsigned grid = (unsigned)((p.C + 31) / 32);
  if (p.part_rows > 16 * kFoldRows) {
    NormParams f = p;
    f.dw = p.part_w + p.part_rows * p.C;
    f.db = p.part_b + p.part_rows * p.C;
    norm_param_grad_kernel<<<dim3(grid, kFoldRows), 1024, 0, st>>>(f);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.part_w = f.dw;
    p.part_b = f.db;
    p.part_rows = kFoldRows;
  }
  norm_param_grad_kernel<<<dim3(grid, 1), 1024, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int V, int K, bool kBlock, bool kSilu>
cudaError_t launch_tokens(NormParams p, bool backward, cudaStream_t st) {
  constexpr int U = K == 1 ? 4 : K == 2 ? 2 : 1;
  const int64_t gv = p.cg / V;
  p.lanes = 1;
  while (!kBlock && p.lanes < 32 && p.lanes * K < gv) p.lanes *= 2;
  const int64_t slots = p.G * p.lanes;
  const int64_t rows = kBlock || slots >= kThreads ? 1 : kThreads / slots;
  const int64_t by = kBlock ? p.G : (slots + kThreads - 1) / kThreads;
  const int64_t steps = (p.N + rows * U - 1) / (rows * U);
  // forward: four blocks' worth of steps an SM at a time, each going on over the samples
  int64_t bx = std::min<int64_t>(steps, std::max<int64_t>(1, 152 * 8 / by));
  if (backward) {
    bx = std::min<int64_t>(steps, std::max<int64_t>(1, kTokenBlocks / by));
    p.part_rows = p.dw || p.db ? bx : 0;
    norm_token_backward_kernel<T, V, K, U, kBlock, kSilu><<<dim3((unsigned)bx, (unsigned)by), kThreads, 0, st>>>(p);
  } else {
    norm_token_forward_kernel<T, V, K, U, kBlock, kSilu><<<dim3((unsigned)bx, (unsigned)by), kThreads, 0, st>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess && backward ? launch_param_grad(p, st) : e;
}

template <typename T, int V, bool kSilu>
cudaError_t launch_as(NormParams p, bool backward, cudaStream_t st) {
  const int64_t gv = p.cg / V;
  if (runs_as_tokens(p.S, p.G, gv)) {
    if (gv <= 32) return launch_tokens<T, V, 1, false, kSilu>(p, backward, st);
    if (gv <= 64) return launch_tokens<T, V, 2, false, kSilu>(p, backward, st);
    if (gv <= 128) return launch_tokens<T, V, 4, false, kSilu>(p, backward, st);
    if (gv <= 256) return launch_tokens<T, V, 1, true, kSilu>(p, backward, st);
    if (gv <= 512) return launch_tokens<T, V, 2, true, kSilu>(p, backward, st);
    return launch_tokens<T, V, 4, true, kSilu>(p, backward, st);
  }
  p.tile_groups = (int32_t)tile_groups(p.G, gv);
  p.part_rows = p.dw || p.db ? p.N * p.chunks : 0;
  const unsigned grid = (unsigned)(p.N * ((p.G + p.tile_groups - 1) / p.tile_groups) * p.chunks);
  if (!backward) {
    norm_map_stats_kernel<T, V><<<grid, kThreads, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    norm_map_apply_kernel<T, V, kSilu><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  norm_map_grad_sums_kernel<T, V, kSilu><<<grid, kThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_map_grad_apply_kernel<T, V, kSilu><<<grid, kThreads, 0, st>>>(p);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_param_grad(p, st) : e;
}

template <typename T, int V>
cudaError_t launch_act(const NormParams& p, bool backward, cudaStream_t st) {
  return p.act == SSD_ACT_SILU ? launch_as<T, V, true>(p, backward, st)
                               : launch_as<T, V, false>(p, backward, st);
}

cudaError_t launch(NormParams p, const group_norm_shape* s, int vec, bool backward, char* ws, cudaStream_t st) {
  const NormPlan L = norm_plan(s, backward);
  p.chunks = L.chunks;
  p.chunk_rows = L.chunk_rows;
  p.stats = reinterpret_cast<float*>(ws + L.stats);
  p.part_w = reinterpret_cast<float*>(ws + L.part_w);
  p.part_b = reinterpret_cast<float*>(ws + L.part_b);
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  if (s->io_dtype == SSD_BF16)
    return vec == 8 ? launch_act<__nv_bfloat16, 8>(p, backward, st)
         : vec == 4 ? launch_act<__nv_bfloat16, 4>(p, backward, st)
         : vec == 2 ? launch_act<__nv_bfloat16, 2>(p, backward, st)
                    : launch_act<__nv_bfloat16, 1>(p, backward, st);
  return vec == 4 ? launch_act<float, 4>(p, backward, st)
       : vec == 2 ? launch_act<float, 2>(p, backward, st)
                  : launch_act<float, 1>(p, backward, st);
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

size_t group_norm_workspace_bytes(const group_norm_shape* shape, int32_t backward) {
  if (check_shape(shape, false) != SSD_OK) return 0;
  return norm_plan(shape, backward != 0).total;
}

ssd_status group_norm_forward(const group_norm_shape* shape, const void* x, const float* weight,
                              const float* bias, void* y, float* mean, float* rstd,
                              void* workspace, size_t workspace_bytes, void* stream) {
  const ssd_status bad = check_shape(shape, false);
  if (bad != SSD_OK) return bad;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  const bool empty = shape->batch == 0 || shape->rows == 0;
  if ((!empty && (!x || !y)) || (mean == nullptr) != (rstd == nullptr)) return SSD_ERR_INVALID_ARG;
  if (misaligned(x, e) || misaligned(y, e) || misaligned(weight, 4) || misaligned(bias, 4) ||
      misaligned(mean, 4) || misaligned(rstd, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, kWsAlign) ||
      workspace_bytes < group_norm_workspace_bytes(shape, 0))
    return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) return SSD_OK;
  NormParams p = norm_params(shape);
  p.x = x;
  p.w = weight;
  p.bias = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  const int vec = call_vec(shape, {x, y}, {p.xs});
  return done(launch(p, shape, vec, false, static_cast<char*>(workspace), st));
}

ssd_status group_norm_backward(const group_norm_shape* shape, const void* x, const void* dy,
                               const float* mean, const float* rstd, const float* weight,
                               const float* bias, void* dx, float* dweight, float* dbias,
                               void* workspace, size_t workspace_bytes, void* stream) {
  const ssd_status bad = check_shape(shape, true);
  if (bad != SSD_OK) return bad;
  const bool bf16 = shape->io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  const bool empty = shape->batch == 0 || shape->rows == 0;
  if (!empty && (!x || !dy || !dx || !mean || !rstd)) return SSD_ERR_INVALID_ARG;
  if (misaligned(x, e) || misaligned(dy, e) || misaligned(dx, e) || misaligned(weight, 4) ||
      misaligned(bias, 4) || misaligned(mean, 4) || misaligned(rstd, 4) ||
      misaligned(dweight, 4) || misaligned(dbias, 4))
    return SSD_ERR_INVALID_ARG;
  if (!workspace || misaligned(workspace, kWsAlign) ||
      workspace_bytes < group_norm_workspace_bytes(shape, 1))
    return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (empty) {
    for (float* d : {dweight, dbias})
      if (d && cudaMemsetAsync(d, 0, sizeof(float) * (size_t)shape->channels, st) != cudaSuccess)
        return SSD_ERR_CUDA;
    return SSD_OK;
  }
  NormParams p = norm_params(shape);
  p.x = x;
  p.dy = dy;
  p.mean_in = mean;
  p.rstd_in = rstd;
  p.w = weight;
  p.bias = bias;
  p.dx = dx;
  p.dw = dweight;
  p.db = dbias;
  const int vec = call_vec(shape, {x, dy, dx}, {p.xs, p.ds});
  return done(launch(p, shape, vec, true, static_cast<char*>(workspace), st));
}

}  // extern "C"
