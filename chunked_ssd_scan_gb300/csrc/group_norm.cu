// Group norm with an activation, channels last (declarations in include/ssdscan.h):
//   xhat = (x - mean) rstd, z = xhat w + b, y = act(z), statistics over the S * C/G values of a
//   sample's group; reverse mode, dz = dy act'(z), q = dz w:
//   dx = rstd (q - mean(q) - xhat mean(q xhat)), dw = sum dz xhat, db = sum dz.
#include "group_norm.cuh"

namespace ssd {
namespace norm {
namespace {

// ------------------------------------------------------------------------------------------------
// Many positions a sample: a sample's positions are cut into chunks, a block takes one chunk of one
// sample by one column tile of whole groups.  Two passes over x: the chunks' statistics, a join of
// them by one warp a group, and the output; the second pass goes through the samples backwards, so
// that what the first read last is still in L2.
//
// 6 x 3969 x 320 f32, 32 groups: 24 us for 61 MB (37 % of the measured copy rate: the statistics take 10 us,
// their join 3, the output 12, of which 5 are writes); 8 x 4096 x 512 bf16 backward: 39 us for 101 MB
// (38 %).  Vectors divide a group, so that a thread's values belong to one group each; a group of 10
// f32 channels takes 8-byte loads.
// ------------------------------------------------------------------------------------------------
// count, mean and sum of squares around the mean; joined pairwise (Chan, Golub and LeVeque), so no
// difference of large squares is formed.  The approximate division is good to 2^-22: it moves a joined mean by so
// much of the two means' distance, and counts in the sum of squares in the second order only.
struct Moments {
  float n, mean, m2;
};
__device__ __forceinline__ Moments join(const Moments& a, const Moments& b) {
  if (b.n == 0.f) return a;
  if (a.n == 0.f) return b;
  const float n = a.n + b.n, f = __fdividef(b.n, n), d = b.mean - a.mean;
  return {n, fmaf(d, f, a.mean), fmaf(d * d, a.n * f, a.m2 + b.m2)};
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
  int64_t n, s0, s1;                // sample (or the first of them), positions [s0, s1)
  int chunk, g0, groups;            // chunk, groups of the tile
  int gv, vecs, cols, rows, row, col;   // vectors of a group and of the tile, thread columns and rows
  __device__ __forceinline__ MapSlot(const NormParams& p, uint32_t block) {
    const uint32_t tiles = ((uint32_t)p.G + p.tile_groups - 1) / p.tile_groups;
    const uint32_t tile = block % tiles, rest = block / tiles;
    chunk = (int)(rest % (uint32_t)p.chunks);
    n = rest / (uint32_t)p.chunks;
    g0 = (int)tile * p.tile_groups;
    groups = min(p.tile_groups, (int)p.G - g0);
    gv = (int)p.cg / V;
    vecs = groups * gv;
    cols = min(vecs, kThreads);
    rows = kThreads / cols;
    row = threadIdx.x / cols;
    col = threadIdx.x % cols;
    s0 = chunk * p.chunk_rows;
    s1 = min(p.S, s0 + p.chunk_rows);
  }
  __device__ __forceinline__ int64_t channel(const NormParams& p, int v) const { return g0 * p.cg + (int64_t)v * V; }
};

// The positions of a thread in x and dy, U of them in flight ahead of those worked on.
template <typename T, int V, int U>
struct Pairs {
  using Raw = typename Pack<T, V>::Raw;
  const T *x, *dy;
  int64_t px, py;
  int left;   // positions still to load
  Raw nx[U], ny[U];
  __device__ __forceinline__ Pairs(const NormParams& p, const MapSlot<V>& t, int64_t c)
      : x(static_cast<const T*>(p.x) + t.n * p.xs[0] + (t.s0 + t.row) * p.xs[1] + c),
        dy(static_cast<const T*>(p.dy) + t.n * p.ds[0] + (t.s0 + t.row) * p.ds[1] + c),
        px(t.rows * p.xs[1]),
        py(t.rows * p.ds[1]),
        left((int)((t.s1 - t.s0 - t.row + t.rows - 1) / t.rows)) {}
  __device__ __forceinline__ void fetch() {
    if (left >= U) {
#pragma unroll
      for (int u = 0; u < U; ++u, x += px, dy += py) {
        nx[u] = Pack<T, V>::raw(x);
        ny[u] = Pack<T, V>::raw(dy);
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        nx[u] = u < left ? Pack<T, V>::raw(x + u * px) : Pack<T, V>::none();
        ny[u] = u < left ? Pack<T, V>::raw(dy + u * py) : Pack<T, V>::none();
      }
    }
    left -= U;
  }
  __device__ __forceinline__ bool pending() const { return left + U > 0; }
  // hands over what has been loaded, and loads on; how many of them there are
  __device__ __forceinline__ int take(Raw (&rx)[U], Raw (&ry)[U]) {
    const int have = min(U, left + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rx[u] = nx[u];
      ry[u] = ny[u];
    }
    fetch();
    return have;
  }
};

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, kMapForward) norm_map_stats_kernel(NormParams p) {
  using Q = Pack<T, V>;
  constexpr int U = 8;   // positions in flight: their moments are formed directly
  __shared__ Moments all[kThreads];
  follow();
  const MapSlot<V> t(p, blockIdx.x);
  Moments m = {0.f, 0.f, 0.f};
  if (t.row < t.rows)
    for (int v = t.col; v < t.vecs; v += kThreads) {
      const T* x = static_cast<const T*>(p.x) + t.n * p.xs[0] + (t.s0 + t.row) * p.xs[1] + t.channel(p, v);
      const int64_t pitch = t.rows * p.xs[1];
      int left = (int)((t.s1 - t.s0 - t.row + t.rows - 1) / t.rows);   // positions still to load
      typename Q::Raw next[U];
      auto fetch = [&]() {
        if (left >= U) {
#pragma unroll
          for (int u = 0; u < U; ++u, x += pitch) next[u] = Q::raw(x);
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) next[u] = u < left ? Q::raw(x + u * pitch) : Q::none();
        }
        left -= U;
      };
      fetch();
      while (left + U > 0) {
        const int have = min(U, left + U);
        float2 f[U][Q::P], sum = make_float2(0.f, 0.f), sq = sum;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          Q::unpack(next[u], f[u]);
#pragma unroll
          for (int e = 0; e < Q::P; ++e) sum = fp::add2(sum, f[u][e]);
        }
        fetch();
        const float n = (float)(have * V), mean = __fdividef(sum.x + sum.y, n);
        auto squares = [&](auto whole) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < Q::P; ++e) {
              const float2 d = decltype(whole)::value || u < have ? minus2<V>(f[u][e], mean) : make_float2(0.f, 0.f);
              sq = fp::fma2(d, d, sq);
            }
        };
        if (have == U) squares(std::true_type());
        else squares(std::false_type());
        m = join(m, {n, mean, sq.x + sq.y});
      }
    }
  all[threadIdx.x] = m;
  __syncthreads();
  // a group's threads are columns [k per, (k + 1) per) of every row: a few of them are joined by one
  // thread, more by a warp
  const int lane = threadIdx.x % 32, per = min(t.gv, t.cols), members = per * t.rows;
  const bool few = members <= 16;
  for (int k = few ? threadIdx.x : threadIdx.x / 32; k < t.groups; k += few ? kThreads : kWarps) {
    Moments g = {0.f, 0.f, 0.f};
    for (int j = few ? 0 : lane; j < members; j += few ? 1 : 32)
      g = join(g, all[j / per * t.cols + k * per + j % per]);
    if (!few) g = join_lanes(g);
    const int64_t at = ((t.n * p.G + t.g0 + k) * p.chunks + t.chunk) * 2;
    if ((few || lane == 0) && SSD_INDEX_OK(p.hdr, at + 1, p.N * p.chunks * p.G * 2, 74))
      *reinterpret_cast<float2*>(p.stats + at) = make_float2(g.mean, g.m2);
  }
}

// Writes a partial sum, or adds to it; one thread alone does so, in its order (the addition is an atomic one
// because it does not wait for the value that it adds to).
__device__ __forceinline__ void put(float* p, float v, bool more) {
  if (more) atomicAdd(p, v);
  else *p = v;
}

// Per chunk and channel, sum dz and sum dz xhat (which are the parameters' gradients' partials), and per
// group their sums times w, which the gradient of x needs.  Where there are more samples than slots, a
// block takes every slots-th sample and adds to the partial row that it wrote for the first.
template <typename T, int V, bool kSilu>
__global__ void __launch_bounds__(kThreads, kMapBackward) norm_map_grad_sums_kernel(NormParams p) {
  using Q = Pack<T, V>;
  constexpr int U = 4;
  __shared__ float4 all[kThreads][Q::P];
  __shared__ float2 wide[kThreads];
  follow();
  MapSlot<V> t(p, blockIdx.x);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (; t.n < p.N; t.n += p.slots) {
    float2 mine = make_float2(0.f, 0.f);   // of the first row's threads: their channels' sums times w
    for (int v0 = 0; v0 < t.vecs; v0 += kThreads) {
      const int v = v0 + t.col;
      float2 dw[Q::P], db[Q::P], w[Q::P];
      Q::zero(dw);
      Q::zero(db);
      Q::zero(w);
      if (t.row < t.rows && v < t.vecs) {
        const int64_t c = t.channel(p, v), at = t.n * p.G + t.g0 + v / t.gv;
        const float mean = __ldg(p.mean_in + at), rstd = __ldg(p.rstd_in + at);
        float2 bias[Q::P];
        Q::param(p.w, c, 1.f, w);
        Q::param(p.bias, c, 0.f, bias);
        Pairs<T, V, U> in(p, t, c);
        in.fetch();
        while (in.pending()) {
          typename Q::Raw rx[U], ry[U];
          in.take(rx, ry);
#pragma unroll
          for (int u = 0; u < U; ++u) {   // past the end dy = 0: nothing is added
            float2 f[Q::P], d[Q::P];
            Q::unpack(rx[u], f);
            Q::unpack(ry[u], d);
#pragma unroll
            for (int e = 0; e < Q::P; ++e) {
              const float2 xh = fp::mul2(minus2<V>(f[e], mean), dup(rstd));
              const float2 dz = times_act_grad2<kSilu>(d[e], fp::fma2(xh, w[e], bias[e]));
              db[e] = fp::add2(db[e], dz);
              dw[e] = fp::fma2(dz, xh, dw[e]);
            }
          }
        }
      }
      // over the block's rows, per channel
      __syncthreads();
#pragma unroll
      for (int e = 0; e < Q::P; ++e) all[threadIdx.x][e] = make_float4(db[e].x, db[e].y, dw[e].x, dw[e].y);
      __syncthreads();
      if (t.row == 0 && v < t.vecs) {
        const bool more = t.n >= p.slots;   // not the block's first sample
        const uint32_t slot = (uint32_t)t.n % (uint32_t)p.slots;   // fewer than 2^31 samples
        const int64_t at = ((int64_t)slot * p.chunks + t.chunk) * p.C + t.channel(p, v);
#pragma unroll
        for (int e = 0; e < Q::P; ++e) {
          for (int r = 1; r < t.rows; ++r) {
            const float4 a = all[r * t.cols + t.col][e];
            db[e] = fp::add2(db[e], make_float2(a.x, a.y));
            dw[e] = fp::add2(dw[e], make_float2(a.z, a.w));
          }
          if (p.part_rows > 0 && SSD_INDEX_OK(p.hdr, at + min(2 * e + 1, V - 1), p.part_rows * p.C, 77)) {
            put(p.part_b + at + 2 * e, db[e].x, more);
            put(p.part_w + at + 2 * e, dw[e].x, more);
            if (V > 1) {
              put(p.part_b + at + 2 * e + 1, db[e].y, more);
              put(p.part_w + at + 2 * e + 1, dw[e].y, more);
            }
          }
          mine.x += fmaf(db[e].x, w[e].x, db[e].y * w[e].y);
          mine.y += fmaf(dw[e].x, w[e].x, dw[e].y * w[e].y);
        }
      }
    }
    wide[threadIdx.x] = mine;
    __syncthreads();
    const int per = min(t.gv, t.cols);
    for (int k = warp; k < t.groups; k += kWarps) {
      float2 s = make_float2(0.f, 0.f);
      for (int j = lane; j < per; j += 32) s = fp::add2(s, wide[k * per + j]);
#pragma unroll
      for (int o = 16; o > 0; o /= 2)
        s = fp::add2(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
      const int64_t at = ((t.n * p.G + t.g0 + k) * p.chunks + t.chunk) * 2;
      if (lane == 0 && SSD_INDEX_OK(p.hdr, at + 1, p.N * p.chunks * p.G * 2, 78))
        *reinterpret_cast<float2*>(p.stats + at) = s;
    }
  }
}

// One warp a (sample, group): the chunks' statistics joined into `joined` [N, G, 2]: mean and rstd, or the
// means of q and q xhat.  The blocks behind the groups' join the parameters' gradients instead (see
// param_grad).
template <bool kGrad>
__global__ void __launch_bounds__(1024) norm_map_join_kernel(NormParams p, uint32_t group_blocks) {
  follow();
  if (blockIdx.x >= group_blocks) {
    if (kGrad) param_grad(p, blockIdx.x - group_blocks);
    return;
  }
  const int64_t at = (int64_t)blockIdx.x * 32 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (at >= p.N * p.G) return;
  const float2* st = reinterpret_cast<const float2*>(p.stats) + at * p.chunks;
  constexpr int kAhead = 4;   // loads of a lane in flight
  float2 out;
  if (kGrad) {
    float2 m = make_float2(0.f, 0.f);
    for (int c0 = lane; c0 < p.chunks; c0 += 32 * kAhead) {
      float2 s[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) s[k] = c0 + 32 * k < p.chunks ? __ldcg(st + c0 + 32 * k) : make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) m = fp::add2(m, s[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2)
      m = fp::add2(m, make_float2(__shfl_xor_sync(0xffffffffu, m.x, o), __shfl_xor_sync(0xffffffffu, m.y, o)));
    const float inv = 1.f / ((float)p.S * (float)p.cg);
    out = make_float2(m.x * inv, m.y * inv);
  } else {
    Moments m = {0.f, 0.f, 0.f};
    for (int c0 = lane; c0 < p.chunks; c0 += 32 * kAhead) {
      float2 s[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) s[k] = c0 + 32 * k < p.chunks ? __ldcg(st + c0 + 32 * k) : make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int c = c0 + 32 * k;
        const float n = (float)(min(p.S, (c + 1) * p.chunk_rows) - c * p.chunk_rows) * (float)p.cg;
        if (c < p.chunks) m = join(m, {n, s[k].x, s[k].y});
      }
    }
    m = join_lanes(m);
    out = make_float2(m.mean, rsqrtf(m.m2 / m.n + p.eps));
    if (lane == 0 && p.mean && SSD_INDEX_OK(p.hdr, at, p.N * p.G, 75)) {
      p.mean[at] = out.x;
      p.rstd[at] = out.y;
    }
  }
  if (lane == 0) reinterpret_cast<float2*>(p.joined)[at] = out;
}

template <typename T, int V, bool kSilu>
__global__ void __launch_bounds__(kThreads, kMapForward) norm_map_apply_kernel(NormParams p) {
  follow();
  using Q = Pack<T, V>;
  constexpr int U = V * (int)sizeof(T) >= 16 ? 4 : 8;
  const MapSlot<V> t(p, gridDim.x - 1 - blockIdx.x);
  if (t.row >= t.rows) return;
  for (int v = t.col; v < t.vecs; v += kThreads) {
    const int64_t c = t.channel(p, v);
    const float2 st = __ldcg(reinterpret_cast<const float2*>(p.joined) + t.n * p.G + t.g0 + v / t.gv);
    float2 a[Q::P], b[Q::P];   // (x - mean) a + b: x a + b' would round around a large mean
    Q::param(p.w, c, 1.f, a);
    Q::param(p.bias, c, 0.f, b);
#pragma unroll
    for (int e = 0; e < Q::P; ++e) a[e] = fp::mul2(a[e], dup(st.y));
    const T* x = static_cast<const T*>(p.x) + t.n * p.xs[0] + (t.s0 + t.row) * p.xs[1] + c;
    T* y = static_cast<T*>(p.y) + (t.n * p.S + t.s0 + t.row) * p.C + c;
    const int64_t pitch = t.rows * p.xs[1], out = t.rows * p.C;
    int left = (int)((t.s1 - t.s0 - t.row + t.rows - 1) / t.rows);
    typename Q::Raw next[U];
    auto fetch = [&]() {
      if (left >= U) {
#pragma unroll
        for (int u = 0; u < U; ++u, x += pitch) next[u] = Q::raw(x);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = u < left ? Q::raw(x + u * pitch) : Q::none();
      }
      left -= U;
    };
    fetch();
    while (left + U > 0) {
      const int have = min(U, left + U);
      typename Q::Raw now[U];
#pragma unroll
      for (int u = 0; u < U; ++u) now[u] = next[u];
      fetch();
      auto write = [&](auto whole) {
#pragma unroll
        for (int u = 0; u < U; ++u, y += out) {
          float2 f[Q::P];
          Q::unpack(now[u], f);
#pragma unroll
          for (int e = 0; e < Q::P; ++e) f[e] = act2<kSilu>(fp::fma2(minus2<V>(f[e], st.x), a[e], b[e]));
          if ((decltype(whole)::value || u < have) &&
              SSD_INDEX_OK(p.hdr, (y - static_cast<T*>(p.y)) + V - 1, p.N * p.S * p.C, 76))
            Q::store(y, f);
        }
      };
      if (have == U) write(std::true_type());
      else write(std::false_type());
    }
  }
}

template <typename T, int V, bool kSilu>
__global__ void __launch_bounds__(kThreads, kMapBackward) norm_map_grad_apply_kernel(NormParams p) {
  follow();
  using Q = Pack<T, V>;
  constexpr int U = 4;
  const MapSlot<V> t(p, gridDim.x - 1 - blockIdx.x);
  if (t.row >= t.rows) return;
  for (int v = t.col; v < t.vecs; v += kThreads) {
    const int64_t c = t.channel(p, v), at = t.n * p.G + t.g0 + v / t.gv;
    const float mean = __ldg(p.mean_in + at), rstd = __ldg(p.rstd_in + at);
    const float2 m = __ldcg(reinterpret_cast<const float2*>(p.joined) + at);
    float2 w[Q::P], bias[Q::P];
    Q::param(p.w, c, 1.f, w);
    Q::param(p.bias, c, 0.f, bias);
    T* dx = static_cast<T*>(p.dx) + (t.n * p.S + t.s0 + t.row) * p.C + c;
    const int64_t out = t.rows * p.C;
    Pairs<T, V, U> in(p, t, c);
    in.fetch();
    while (in.pending()) {
      typename Q::Raw rx[U], ry[U];
      const int have = in.take(rx, ry);
      auto write = [&](auto whole) {
#pragma unroll
        for (int u = 0; u < U; ++u, dx += out) {
          float2 f[Q::P], d[Q::P];
          Q::unpack(rx[u], f);
          Q::unpack(ry[u], d);
#pragma unroll
          for (int e = 0; e < Q::P; ++e) {
            const float2 xh = fp::mul2(minus2<V>(f[e], mean), dup(rstd));
            const float2 q = fp::mul2(times_act_grad2<kSilu>(d[e], fp::fma2(xh, w[e], bias[e])), w[e]);
            f[e] = fp::mul2(dup(rstd), fp::fma2(xh, dup(-m.y), fp::add2(q, dup(-m.x))));
          }
          if ((decltype(whole)::value || u < have) &&
              SSD_INDEX_OK(p.hdr, (dx - static_cast<T*>(p.dx)) + V - 1, p.N * p.S * p.C, 79))
            Q::store(dx, f);
        }
      };
      if (have == U) write(std::true_type());
      else write(std::false_type());
    }
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
struct NormPlan {
  int64_t part_rows = 0;
  int32_t chunks = 1;
  int64_t chunk_rows = 1;
  size_t stats = 0, joined = 0, part_w = 0, part_b = 0, total = 0;
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

// Samples side by side in the gradient sums; samples in chunks are few.
int64_t map_slots(int64_t N, int64_t chunks) { return chunks > 1 ? N : std::min<int64_t>(N, kMapRows); }

NormPlan norm_plan(const group_norm_shape* s, bool backward) {
  NormPlan L;
  const int64_t cg = s->channels / s->groups, gv = cg / max_vec(s), N = s->batch, S = s->rows;
  const int64_t tg = tile_groups(s->groups, gv);
  const int64_t blocks = std::max<int64_t>(1, N * ((s->groups + tg - 1) / tg));
  // enough chunks for one round of blocks, none shorter than 16 positions, at most 1024 of them
  const int64_t round = (int64_t)kGridBlocks * (backward ? kMapBackward : kMapForward);
  L.chunks = (int32_t)std::max<int64_t>(1, std::min<int64_t>({round / blocks, (S + 15) / 16, 1024}));
  L.chunk_rows = std::max<int64_t>(1, (S + L.chunks - 1) / L.chunks);
  L.chunks = (int32_t)std::max<int64_t>(1, (S + L.chunk_rows - 1) / L.chunk_rows);
  size_t off = sizeof(WsHeader);
  L.stats = off;
  off = align_up(off + sizeof(float) * 2 * (size_t)(N * L.chunks * s->groups), kWsAlign);
  L.joined = off;
  off = align_up(off + sizeof(float) * 2 * (size_t)(N * s->groups), kWsAlign);
  if (backward) {
    // a narrower vector (rows that are not aligned) may send a token's group to the map kernels
    const int64_t maps = map_slots(N, L.chunks) * L.chunks;
    L.part_rows = runs_as_tokens(S, s->groups, cg) ? kTokenBlocks
                : runs_as_tokens(S, s->groups, gv) ? std::max<int64_t>(kTokenBlocks, maps)
                                                   : maps;
    L.part_w = off;
    off = align_up(off + sizeof(float) * (size_t)(L.part_rows * s->channels), kWsAlign);
    L.part_b = off;
    off = align_up(off + sizeof(float) * (size_t)(L.part_rows * s->channels), kWsAlign);
  }
  L.total = off;
  return L;
}

// Vector width of a call: max_vec, or less where the arrays' rows are not aligned to it.  The gradient of
// a map takes 8 bytes at most: with 16 its registers leave room for one block an SM less (8 x 4096 x 512
// bf16: 39 us, 63 us with 16; tokens: 47 us with 16, 67 us with 8, forward 29 and 42 us).
int call_vec(const group_norm_shape* s, std::initializer_list<const void*> arrays,
             std::initializer_list<const int64_t*> strides, bool backward, bool* aligned) {
  const uint64_t e = s->io_dtype == SSD_BF16 ? 2 : 4;
  uint64_t bits = backward && s->rows > 1 ? 8 : 0;
  for (const void* a : arrays) bits |= reinterpret_cast<uintptr_t>(a);
  for (const int64_t* st : strides) bits |= (uint64_t)(st[0] | st[1]) * e;
  *aligned = ((bits & ~(uint64_t)(backward && s->rows > 1 ? 8 : 0)) | (uint64_t)s->channels * e) % 16 == 0;
  int v = max_vec(s);
  while (v > 1 && bits % (v * e) != 0) v /= 2;
  return v;
}

// The map kernels' tiles for vectors of V values; blocks of one sample.
int64_t map_tiles(NormParams& p, int V) {
  p.tile_groups = (int32_t)tile_groups(p.G, p.cg / V);
  return (p.G + p.tile_groups - 1) / p.tile_groups * p.chunks;
}

template <typename T, int V, bool kSilu>
cudaError_t launch_map_forward(NormParams p, cudaStream_t st) {
  const unsigned grid = (unsigned)(p.N * map_tiles(p, V)), group_blocks = (unsigned)((p.N * p.G + 31) / 32);
  norm_map_stats_kernel<T, V><<<grid, kThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_next(norm_map_join_kernel<false>, group_blocks, 1024, 0, st, p, group_blocks);
  if (e != cudaSuccess) return e;
  return launch_next(norm_map_apply_kernel<T, V, kSilu>, grid, kThreads, 0, st, p);
}

template <typename T, int V, bool kSilu>
cudaError_t launch_map_backward(NormParams p, cudaStream_t st) {
  const int64_t blocks = map_tiles(p, V);
  const unsigned group_blocks = (unsigned)((p.N * p.G + 31) / 32);
  p.slots = map_slots(p.N, p.chunks);
  p.part_rows = p.dw || p.db ? p.slots * p.chunks : 0;
  norm_map_grad_sums_kernel<T, V, kSilu><<<(unsigned)(p.slots * blocks), kThreads, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the join's launch takes the parameters' gradients along
  const unsigned more = p.part_rows > 0 ? (unsigned)((p.C + 31) / 32) : 0u;
  e = launch_next(norm_map_join_kernel<true>, group_blocks + more, 1024, 0, st, p, group_blocks);
  if (e != cudaSuccess) return e;
  return launch_next(norm_map_grad_apply_kernel<T, V, kSilu>, (unsigned)(p.N * blocks), kThreads, 0, st, p);
}

template <typename T, int V, bool kSilu>
cudaError_t launch_as(const NormParams& p, bool backward, cudaStream_t st) {
  if (runs_as_tokens(p.S, p.G, p.cg / V)) return run_tokens<T, V>(p, backward, st);
  if (!backward) return launch_map_forward<T, V, kSilu>(p, st);
  // gradients take 8 bytes at most, as of maps (call_vec): 16384 x 16384 bf16 in one group 5.0 ms with 16, whose
  // registers spilled, and 2.8 with 8
  return launch_map_backward<T, (V * (int)sizeof(T) > 8 ? V / 2 : V), kSilu>(p, st);
}

template <typename T, int V>
cudaError_t launch_act(const NormParams& p, bool backward, cudaStream_t st) {
  return p.act == SSD_ACT_SILU ? launch_as<T, V, true>(p, backward, st)
                               : launch_as<T, V, false>(p, backward, st);
}

// Tokens whose groups only narrow vectors divide, but whose rows take wide ones.  Not for few of them: the
// joins' barriers cost 64 x 520 bf16 2.4 us more (6.5 against 4.1), and save 23795 x 520 18 us (37
// against 55).
constexpr int64_t kStraddleValues = 1 << 17;
bool straddles(const group_norm_shape* s, int vec, bool aligned) {
  const int64_t cg = s->channels / s->groups, e = s->io_dtype == SSD_BF16 ? 2 : 4;
  return s->rows == 1 && aligned && vec * e <= 4 && cg * e >= kStraddleLeast && cg <= kThreads &&
         s->groups <= 65535 && s->batch * s->channels >= kStraddleValues;
}

cudaError_t launch(NormParams p, const group_norm_shape* s, int vec, bool aligned, bool backward, char* ws,
                   cudaStream_t st) {
  const NormPlan L = norm_plan(s, backward);
  p.chunks = L.chunks;
  p.chunk_rows = L.chunk_rows;
  p.stats = reinterpret_cast<float*>(ws + L.stats);
  p.joined = reinterpret_cast<float*>(ws + L.joined);
  p.part_w = reinterpret_cast<float*>(ws + L.part_w);
  p.part_b = reinterpret_cast<float*>(ws + L.part_b);
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  if (straddles(s, vec, aligned))
    return s->io_dtype == SSD_BF16 ? run_straddle<__nv_bfloat16>(p, backward, st) : run_straddle<float>(p, backward, st);
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
}  // namespace norm
}  // namespace ssd

using namespace ssd;
using namespace ssd::norm;

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
  if (empty) {   // samples without positions: the mean of nothing is NaN, all its bits set
    const size_t bytes = sizeof(float) * (size_t)(shape->batch * shape->groups);
    for (float* d : {mean, rstd})
      if (d && bytes > 0 && cudaMemsetAsync(d, 0xff, bytes, st) != cudaSuccess) return SSD_ERR_CUDA;
    return SSD_OK;
  }
  NormParams p = norm_params(shape);
  p.x = x;
  p.w = weight;
  p.bias = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  bool aligned = false;
  const int vec = call_vec(shape, {x, y}, {p.xs}, false, &aligned);
  return done(launch(p, shape, vec, aligned, false, static_cast<char*>(workspace), st));
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
  bool aligned = false;
  const int vec = call_vec(shape, {x, dy, dx}, {p.xs, p.ds}, true, &aligned);
  return done(launch(p, shape, vec, aligned, true, static_cast<char*>(workspace), st));
}

}  // extern "C"
