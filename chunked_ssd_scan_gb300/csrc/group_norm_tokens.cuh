#pragma once
// Group norm of tokens (one position a sample) and its gradient; see group_norm.cu for the formulas.
#include "group_norm.cuh"

namespace ssd {
namespace norm {
namespace {

// ------------------------------------------------------------------------------------------------
// One position a sample (the norm of every token): a group's values stay in the registers of `lanes`
// neighbouring lanes (or of a whole block), K vectors of V values each; the mean and then the
// squares around it are summed over them by shuffles.  A thread keeps its channels for all the
// samples that its block takes, so weight and bias are read once, and has U samples in flight.
// Bound by memory: x and y once each.  16384 x 2048 bf16, 32 groups: forward 28.7 us, 4.8 TB/s of 138 MB
// (71 % of the measured copy rate; 18 instructions and two special functions a value with SiLU);
// backward 47 us, 4.3 TB/s of 206 MB (64 %; the gradients' sums and both parameters in registers
// leave two blocks an SM).
// ------------------------------------------------------------------------------------------------
template <bool kBlock, int M>
__device__ __forceinline__ void group_sum(float (&v)[M], int lanes, float (&part)[2][kWarps][M], int& phase) {
  if (!kBlock) {
    for (int o = lanes / 2; o > 0; o /= 2) {
#pragma unroll
      for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
    }
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
#pragma unroll
    for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], o);
  }
  if (threadIdx.x % 32 == 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) part[phase][threadIdx.x / 32][m] = v[m];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; ++m) {
    v[m] = part[phase][0][m];
#pragma unroll
    for (int k = 1; k < kWarps; ++k) v[m] += part[phase][k][m];
  }
  phase ^= 1;   // the next sum writes elsewhere, and its barrier ends the reads of this one
}

// What a thread of a token kernel works on.
template <int V, int K, bool kBlock>
struct TokenSlot {
  int64_t g, c;           // its group and its first channel
  int row, rows;          // its sample within a block's step, samples of a step
  bool in[K];             // which of its vectors lie inside the group
  int step;               // channels from one of its vectors to the next
  __device__ __forceinline__ TokenSlot(const NormParams& p) {
    int l;
    row = 0;
    rows = 1;
    if (kBlock) {
      g = blockIdx.y;
      l = threadIdx.x;
      step = kThreads * V;
    } else {
      const int64_t slots = p.G * p.lanes;
      int64_t s = (int64_t)blockIdx.y * kThreads + threadIdx.x;
      if (slots < kThreads) {
        rows = kThreads / (int)slots;
        row = threadIdx.x / (int)slots;
        s = row < rows ? threadIdx.x % (int)slots : slots;   // slots: a thread too many
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

// kFull: every thread has all its K vectors inside its group (and there are none too many).
template <typename T, int V, int K, int U, bool kBlock, bool kSilu, bool kFull>
__global__ void __launch_bounds__(kThreads, kBlock || K > 1 ? 1 : 3) norm_token_forward_kernel(NormParams p) {
  using Q = Pack<T, V>;
  __shared__ float part[2][kWarps][U];
  int phase = 0;
  const TokenSlot<V, K, kBlock> t(p);
  const int lanes = p.lanes;
  float2 w[K][Q::P], bias[K][Q::P];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    Q::zero(w[k]);
    Q::zero(bias[k]);
    if (t.in[k]) {
      Q::param(p.w, t.c + k * t.step, 1.f, w[k]);
      Q::param(p.bias, t.c + k * t.step, 0.f, bias[k]);
    }
  }
  const float inv = 1.f / (float)p.cg;
  const bool first = p.mean && t.in[0] && t.c == t.g * p.cg;   // the lane that writes the statistics
  const int64_t stride = (int64_t)gridDim.x * t.rows * U;
  int64_t n0 = (int64_t)blockIdx.x * t.rows * U;   // the block's first sample
  const T* x_at = static_cast<const T*>(p.x) + (n0 + t.row) * p.xs[0] + t.c;
  T* y_at = static_cast<T*>(p.y) + (n0 + t.row) * p.C + t.c;
  const int64_t px = t.rows * p.xs[0], py = t.rows * p.C;   // from one of the U samples to the next
  typename Q::Raw next[U][K];   // loads in flight while the samples before them are worked on
  auto fetch = [&](int64_t at, auto whole) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < K; ++k)
        next[u][k] = (kFull || t.in[k]) && (decltype(whole)::value || at + u * t.rows + t.row < p.N)
                         ? Q::raw(x_at + u * px + k * t.step)
                         : Q::none();
    x_at += gridDim.x * (U * px);
  };
  auto fetch_any = [&](int64_t at) {
    if (at + U * t.rows <= p.N) fetch(at, std::true_type());
    else fetch(at, std::false_type());
  };
  auto work = [&](auto whole) {
    float2 x[U][K][Q::P];
    float mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < K; ++k) Q::unpack(next[u][k], x[u][k]);
    fetch_any(n0 + stride);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < Q::P; ++e) s = fp::add2(s, x[u][k][e]);
      mean[u] = s.x + s.y;
    }
    group_sum<kBlock>(mean, lanes, part, phase);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mean[u] *= inv;
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < Q::P; ++e) {
          x[u][k][e] = kFull || t.in[k] ? minus2<V>(x[u][k][e], mean[u]) : make_float2(0.f, 0.f);
          s = fp::fma2(x[u][k][e], x[u][k][e], s);
        }
      rstd[u] = s.x + s.y;
    }
    group_sum<kBlock>(rstd, lanes, part, phase);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rstd[u] = rsqrtf(fmaf(rstd[u], inv, p.eps));
      const bool live = decltype(whole)::value || n0 + u * t.rows + t.row < p.N;
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < Q::P; ++e)
          x[u][k][e] = act2<kSilu>(fp::fma2(fp::mul2(x[u][k][e], dup(rstd[u])), w[k][e], bias[k][e]));
        T* to = y_at + u * py + k * t.step;
        if ((kFull || t.in[k]) && live &&
            SSD_INDEX_OK(p.hdr, (to - static_cast<T*>(p.y)) + V - 1, p.N * p.C, 70))
          Q::store(to, x[u][k]);
      }
    }
    if (first) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t n = n0 + u * t.rows + t.row;
        if (n < p.N && SSD_INDEX_OK(p.hdr, n * p.G + t.g, p.N * p.G, 71)) {
          p.mean[n * p.G + t.g] = mean[u];
          p.rstd[n * p.G + t.g] = rstd[u];
        }
      }
    }
    y_at += gridDim.x * (U * py);
  };
  fetch_any(n0);
  for (; n0 < p.N; n0 += stride) {
    if (n0 + U * t.rows <= p.N) work(std::true_type());
    else work(std::false_type());
  }
}

template <typename T, int V, int K, int U, bool kBlock, bool kSilu, bool kFull>
__global__ void __launch_bounds__(kThreads) norm_token_backward_kernel(NormParams p) {
  follow();
  using Q = Pack<T, V>;
  __shared__ float part[2][kWarps][2 * U];
  int phase = 0;
  const TokenSlot<V, K, kBlock> t(p);
  const int lanes = p.lanes;
  float2 w[K][Q::P], bias[K][Q::P], dw[K][Q::P], db[K][Q::P];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    Q::zero(w[k]);
    Q::zero(bias[k]);
    Q::zero(dw[k]);
    Q::zero(db[k]);
    if (t.in[k]) {
      Q::param(p.w, t.c + k * t.step, 1.f, w[k]);
      Q::param(p.bias, t.c + k * t.step, 0.f, bias[k]);
    }
  }
  const float inv = 1.f / (float)p.cg;
  const int64_t stride = (int64_t)gridDim.x * t.rows * U;
  int64_t n0 = (int64_t)blockIdx.x * t.rows * U;
  const T* x_at = static_cast<const T*>(p.x) + (n0 + t.row) * p.xs[0] + t.c;
  const T* dy_at = static_cast<const T*>(p.dy) + (n0 + t.row) * p.ds[0] + t.c;
  T* dx_at = static_cast<T*>(p.dx) + (n0 + t.row) * p.C + t.c;
  int64_t st_at = (n0 + t.row) * p.G + t.g;
  const int64_t px = t.rows * p.xs[0], pd = t.rows * p.ds[0], po = t.rows * p.C, ps = t.rows * p.G;
  typename Q::Raw nx[U][K], ny[U][K];   // loads in flight; dy = 0 where there is nothing adds nothing
  float2 nst[U];
  auto fetch = [&](int64_t at, auto whole) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = decltype(whole)::value || at + u * t.rows + t.row < p.N;
      nst[u] = (kFull || t.g < p.G) && live
                   ? make_float2(__ldg(p.mean_in + st_at + u * ps), __ldg(p.rstd_in + st_at + u * ps))
                   : dup(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const bool in = (kFull || t.in[k]) && live;
        nx[u][k] = in ? Q::raw(x_at + u * px + k * t.step) : Q::none();
        ny[u][k] = in ? Q::raw(dy_at + u * pd + k * t.step) : Q::none();
      }
    }
    x_at += gridDim.x * (U * px);
    dy_at += gridDim.x * (U * pd);
    st_at += gridDim.x * (U * ps);
  };
  auto fetch_any = [&](int64_t at) {
    if (at + U * t.rows <= p.N) fetch(at, std::true_type());
    else fetch(at, std::false_type());
  };
  auto work = [&](auto whole) {
    float2 x[U][K][Q::P], q[U][K][Q::P];
    float rstd[U], mean[U], sums[2 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mean[u] = nst[u].x;
      rstd[u] = nst[u].y;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Q::unpack(nx[u][k], x[u][k]);
        Q::unpack(ny[u][k], q[u][k]);
      }
    }
    fetch_any(n0 + stride);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 s = make_float2(0.f, 0.f), sx = s;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < Q::P; ++e) {
          const float2 xh = fp::mul2(minus2<V>(x[u][k][e], mean[u]), dup(rstd[u]));
          const float2 dz = times_act_grad2<kSilu>(q[u][k][e], fp::fma2(xh, w[k][e], bias[k][e]));
          db[k][e] = fp::add2(db[k][e], dz);
          dw[k][e] = fp::fma2(dz, xh, dw[k][e]);
          x[u][k][e] = xh;
          q[u][k][e] = fp::mul2(dz, w[k][e]);
          s = fp::add2(s, q[u][k][e]);
          sx = fp::fma2(q[u][k][e], xh, sx);
        }
      sums[2 * u] = s.x + s.y;
      sums[2 * u + 1] = sx.x + sx.y;
    }
    group_sum<kBlock>(sums, lanes, part, phase);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool live = decltype(whole)::value || n0 + u * t.rows + t.row < p.N;
      const float2 ms = dup(-sums[2 * u] * inv), mx = dup(-sums[2 * u + 1] * inv);
#pragma unroll
      for (int k = 0; k < K; ++k) {
#pragma unroll
        for (int e = 0; e < Q::P; ++e)
          x[u][k][e] = fp::mul2(dup(rstd[u]), fp::fma2(x[u][k][e], mx, fp::add2(q[u][k][e], ms)));
        T* to = dx_at + u * po + k * t.step;
        if ((kFull || t.in[k]) && live &&
            SSD_INDEX_OK(p.hdr, (to - static_cast<T*>(p.dx)) + V - 1, p.N * p.C, 72))
          Q::store(to, x[u][k]);
      }
    }
    dx_at += gridDim.x * (U * po);
  };
  fetch_any(n0);
  for (; n0 < p.N; n0 += stride) {
    if (n0 + U * t.rows <= p.N) work(std::true_type());
    else work(std::false_type());
  }
  if (p.part_rows == 0) return;
  __shared__ float4 rows[kThreads][Q::P];   // the block's rows of samples joined, one partial a block
  const int slots = (int)min((int64_t)kThreads, p.G * lanes);   // threads of one row
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (!kBlock && t.rows > 1) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < Q::P; ++e) rows[threadIdx.x][e] = make_float4(dw[k][e].x, dw[k][e].y, db[k][e].x, db[k][e].y);
      __syncthreads();
      if (t.row > 0) continue;
      for (int r = 1; r < t.rows; ++r) {
#pragma unroll
        for (int e = 0; e < Q::P; ++e) {
          const float4 v = rows[threadIdx.x + r * slots][e];
          dw[k][e] = fp::add2(dw[k][e], make_float2(v.x, v.y));
          db[k][e] = fp::add2(db[k][e], make_float2(v.z, v.w));
        }
      }
    }
    const int64_t at = (int64_t)blockIdx.x * p.C + t.c + k * t.step;
    if (!t.in[k] || !SSD_INDEX_OK(p.hdr, at + V - 1, p.part_rows * p.C, 73)) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      p.part_w[at + e] = e % 2 ? dw[k][e / 2].y : dw[k][e / 2].x;
      p.part_b[at + e] = e % 2 ? db[k][e / 2].y : db[k][e / 2].x;
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Groups that no wide vector divides (an odd number of channels, say): a thread still takes 16 bytes of a
// row, which then hold the end of one group (`low`, its first `split` values) and the start of the
// next (`high`); a group is never narrower than a vector.  A block takes whole groups, V of them or a
// multiple, so that its channels are whole vectors too.  Every thread leaves its two partial sums in
// shared memory, and a thread a group adds the few of its group.
// 23795 x 520 bf16 in groups of 13: forward 37 us, backward 42 us (value by value 55 and 82); bound by the
// two joins' barriers of every few samples.
// ------------------------------------------------------------------------------------------------
template <int V>
struct StraddleSlot {
  int64_t c;                         // the thread's first channel
  int64_t g0;                        // the tile's first group
  int groups, cols, rows, row, col;  // groups and vectors of a full tile's row, rows of a block
  int low, split;                    // the group of its first value (within the tile), how many are in it
  bool in, two;
  __device__ __forceinline__ StraddleSlot(const NormParams& p) {
    const int cg = (int)p.cg;
    groups = (int)min(p.G, (int64_t)p.tile_groups);
    cols = groups * cg / V;
    rows = kThreads / cols;
    row = threadIdx.x / cols;
    col = threadIdx.x % cols;
    g0 = (int64_t)blockIdx.y * p.tile_groups;
    const int here = (int)min((int64_t)groups, p.G - g0);   // groups of this tile
    in = row < rows && col * V < here * cg;
    c = g0 * p.cg + col * V;
    low = col * V / cg;
    split = (low + 1) * cg - col * V;
    two = split < V;
  }
  // value pair e belongs to: x and y of (low's, high's)
  __device__ __forceinline__ float2 pick(int e, float lo, float hi) const {
    return make_float2(2 * e < split ? lo : hi, 2 * e + 1 < split ? lo : hi);
  }
};
// Adds the partial sums of group q % groups of row q / groups: `at(v)` is vector v's (low, high) sum.
template <int V, typename F>
__device__ __forceinline__ float2 straddle_sum(int cg, int g, F at) {
  const int first = g * cg / V, last = (g * cg + cg - 1) / V;
  float2 s = at(first, first * V < g * cg);
  for (int v = first + 1; v <= last; ++v) s = fp::add2(s, at(v, false));
  return s;
}

template <typename T, bool kSilu>
__global__ void __launch_bounds__(kThreads, 2) norm_straddle_forward_kernel(NormParams p) {
  constexpr int V = 16 / (int)sizeof(T), P = V / 2, U = 4;
  using Q = Pack<T, V>;
  __shared__ float2 part[U][kThreads];   // (low, high) of every thread
  __shared__ float stat[U][kThreads];    // of every group of every row
  const StraddleSlot<V> t(p);
  const int cg = (int)p.cg, teams = t.rows * t.groups;
  float2 w[P], bias[P];
  Q::zero(w);
  Q::zero(bias);
  if (t.in) {
    Q::param(p.w, t.c, 1.f, w);
    Q::param(p.bias, t.c, 0.f, bias);
  }
  const float inv = 1.f / (float)p.cg;
  const int64_t stride = (int64_t)gridDim.x * t.rows * U;
  const int mine = t.row * t.groups + t.low;   // where this thread's statistics lie
  typename Q::Raw next[U];
  auto fetch = [&](int64_t n0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u * t.rows + t.row;
      next[u] = t.in && n < p.N ? Q::raw(static_cast<const T*>(p.x) + n * p.xs[0] + t.c) : Q::none();
    }
  };
  // every group's sum of `part`, into stat
  auto join = [&](auto finish) {
    __syncthreads();
    for (int q = threadIdx.x; q < teams * U; q += kThreads) {
      const int u = q / teams, k = q % teams, row = k / t.groups, g = k % t.groups;
      const float2* s = part[u] + row * t.cols;
      stat[u][k] = finish(straddle_sum<V>(cg, g, [&](int v, bool high) {
                     return make_float2(high ? s[v].y : s[v].x, 0.f);
                   }).x);
    }
    __syncthreads();
  };
  int64_t n0 = (int64_t)blockIdx.x * t.rows * U;
  fetch(n0);
  for (; n0 < p.N; n0 += stride) {
    float2 x[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Q::unpack(next[u], x[u]);
      float lo = 0.f, hi = 0.f;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        if (2 * e < t.split) lo += x[u][e].x; else hi += x[u][e].x;
        if (2 * e + 1 < t.split) lo += x[u][e].y; else hi += x[u][e].y;
      }
      part[u][threadIdx.x] = make_float2(lo, hi);
    }
    fetch(n0 + stride);
    join([&](float s) { return s * inv; });
    float mean_lo[U], mean_hi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float ml = t.in ? stat[u][mine] : 0.f, mh = t.in && t.two ? stat[u][mine + 1] : 0.f;
      mean_lo[u] = ml;
      mean_hi[u] = mh;
      float lo = 0.f, hi = 0.f;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 m = t.pick(e, -ml, -mh);
        x[u][e] = fp::add2(x[u][e], m);
        const float2 q = fp::mul2(x[u][e], x[u][e]);
        if (2 * e < t.split) lo += q.x; else hi += q.x;
        if (2 * e + 1 < t.split) lo += q.y; else hi += q.y;
      }
      part[u][threadIdx.x] = make_float2(lo, hi);
    }
    join([&](float s) { return rsqrtf(fmaf(s, inv, p.eps)); });
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u * t.rows + t.row;
      const float rl = t.in ? stat[u][mine] : 0.f, rh = t.in && t.two ? stat[u][mine + 1] : 0.f;
#pragma unroll
      for (int e = 0; e < P; ++e)
        x[u][e] = act2<kSilu>(fp::fma2(fp::mul2(x[u][e], t.pick(e, rl, rh)), w[e], bias[e]));
      const int64_t at = n * p.C + t.c;
      if (t.in && n < p.N && SSD_INDEX_OK(p.hdr, at + V - 1, p.N * p.C, 86))
        Q::store(static_cast<T*>(p.y) + at, x[u]);
      // the thread that holds a group's first value writes its statistics
      if (p.mean && t.in && n < p.N && t.col * V == t.low * cg &&
          SSD_INDEX_OK(p.hdr, n * p.G + t.g0 + t.low, p.N * p.G, 87)) {
        p.mean[n * p.G + t.g0 + t.low] = mean_lo[u];
        p.rstd[n * p.G + t.g0 + t.low] = rl;
      }
      if (p.mean && t.in && n < p.N && t.two && SSD_INDEX_OK(p.hdr, n * p.G + t.g0 + t.low + 1, p.N * p.G, 87)) {
        p.mean[n * p.G + t.g0 + t.low + 1] = mean_hi[u];
        p.rstd[n * p.G + t.g0 + t.low + 1] = rh;
      }
    }
    __syncthreads();   // stat and part are written again
  }
}

template <typename T, bool kSilu>
__global__ void __launch_bounds__(kThreads, 2) norm_straddle_backward_kernel(NormParams p) {
  constexpr int V = 16 / (int)sizeof(T), P = V / 2, U = 2;
  using Q = Pack<T, V>;
  __shared__ float4 part[U][kThreads];   // (low q, low q xhat, high q, high q xhat) of every thread
  __shared__ float2 stat[U][kThreads];
  follow();
  const StraddleSlot<V> t(p);
  const int cg = (int)p.cg, teams = t.rows * t.groups;
  float2 w[P], bias[P], dw[P], db[P];
  Q::zero(w);
  Q::zero(bias);
  Q::zero(dw);
  Q::zero(db);
  if (t.in) {
    Q::param(p.w, t.c, 1.f, w);
    Q::param(p.bias, t.c, 0.f, bias);
  }
  const float inv = 1.f / (float)p.cg;
  const int64_t stride = (int64_t)gridDim.x * t.rows * U;
  const int mine = t.row * t.groups + t.low;
  typename Q::Raw nx[U], ny[U];
  float4 nst[U];   // mean and rstd of the two groups
  auto fetch = [&](int64_t n0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u * t.rows + t.row;
      const bool live = t.in && n < p.N;
      nx[u] = live ? Q::raw(static_cast<const T*>(p.x) + n * p.xs[0] + t.c) : Q::none();
      ny[u] = live ? Q::raw(static_cast<const T*>(p.dy) + n * p.ds[0] + t.c) : Q::none();
      const int64_t at = n * p.G + t.g0 + t.low;
      nst[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (live) nst[u].x = __ldg(p.mean_in + at), nst[u].y = __ldg(p.rstd_in + at);
      if (live && t.two) nst[u].z = __ldg(p.mean_in + at + 1), nst[u].w = __ldg(p.rstd_in + at + 1);
    }
  };
  int64_t n0 = (int64_t)blockIdx.x * t.rows * U;
  fetch(n0);
  for (; n0 < p.N; n0 += stride) {
    float2 x[U][P], q[U][P];
    float4 st[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Q::unpack(nx[u], x[u]);
      Q::unpack(ny[u], q[u]);
      st[u] = nst[u];
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 xh = fp::mul2(fp::add2(x[u][e], t.pick(e, -st[u].x, -st[u].z)), t.pick(e, st[u].y, st[u].w));
        const float2 dz = times_act_grad2<kSilu>(q[u][e], fp::fma2(xh, w[e], bias[e]));
        db[e] = fp::add2(db[e], dz);
        dw[e] = fp::fma2(dz, xh, dw[e]);
        x[u][e] = xh;
        q[u][e] = fp::mul2(dz, w[e]);
        const float2 qx = fp::mul2(q[u][e], xh);
        if (2 * e < t.split) s.x += q[u][e].x, s.y += qx.x; else s.z += q[u][e].x, s.w += qx.x;
        if (2 * e + 1 < t.split) s.x += q[u][e].y, s.y += qx.y; else s.z += q[u][e].y, s.w += qx.y;
      }
      part[u][threadIdx.x] = s;
    }
    fetch(n0 + stride);
    __syncthreads();
    for (int k = threadIdx.x; k < teams * U; k += kThreads) {
      const int u = k / teams, at = k % teams, row = at / t.groups, g = at % t.groups;
      const float4* s = part[u] + row * t.cols;
      const float2 v = straddle_sum<V>(cg, g, [&](int c, bool high) {
        return high ? make_float2(s[c].z, s[c].w) : make_float2(s[c].x, s[c].y);
      });
      stat[u][at] = make_float2(-v.x * inv, -v.y * inv);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t n = n0 + u * t.rows + t.row;
      const float2 a = t.in ? stat[u][mine] : make_float2(0.f, 0.f);
      const float2 b = t.in && t.two ? stat[u][mine + 1] : make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < P; ++e)
        x[u][e] = fp::mul2(t.pick(e, st[u].y, st[u].w),
                           fp::fma2(x[u][e], t.pick(e, a.y, b.y), fp::add2(q[u][e], t.pick(e, a.x, b.x))));
      const int64_t at = n * p.C + t.c;
      if (t.in && n < p.N && SSD_INDEX_OK(p.hdr, at + V - 1, p.N * p.C, 88))
        Q::store(static_cast<T*>(p.dx) + at, x[u]);
    }
    __syncthreads();
  }
  if (p.part_rows == 0) return;
  __shared__ float4 rows[kThreads][P];   // the block's rows joined, one partial a block
#pragma unroll
  for (int e = 0; e < P; ++e) rows[threadIdx.x][e] = make_float4(dw[e].x, dw[e].y, db[e].x, db[e].y);
  __syncthreads();
  if (t.row > 0 || !t.in) return;
  const int64_t at = (int64_t)blockIdx.x * p.C + t.c;
  if (!SSD_INDEX_OK(p.hdr, at + V - 1, p.part_rows * p.C, 89)) return;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    float4 s = rows[threadIdx.x][e];
    for (int r = 1; r < t.rows; ++r) {
      const float4 v = rows[r * t.cols + t.col][e];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    p.part_w[at + 2 * e] = s.x;
    p.part_w[at + 2 * e + 1] = s.y;
    p.part_b[at + 2 * e] = s.z;
    p.part_b[at + 2 * e + 1] = s.w;
  }
}

template <typename T, int V, int K, bool kBlock, bool kSilu>
cudaError_t launch_tokens(NormParams p, bool backward, cudaStream_t st) {
  constexpr int UF = K == 1 ? 4 : K == 2 ? 2 : 1, UB = K == 1 ? 2 : 1;   // samples in flight
  const int64_t gv = p.cg / V;
  p.lanes = 1;
  while (!kBlock && p.lanes < 32 && p.lanes * K < gv) p.lanes *= 2;
  const int64_t slots = p.G * p.lanes;
  const int64_t rows = kBlock || slots >= kThreads ? 1 : kThreads / slots;
  const int64_t by = kBlock ? p.G : (slots + kThreads - 1) / kThreads;
  // exact fits of the common kind have a form without checks
  constexpr bool kHasFull = K == 1 && !kBlock && V > 1;
  const bool full = kHasFull && gv == p.lanes && (slots >= kThreads ? slots % kThreads : kThreads % slots) == 0;
  const int U = backward ? UB : UF;
  auto* fwd = full ? norm_token_forward_kernel<T, V, K, UF, kBlock, kSilu, kHasFull>
                   : norm_token_forward_kernel<T, V, K, UF, kBlock, kSilu, false>;
  auto* bwd = full ? norm_token_backward_kernel<T, V, K, UB, kBlock, kSilu, kHasFull>
                   : norm_token_backward_kernel<T, V, K, UB, kBlock, kSilu, false>;
  auto* kernel = backward ? bwd : fwd;
  int blocks = 0;
  cudaError_t e = resident_blocks(kernel, kThreads, 0, &blocks);
  if (e != cudaSuccess) return e;
  if (backward) blocks = std::min(blocks, kTokenBlocks);
  const int64_t steps = (p.N + rows * U - 1) / (rows * U);
  const int64_t bx = std::min<int64_t>(steps, std::max<int64_t>(1, blocks / by));
  p.part_rows = backward && (p.dw || p.db) ? bx : 0;
  kernel<<<dim3((unsigned)bx, (unsigned)by), kThreads, 0, st>>>(p);
  e = cudaGetLastError();
  return e == cudaSuccess && backward ? launch_param_grad(p, st) : e;
}

template <typename T, int V, bool kSilu>
cudaError_t run(const NormParams& p, bool backward, cudaStream_t st) {
  const int64_t gv = p.cg / V;
  if (gv <= 32) return launch_tokens<T, V, 1, false, kSilu>(p, backward, st);
  if (gv <= 64) return launch_tokens<T, V, 2, false, kSilu>(p, backward, st);
  if (gv <= 128) return launch_tokens<T, V, 4, false, kSilu>(p, backward, st);
  if (gv <= 256) return launch_tokens<T, V, 1, true, kSilu>(p, backward, st);
  if (gv <= 512) return launch_tokens<T, V, 2, true, kSilu>(p, backward, st);
  return launch_tokens<T, V, 4, true, kSilu>(p, backward, st);
}

template <typename T, bool kSilu>
cudaError_t run_straddle_as(NormParams p, bool backward, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T), kFwd = 4, kBwd = 2;   // samples of a row of threads in flight
  p.tile_groups = (int32_t)(kThreads / p.cg * V);
  const int64_t groups = std::min<int64_t>(p.G, p.tile_groups), rows = kThreads / (groups * p.cg / V);
  const int64_t by = (p.G + p.tile_groups - 1) / p.tile_groups;
  auto* kernel = backward ? norm_straddle_backward_kernel<T, kSilu> : norm_straddle_forward_kernel<T, kSilu>;
  int blocks = 0;
  cudaError_t e = resident_blocks(kernel, kThreads, 0, &blocks);
  if (e != cudaSuccess) return e;
  if (backward) blocks = std::min(blocks, kTokenBlocks);
  const int64_t per = rows * (backward ? kBwd : kFwd), steps = (p.N + per - 1) / per;
  const int64_t bx = std::min<int64_t>(steps, std::max<int64_t>(1, blocks / by));
  p.part_rows = backward && (p.dw || p.db) ? bx : 0;
  kernel<<<dim3((unsigned)bx, (unsigned)by), kThreads, 0, st>>>(p);
  e = cudaGetLastError();
  return e == cudaSuccess && backward ? launch_param_grad(p, st) : e;
}

}  // namespace

template <typename T>
cudaError_t run_straddle(const NormParams& p, bool backward, cudaStream_t st) {
  return p.act == SSD_ACT_SILU ? run_straddle_as<T, true>(p, backward, st) : run_straddle_as<T, false>(p, backward, st);
}

template <typename T, int V>
cudaError_t run_tokens(const NormParams& p, bool backward, cudaStream_t st) {
  return p.act == SSD_ACT_SILU ? run<T, V, true>(p, backward, st) : run<T, V, false>(p, backward, st);
}
#if NORM_TOKENS_F32
template cudaError_t run_straddle<float>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<float, 4>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<float, 2>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<float, 1>(const NormParams&, bool, cudaStream_t);
#else
template cudaError_t run_straddle<__nv_bfloat16>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<__nv_bfloat16, 8>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<__nv_bfloat16, 4>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<__nv_bfloat16, 2>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<__nv_bfloat16, 1>(const NormParams&, bool, cudaStream_t);
#endif

}  // namespace norm
}  // namespace ssd
