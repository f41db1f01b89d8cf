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

}  // namespace

template <typename T, int V>
cudaError_t run_tokens(const NormParams& p, bool backward, cudaStream_t st) {
  return p.act == SSD_ACT_SILU ? run<T, V, true>(p, backward, st) : run<T, V, false>(p, backward, st);
}
#if NORM_TOKENS_F32
template cudaError_t run_tokens<float, 4>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<float, 2>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<float, 1>(const NormParams&, bool, cudaStream_t);
#else
template cudaError_t run_tokens<__nv_bfloat16, 8>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<__nv_bfloat16, 4>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<__nv_bfloat16, 2>(const NormParams&, bool, cudaStream_t);
template cudaError_t run_tokens<__nv_bfloat16, 1>(const NormParams&, bool, cudaStream_t);
#endif

}  // namespace norm
}  // namespace ssd
