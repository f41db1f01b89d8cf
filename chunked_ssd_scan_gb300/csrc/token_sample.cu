// Drawing of tokens (declaration in include/ssdscan.h): temperature, top-k, min-p, top-p and the inverse of the running
// sum at a given random number, one block a row.
// A choice hangs on sums over the whole vocabulary, next to which the border between two tokens is at times 1e-6 wide:
// fp32 sums would draw another token in one row of a few hundred, and in another order another one.  So weights are
// fixed-point numbers, 2^s for the largest logit with V 2^s <= 2^62, and their sums are exact in any order.  A weight is
// 2^-t with t = (largest - logit) log2(e) / temperature carried as two floats (fp64 would take 44 us for one addition per
// value of 512 x 50000), its fraction as 32 bits, and a polynomial in 32-bit integers (a fit of degree 8; it is off by
// at most 3 units of 2^-31).
#include <math.h>
#include <string.h>

#include "pack.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 1024;      // of the logits below the largest, over the range in which weights are not zero
constexpr int kList = 1024;      // tokens of one bin that are searched in shared memory
constexpr float kNegInf = -INFINITY;

struct SampleParams {
  const void* logits;
  const float *u, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int64_t* ids;
  float* logprob;
  int64_t rows, stride;
  int32_t V, top_k_all, shift;   // weights are 2^shift for the largest logit
  float temperature_all, top_p_all, min_p_all;
};

// The weight of a logit.
struct Weight {
  float most, ch, cl;   // largest logit; log2(e) / temperature in two parts
  int shift;
  __device__ __forceinline__ uint64_t operator()(float x) const {
    if (x == most) return 1ull << shift;
    const float d = most - x;
    const float ph = d * ch;
    if (!(ph < 62.5f)) return 0;   // also an infinite largest logit, and NaN of -inf at an infinite temperature
    const float back = d - most, dl = (most - (d - back)) - (x + back);   // what d's rounding left
    const float pl = fmaf(d, ch, -ph) + fmaf(d, cl, dl * ch);
    const float whole = truncf(ph);
    // fraction in units of 2^-32, the small part added as an integer
    int64_t t = (int64_t)(((uint64_t)(uint32_t)whole << 32) + __float2uint_rz((ph - whole) * 4294967296.f));
    t += __float2ll_rn(pl * 4294967296.f);
    t = t < 0 ? 0 : t;
    const uint32_t f = (uint32_t)t, n = (uint32_t)(t >> 32);
    uint32_t m = 0x7ddu;
    m = 0x7a43u - __umulhi(f, m);
    m = 0x50690u - __umulhi(f, m);
    m = 0x2badc5u - __umulhi(f, m);
    m = 0x13b299cu - __umulhi(f, m);
    m = 0x71ac1ffu - __umulhi(f, m);
    m = 0x1ebfbdfau - __umulhi(f, m);
    m = 0x58b90bfcu - __umulhi(f, m);
    m = 0x80000000u - __umulhi(f, m);
    return n > 62 ? 0 : ((uint64_t)m << (shift - 31)) >> n;
  }
};

// Order of falling logits: larger keys first.  Equal logits have equal keys (-0 counts as 0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// f(index, logit) for the tokens [begin, end) of a row, spread over `threads` of which this is `t`.  NaN is -inf.
template <typename T, typename F>
__device__ __forceinline__ void for_tokens(const T* row, int begin, int end, int t, int threads, const F& f) {
  constexpr int W = 16 / (int)sizeof(T);
  auto one = [&](int i, float x) { f(i, x != x ? kNegInf : x); };
  // from the first 16-byte border on by vectors, four on their way at once
  const int lead = min(end - begin, (int)((16 - (reinterpret_cast<uintptr_t>(row + begin) & 15)) & 15) / (int)sizeof(T));
  for (int i = begin + t; i < begin + lead; i += threads) one(i, ld_f32(row + i));
  const int start = begin + lead, nvec = (end - start) / W;
  int v = t;
  for (; v + 3 * threads < nvec; v += 4 * threads) {
    typename Pack<T, W>::Raw r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = Pack<T, W>::raw(row + start + (int64_t)(v + k * threads) * W);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 x[W / 2];
      Pack<T, W>::unpack(r[k], x);
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        one(start + (v + k * threads) * W + 2 * j, x[j].x);
        one(start + (v + k * threads) * W + 2 * j + 1, x[j].y);
      }
    }
  }
  for (; v < nvec; v += threads) {
    float2 x[W / 2];
    Pack<T, W>::unpack(Pack<T, W>::raw(row + start + (int64_t)v * W), x);
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      one(start + v * W + 2 * j, x[j].x);
      one(start + v * W + 2 * j + 1, x[j].y);
    }
  }
  for (int i = start + nvec * W + t; i < end; i += threads) one(i, ld_f32(row + i));
}

struct SampleSmem {
  uint64_t part[kWarps];
  uint32_t count[kBins], low[kBins], high[kBins];   // of a bin: tokens, sum of weights
  uint32_t list_key[kList];
  int32_t list_id[kList];
  uint64_t list_w[kList];
  uint64_t out[4];
  int32_t listed;
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t block_sum(SampleSmem& sm, uint64_t v) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.part[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(sm.part[threadIdx.x & 31]);
}
// Number of the first of 32 warps' sums whose running sum exceeds `target`, and the sum before it.
__device__ __forceinline__ int pick_warp(SampleSmem& sm, uint64_t mine, uint64_t target, uint64_t* before) {
  mine = warp_sum(mine);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.part[threadIdx.x >> 5] = mine;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const uint64_t own = sm.part[lane];
  uint64_t upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  const uint32_t past = __ballot_sync(0xffffffffu, upto > target);
  const int at = past ? __ffs(past) - 1 : 31;
  *before = __shfl_sync(0xffffffffu, upto - own, at);
  return at;
}

// What a row keeps: tokens whose key is above `key`, and those of that key up to index `last`; of these the ones with a
// weight of at least `least` (min_p).
struct Cut {
  uint32_t key;
  int32_t last;
  uint64_t least;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= last); }
  __device__ __forceinline__ uint64_t of(uint64_t w) const { return w >= least ? w : 0; }
};

__device__ __forceinline__ int bin_of(const Weight& w, float inv, float x) {
  const float d = (w.most - x) * inv;
  return x == w.most ? 0 : d < (float)(kBins - 1) ? (int)d : kBins - 1;   // NaN (of infinities): the last
}

// The first token, in falling order, at which the running count (kMass: the running sum of weights) of what `have` keeps
// reaches `want` >= 1; all of `have` where it never does.  With kMass *sum is the weights' sum up to it on return.
// (A count takes no account of min_p: what that leaves is a beginning of the same order.)
template <bool kMass, typename T>
__device__ Cut find_cut(SampleSmem& sm, const T* row, int V, const Weight& w, float inv, const Cut& have, uint64_t want,
                        uint64_t* sum) {
  const int tid = threadIdx.x, lane = tid & 31;
  __syncthreads();
  sm.count[tid] = 0;
  sm.low[tid] = sm.high[tid] = 0;
  if (tid == 0) sm.listed = 0;
  __syncthreads();
  for_tokens(row, 0, V, tid, kThreads, [&](int i, float x) {
    if (x == kNegInf || !have.keeps(key_of(x), i)) return;
    const int b = bin_of(w, inv, x);
    if constexpr (kMass) {
      const uint64_t m = have.of(w(x));
      if (m) {
        // in two halves (a 64-bit addition in shared memory is a loop): the lower one's carry goes with the upper
        const uint32_t lo = (uint32_t)m, old = atomicAdd(&sm.low[b], lo), up = (uint32_t)(m >> 32) + (old + lo < lo);
        if (up) atomicAdd(&sm.high[b], up);
        atomicAdd(&sm.count[b], 1u);
      }
    } else {
      atomicAdd(&sm.count[b], 1u);
    }
  });
  __syncthreads();
  // the bin in which it happens: sums over 32 bins by warp, then within
  uint64_t before;
  const uint64_t mine = kMass ? (uint64_t)sm.high[tid] << 32 | sm.low[tid] : sm.count[tid];
  const int warp = pick_warp(sm, mine, want - 1, &before);
  if ((tid >> 5) == warp) {
    uint64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto >= want);
    const int at = past ? __ffs(past) - 1 : 31;
    if (lane == at) {
      sm.out[0] = past ? (uint64_t)tid : kBins;
      sm.out[1] = want - (before + upto - mine);   // still wanted within the bin
      sm.out[2] = before + upto - mine;
    }
  }
  __syncthreads();
  const int bin = (int)sm.out[0];
  if (bin == kBins) {
    if (kMass) *sum = block_sum(sm, mine);
    return have;
  }
  const uint64_t rest = sm.out[1], base = sm.out[2];
  const uint32_t n = sm.count[bin];
  auto in_bin = [&](int i, float x, uint32_t& k) {
    if (x == kNegInf || bin_of(w, inv, x) != bin) return false;
    k = key_of(x);
    return have.keeps(k, i) && (!kMass || have.of(w(x)) != 0);
  };
  if (n <= kList) {   // every one of the bin's tokens counts those before it
    for_tokens(row, 0, V, tid, kThreads, [&](int i, float x) {
      uint32_t k;
      if (!in_bin(i, x, k)) return;
      const int at = atomicAdd(&sm.listed, 1);
      sm.list_key[at] = k;
      sm.list_id[at] = i;
      if (kMass) sm.list_w[at] = w(x);
    });
    __syncthreads();
    if (tid < (int)n) {
      const uint32_t k = sm.list_key[tid];
      const int id = sm.list_id[tid];
      const uint64_t own = kMass ? sm.list_w[tid] : 1;
      uint64_t above = 0;
      for (int j = 0; j < (int)n; ++j) {
        const uint32_t kj = sm.list_key[j];
        if (kj > k || (kj == k && sm.list_id[j] < id)) above += kMass ? sm.list_w[j] : 1;
      }
      if (above < rest && above + own >= rest) {
        sm.out[0] = k;
        sm.out[1] = (uint64_t)(uint32_t)id;
        sm.out[3] = base + above + own;
      }
    }
    __syncthreads();
    if (kMass) *sum = sm.out[3];
    return {(uint32_t)sm.out[0], (int32_t)(uint32_t)sm.out[1], have.least};
  }
  // more than fit (many equal logits): by bisection of their keys, a pass over the row a step
  uint32_t lo = 0xffffffffu, hi = 0;
  for_tokens(row, 0, V, tid, kThreads, [&](int i, float x) {
    uint32_t k;
    if (!in_bin(i, x, k)) return;
    lo = min(lo, k);
    hi = max(hi, k);
  });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  __syncthreads();
  if (lane == 0) sm.part[tid >> 5] = (uint64_t)hi << 32 | lo;
  __syncthreads();
  const uint64_t pair = sm.part[lane];
  lo = __reduce_min_sync(0xffffffffu, (uint32_t)pair);
  hi = __reduce_max_sync(0xffffffffu, (uint32_t)(pair >> 32));
  auto value_of = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); };
  auto summed = [&](auto&& f) {   // the sum of f(key, index) over the bin's tokens
    uint64_t s = 0;
    for_tokens(row, 0, V, tid, kThreads, [&](int i, float x) {
      uint32_t k;
      if (in_bin(i, x, k)) s += f(k, i);
    });
    return block_sum(sm, s);
  };
  // the largest key with count (sum) of keys >= it at least `rest`
  while (lo < hi) {
    const uint32_t mid = lo + (hi - lo) / 2 + 1;
    if (summed([&](uint32_t k, int) { return k >= mid ? kMass ? w(value_of(k)) : 1 : 0; }) >= rest) lo = mid;
    else hi = mid - 1;
  }
  const uint64_t above = summed([&](uint32_t k, int) { return k > lo ? kMass ? w(value_of(k)) : 1 : 0; });
  const uint64_t ties = summed([&](uint32_t k, int) { return k == lo ? 1ull : 0ull; });
  const uint64_t each = kMass ? w(value_of(lo)) : 1;
  const uint64_t need = min((rest - above + each - 1) / each, ties);   // of the equal ones, >= 1
  if (kMass) *sum = base + above + need * each;
  int from = 0, to = V - 1;   // the smallest index with `need` of the equal ones up to it
  while (from < to) {
    const int mid = from + (to - from) / 2;
    if (summed([&](uint32_t k, int i) { return k == lo && i <= mid ? 1ull : 0ull; }) >= need) to = mid;
    else from = mid + 1;
  }
  return {lo, from, have.least};
}

__device__ __forceinline__ uint64_t fixed64(float v) {   // v in [0, 1) as v 2^64
  return __float2ull_rz(v * 18446744073709551616.f);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) token_sample_kernel(const __grid_constant__ SampleParams p) {
  __shared__ SampleSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = p.V;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const T* row = static_cast<const T*>(p.logits) + r * p.stride;
    float temp = p.temperature ? __ldg(p.temperature + r) : p.temperature_all;
    const float top_p = p.top_p ? __ldg(p.top_p + r) : p.top_p_all;
    float min_p = p.min_p ? __ldg(p.min_p + r) : p.min_p_all;
    const int32_t top_k = p.top_k ? __ldg(p.top_k + r) : p.top_k_all;
    if (!(temp >= 0.f)) temp = 1.f;
    const bool by_sum = top_p < 1.f;   // not for NaN
    if (!(min_p > 0.f)) min_p = 0.f;
    // the largest logit and its first index
    uint64_t best = 0;
    for_tokens(row, 0, V, tid, kThreads, [&](int i, float x) {
      const uint64_t k = (uint64_t)key_of(x) << 32 | (uint32_t)~i;
      best = k > best ? k : best;
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t v = __shfl_xor_sync(0xffffffffu, best, o);
      best = v > best ? v : best;
    }
    __syncthreads();
    if (lane == 0) sm.part[warp] = best;
    __syncthreads();
    best = sm.part[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const uint64_t v = __shfl_xor_sync(0xffffffffu, best, o);
      best = v > best ? v : best;
    }
    const uint32_t top_key = (uint32_t)(best >> 32);
    Weight w;
    w.most = __uint_as_float(top_key & 0x80000000u ? top_key & 0x7fffffffu : ~top_key);
    if (w.most == kNegInf || temp == 0.f) {
      if (tid == 0) {
        p.ids[r] = w.most == kNegInf ? -1 : (int64_t)(uint32_t)~(uint32_t)best;
        if (p.logprob) p.logprob[r] = w.most == kNegInf ? NAN : 0.f;
      }
      continue;
    }
    // log2(e) / temperature in two floats: the quotient, and what its product with the temperature leaves
    const float tt = fmaxf(temp, 1e-30f);
    w.ch = 1.44269502f / tt;
    w.cl = (fmaf(-w.ch, tt, 1.44269502f) + 1.92596299e-8f) / tt;
    w.shift = p.shift;
    Cut cut = {0, V, 1};
    if (min_p > 0.f) {   // a bound on the weights, rounded up
      const uint64_t one = 1ull << w.shift, f = min_p < 1.f ? fixed64(min_p) : 0;
      const uint64_t least = __umul64hi(f, one) + (f * one ? 1 : 0);
      cut.least = min_p < 1.f ? (least ? least : 1) : one;
    }
    uint64_t total = 0;
    bool summed = false;
    const float inv = (float)kBins / 43.5f / tt;   // weights end at 2^-62.5 = e^-43.3
    if (top_k > 0 && top_k < V) cut = find_cut<false>(sm, row, V, w, inv, cut, (uint64_t)top_k, nullptr);
    if (by_sum) {
      uint64_t s = 0;
      for_tokens(row, 0, V, tid, kThreads, [&](int i, float x) { s += cut.keeps(key_of(x), i) ? cut.of(w(x)) : 0; });
      total = block_sum(sm, s);
      const uint64_t f = fixed64(fmaxf(top_p, 0.f));
      const uint64_t want = __umul64hi(f, total) + (f * total ? 1 : 0);   // p total, rounded up
      cut = find_cut<true>(sm, row, V, w, inv, cut, want ? want : 1, &total);
      summed = true;
    }
    // the draw: sums of 32 parts of the row by warp, of 32 parts of the chosen one, then token by token
    int begin = 0, end = V;
    uint64_t target = 0, before;
    for (int level = 0; level < 2; ++level) {
      const int len = ((end - begin + kWarps - 1) / kWarps + 7) / 8 * 8;
      const int b0 = min(end, begin + warp * len), b1 = min(end, b0 + len);
      uint64_t s = 0;
      for_tokens(row, b0, b1, lane, 32, [&](int i, float x) { s += cut.keeps(key_of(x), i) ? cut.of(w(x)) : 0; });
      if (level == 0) {
        if (!summed) total = block_sum(sm, s);
        const float u = __ldg(p.u + r);
        target = u >= 1.f ? total - 1 : u > 0.f ? __umul64hi(fixed64(u), total) : 0;
      }
      const int at = pick_warp(sm, s, target, &before);
      target -= before;
      end = min(end, begin + (at + 1) * len);
      begin = min(end, begin + at * len);
    }
    if (warp == 0) {
      int found = -1;
      for (int i0 = begin; i0 < end && found < 0; i0 += 32) {
        const int i = i0 + lane;
        float x = i < end ? ld_f32(row + i) : kNegInf;
        if (x != x) x = kNegInf;
        const uint64_t own = i < end && cut.keeps(key_of(x), i) ? cut.of(w(x)) : 0;
        uint64_t upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, upto > target);
        if (past) found = i0 + __ffs(past) - 1;
        target -= __shfl_sync(0xffffffffu, upto, 31);
      }
      if (lane == 0) {
        p.ids[r] = found;
        if (p.logprob) {
          const float x = found >= 0 ? ld_f32(row + found) : w.most;
          const float z = x == w.most ? 0.f : (x - w.most) / tt;
          // the sum is at least the largest weight: its logarithm by that of its 24 leading bits
          p.logprob[r] = z - logf((float)total * __uint_as_float((uint32_t)(127 - w.shift) << 23));
        }
      }
    }
  }
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" ssd_status token_sample(const token_sample_shape* shape, const void* logits, const float* u,
                                   const float* temperature, const int32_t* top_k, const float* top_p,
                                   const float* min_p, int64_t* ids, float* logprob, void* stream) {
  if (!shape || shape->rows < 0 || shape->vocab < 1 || shape->logits_stride < 0) return SSD_ERR_INVALID_ARG;
  if (shape->io_dtype != SSD_F32 && shape->io_dtype != SSD_BF16) return SSD_ERR_INVALID_ARG;
  if (shape->vocab > 1 << 20) return SSD_ERR_UNSUPPORTED;
  if (shape->rows == 0) return SSD_OK;
  const uintptr_t e = shape->io_dtype == SSD_BF16 ? 2 : 4;
  auto off = [](const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; };
  if (!logits || !u || !ids || off(logits, e) || off(u, 4) || off(temperature, 4) || off(top_k, 4) || off(top_p, 4) ||
      off(min_p, 4) || off(ids, 8) || off(logprob, 4))
    return SSD_ERR_INVALID_ARG;
  SampleParams p;
  memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.u = u;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.ids = ids;
  p.logprob = logprob;
  p.rows = shape->rows;
  p.stride = shape->logits_stride;
  p.V = (int32_t)shape->vocab;
  p.temperature_all = shape->temperature;
  p.top_k_all = shape->top_k;
  p.top_p_all = shape->top_p;
  p.min_p_all = shape->min_p;
  int bits = 0;
  while ((int64_t)1 << bits < shape->vocab) ++bits;
  p.shift = 62 - bits;
  const unsigned grid = (unsigned)(shape->rows < (1 << 20) ? shape->rows : 1 << 20);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (shape->io_dtype == SSD_BF16) token_sample_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p);
  else token_sample_kernel<float><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
