// Drawing of tokens (declaration in include/ssdscan.h): temperature, top-k, min-p, top-p and the inverse of the running
// sum at a given random number, a block a row, or up to eight (a cluster) where there are few rows.
// A choice hangs on sums over the whole vocabulary, next to which the border between two tokens is at times 1e-6 wide:
// fp32 sums would draw another token in one row of a few hundred, and in another order another one.  So weights are
// fixed-point numbers, 2^s for the largest logit with V 2^s <= 2^62, and their sums are exact in any order.  A weight is
// 2^-t with t = (largest - logit) log2(e) / temperature carried as two floats (fp64 would take 44 us for one addition per
// value of 512 x 50000): 256 values of 2^-j/256 as 32-bit integers, made by a polynomial (a fit of degree 8, off by at most
// 3 units of 2^-31), and what is left of the exponent, below 1/512, in fp32.  (A polynomial in integers for every weight,
// with its conversions, took three times as long.)
#include <cooperative_groups.h>
#include <math.h>
#include <string.h>

#include "pack.cuh"

namespace ssd {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBins = 1024;      // of the logits below the largest, over the range in which weights are not zero
constexpr int kTail = 384;       // the bin of weights of about 2^-23 of the largest
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

// 2^31 2^-f for a fraction of 32 bits.
__device__ __forceinline__ uint32_t exp2_fraction(uint32_t f) {
  uint32_t m = 0x7ddu;
  m = 0x7a43u - __umulhi(f, m);
  m = 0x50690u - __umulhi(f, m);
  m = 0x2badc5u - __umulhi(f, m);
  m = 0x13b299cu - __umulhi(f, m);
  m = 0x71ac1ffu - __umulhi(f, m);
  m = 0x1ebfbdfau - __umulhi(f, m);
  m = 0x58b90bfcu - __umulhi(f, m);
  return 0x80000000u - __umulhi(f, m);
}

__device__ __forceinline__ float exp2f_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// The weight of a logit.
struct Weight {
  const uint2* table;   // 2^31 2^-j/256 as an integer and as a float
  float half, ch, cl;   // half the largest logit; 2 log2(e) / temperature in two parts
  int shift;
  __device__ __forceinline__ uint64_t operator()(float x) const {   // without a branch
    // half the distance: two finite logits may lie further apart than the largest number
    const float d = fmaf(x, -0.5f, half);
    const float ph = d * ch;
    const float back = d - half, dl = (half - (d - back)) - fmaf(x, 0.5f, back);   // what d's rounding left
    const float pl = fmaf(d, ch, -ph) + fmaf(d, cl, dl * ch);
    // the nearest 256th, by an addition that leaves its number in the lowest bits
    const float at = fmaf(ph, 256.f, 12582912.f);
    const int k = __float_as_int(at) - 0x4b400000;
    const float a = -0.693147181f * (fmaf(at - 12582912.f, -1.f / 256.f, ph) + pl);
    const float g = fmaf(a * a, fmaf(a, 1.f / 6.f, 0.5f), a);   // e^a - 1, |a| < 0.0014
    const uint2 t = table[k & 255];
    const uint32_t m = t.x + (uint32_t)(__float_as_int(fmaf(__uint_as_float(t.y), g, 12582912.f)) - 0x4b400000);
    const uint64_t w = ((uint64_t)m << (shift - 31)) >> ((k >> 8) & 63);
    // nothing far below, beneath an infinite largest logit, or of -inf at an infinite temperature (NaN)
    return d > 0.f ? ph < 62.5f ? w : 0 : 1ull << shift;   // (of two infinite logits d is NaN)
  }
};

// Order of falling logits: larger keys first.  Equal logits have equal keys (-0 counts as 0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// f(index, logit) for the tokens [begin, end) of a row, spread over `threads` of which this is `t`.  NaN is -inf.  U vectors
// are on their way at once; one where f is long (its code is there W U times: with four of eight values, 1400
// instructions a pass, fetching them took most of the time).
template <int U, typename T, typename F>
__device__ __forceinline__ void for_tokens(const T* row, int begin, int end, int t, int threads, const F& f) {
  constexpr int W = 16 / (int)sizeof(T);
  auto one = [&](int i, float x) { f(i, x != x ? kNegInf : x); };
  // from the first 16-byte border on by vectors, four on their way at once
  const int lead = min(end - begin, (int)((16 - (reinterpret_cast<uintptr_t>(row + begin) & 15)) & 15) / (int)sizeof(T));
  for (int i = begin + t; i < begin + lead; i += threads) one(i, ld_f32(row + i));
  const int start = begin + lead, nvec = (end - start) / W;
  int v = t;
  auto vector = [&](const typename Pack<T, W>::Raw& r, int at) {
    float2 x[W / 2];
    Pack<T, W>::unpack(r, x);
#pragma unroll
    for (int j = 0; j < W / 2; ++j) {
      one(start + at * W + 2 * j, x[j].x);
      one(start + at * W + 2 * j + 1, x[j].y);
    }
  };
  if constexpr (U > 1) {
    for (; v + (U - 1) * threads < nvec; v += U * threads) {
      typename Pack<T, W>::Raw r[U];
#pragma unroll
      for (int k = 0; k < U; ++k) r[k] = Pack<T, W>::raw(row + start + (int64_t)(v + k * threads) * W);
#pragma unroll
      for (int k = 0; k < U; ++k) vector(r[k], v + k * threads);
    }
  }
  for (; v < nvec; v += threads) vector(Pack<T, W>::raw(row + start + (int64_t)v * W), v);
  for (int i = start + nvec * W + t; i < end; i += threads) one(i, ld_f32(row + i));
}

struct SampleSmem {
  uint2 table[256];
  uint64_t part[kWarps];
  uint64_t of_block[2][8];
  uint32_t count[kBins], low[kBins], high[kBins];   // of a bin: tokens, sum of weights
  uint64_t list[kList], list_w[kList];   // (key, falling index) of a bin's tokens, and their weights
  uint64_t out[4];
  int32_t listed;
};

// The blocks of a row.  Each has a slice of the vocabulary; sums and choices are the same in all of them.
template <bool kMany>
struct Row {
  SampleSmem& sm;
  int rank, blocks;
  int turn;   // of of_block: a block may be a reduction ahead of another's reading
  __device__ __forceinline__ void sync() const {
    if constexpr (kMany) cg::this_cluster().sync();
    else __syncthreads();
  }
  __device__ __forceinline__ SampleSmem& of(int r) const {
    if constexpr (kMany) return *cg::this_cluster().map_shared_rank(&sm, r);
    else return sm;
  }
  // Every block's value to every block.
  __device__ __forceinline__ const uint64_t* exchange(uint64_t mine) {
    turn ^= 1;
    if (threadIdx.x < blocks) of(threadIdx.x).of_block[turn][rank] = mine;
    sync();
    return sm.of_block[turn];
  }
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
template <bool kMany>
__device__ __forceinline__ uint64_t row_sum(Row<kMany>& row, uint64_t v) {
  v = block_sum(row.sm, v);
  if constexpr (kMany) {
    const uint64_t* all = row.exchange(v);
    v = 0;
    for (int r = 0; r < row.blocks; ++r) v += all[r];
  }
  return v;
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
  const float d = fmaf(x, -0.5f, w.half), at = d * inv;
  return !(d > 0.f) ? 0 : at < (float)(kBins - 1) ? (int)at : kBins - 1;   // NaN (inf 0): the last
}

// The first token, in falling order, at which the running count of what `have` keeps reaches `want` >= 1 (kMass: the running
// sum of weights the share `want` 2^-64 of their sum); all of `have` where it never does.  With kMass *sum is the weights'
// sum up to it on return.  (A count takes no account of min_p: what that leaves is a beginning of the same order.)
// Most tokens weigh next to nothing: from kTail on their weights are summed in registers, and only if the cut should lie
// there, which takes a very flat row, they enter the bins in a second pass.
template <bool kMass, bool kMany, typename T>
__device__ Cut find_cut(Row<kMany>& all, const T* row, int begin, int end, int V, const Weight& w, float inv,
                        const Cut& have, uint64_t want, uint64_t* sum) {
  SampleSmem& sm = all.sm;
  const int tid = threadIdx.x, lane = tid & 31;
  __syncthreads();
  sm.count[tid] = 0;
  sm.low[tid] = sm.high[tid] = 0;
  if (tid == 0) sm.listed = 0;
  __syncthreads();
  uint64_t tail = 0;
  auto enter = [&](int b, uint64_t m) {
    // in two halves (a 64-bit addition in shared memory is a loop): the lower one's carry goes with the upper
    const uint32_t lo = (uint32_t)m, old = atomicAdd(&sm.low[b], lo), up = (uint32_t)(m >> 32) + (old + lo < lo);
    if (up) atomicAdd(&sm.high[b], up);
    atomicAdd(&sm.count[b], 1u);
  };
  for_tokens<1>(row, begin, end, tid, kThreads, [&](int i, float x) {
    if (x == kNegInf || !have.keeps(key_of(x), i)) return;
    const int b = bin_of(w, inv, x);
    if constexpr (kMass) {
      const uint64_t m = have.of(w(x));
      if (b >= kTail) tail += m;
      else if (m) enter(b, m);
    } else {
      atomicAdd(&sm.count[b], 1u);
    }
  });
  if constexpr (kMass) {
    tail = row_sum(all, tail);
    const uint64_t head = row_sum(all, (uint64_t)sm.high[tid] << 32 | sm.low[tid]);
    want = __umul64hi(want, head + tail) + (want * (head + tail) ? 1 : 0);   // the share, rounded up
    want = want ? want : 1;
    if (want > head)
      for_tokens<1>(row, begin, end, tid, kThreads, [&](int i, float x) {
        if (x == kNegInf || !have.keeps(key_of(x), i)) return;
        const int b = bin_of(w, inv, x);
        const uint64_t m = b >= kTail ? have.of(w(x)) : 0;
        if (m) enter(b, m);
      });
  }
  all.sync();
  // the bin in which it happens: sums over 32 bins by warp, then within
  uint64_t before, mine = 0;
  uint32_t tokens = 0;
  for (int r = 0; r < all.blocks; ++r) {
    const SampleSmem& o = all.of(r);
    const uint32_t c = o.count[tid];
    tokens += c;
    mine += kMass ? (uint64_t)o.high[tid] << 32 | o.low[tid] : c;
  }
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
      sm.out[3] = tokens;
    }
  }
  __syncthreads();
  const int bin = (int)sm.out[0];
  if (bin == kBins) {
    if (kMass) *sum = block_sum(sm, mine);   // bins of the whole row
    all.sync();   // the others may still be reading this block's bins
    return have;
  }
  const uint64_t rest = sm.out[1], base = sm.out[2];
  const uint32_t n = (uint32_t)sm.out[3];
  auto in_bin = [&](int i, float x, uint32_t& k) {
    if (x == kNegInf || bin_of(w, inv, x) != bin) return false;
    k = key_of(x);
    return have.keeps(k, i) && (!kMass || have.of(w(x)) != 0);
  };
  if (n <= kList) {   // every one of the bin's tokens, in the first block, counts those before it
    SampleSmem& to = all.of(0);
    for_tokens<1>(row, begin, end, tid, kThreads, [&](int i, float x) {
      uint32_t k;
      if (!in_bin(i, x, k)) return;
      const int at = atomicAdd(&to.listed, 1);
      to.list[at] = (uint64_t)k << 32 | (uint32_t)~i;
      to.list_w[at] = kMass ? w(x) : 1;
    });
    all.sync();
    if (all.rank == 0) {   // a warp a token
      for (int e = tid >> 5; e < (int)n; e += kWarps) {
        const uint64_t mine = sm.list[e], own = sm.list_w[e];
        uint64_t above = 0;
        for (int j = lane; j < (int)n; j += 32) above += sm.list[j] > mine ? sm.list_w[j] : 0;
        above = warp_sum(above);
        if (above < rest && above + own >= rest && lane < all.blocks) {
          SampleSmem& o = all.of(lane);
          o.out[0] = mine >> 32;
          o.out[1] = (uint32_t)~(uint32_t)mine;
          o.out[3] = base + above + own;
        }
      }
    }
    all.sync();
    if (kMass) *sum = sm.out[3];
    return {(uint32_t)sm.out[0], (int32_t)(uint32_t)sm.out[1], have.least};
  }
  // more than fit (many equal logits): by bisection of their keys, a pass over the row a step
  uint32_t lo = 0xffffffffu, hi = 0;
  for_tokens<1>(row, begin, end, tid, kThreads, [&](int i, float x) {
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
  uint64_t pair = sm.part[lane];
  lo = __reduce_min_sync(0xffffffffu, (uint32_t)pair);
  hi = __reduce_max_sync(0xffffffffu, (uint32_t)(pair >> 32));
  if constexpr (kMany) {
    const uint64_t* pairs = all.exchange((uint64_t)hi << 32 | lo);
    for (int r = 0; r < all.blocks; ++r) {
      lo = min(lo, (uint32_t)pairs[r]);
      hi = max(hi, (uint32_t)(pairs[r] >> 32));
    }
  }
  auto value_of = [](uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); };
  auto summed = [&](auto&& f) {   // the sum of f(key, index) over the bin's tokens
    uint64_t s = 0;
    for_tokens<1>(row, begin, end, tid, kThreads, [&](int i, float x) {
      uint32_t k;
      if (in_bin(i, x, k)) s += f(k, i);
    });
    return row_sum(all, s);
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

template <typename T, bool kMany>
__global__ void __launch_bounds__(kThreads) token_sample_kernel(const __grid_constant__ SampleParams p) {
  __shared__ SampleSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = p.V;
  Row<kMany> all = {sm, 0, 1, 0};
  if constexpr (kMany) {
    all.rank = (int)cg::this_cluster().block_rank();
    all.blocks = (int)cg::this_cluster().num_blocks();
  }
  // this block's slice, in whole vectors
  const int slice = ((V + all.blocks - 1) / all.blocks + 7) / 8 * 8, begin = min(V, all.rank * slice), end = min(V, begin + slice);
  if (tid < 256) {
    const uint32_t m = exp2_fraction((uint32_t)tid << 24);
    sm.table[tid] = make_uint2(m, __float_as_uint((float)m));
  }
  all.sync();   // every block of the row has begun
  for (int64_t r = blockIdx.x / all.blocks; r < p.rows; r += gridDim.x / all.blocks) {
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
    for_tokens<4>(row, begin, end, tid, kThreads, [&](int i, float x) {
      const uint64_t k = (uint64_t)key_of(x) << 32 | (uint32_t)~i;
      best = k > best ? k : best;
    });
    auto larger = [](uint64_t a, uint64_t b) { return a > b ? a : b; };
#pragma unroll
    for (int o = 16; o; o >>= 1) best = larger(best, __shfl_xor_sync(0xffffffffu, best, o));
    __syncthreads();
    if (lane == 0) sm.part[warp] = best;
    __syncthreads();
    best = sm.part[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) best = larger(best, __shfl_xor_sync(0xffffffffu, best, o));
    if constexpr (kMany) {
      const uint64_t* of = all.exchange(best);
      for (int b = 0; b < all.blocks; ++b) best = larger(best, of[b]);
    }
    const uint32_t top_key = (uint32_t)(best >> 32);
    Weight w;
    w.table = sm.table;
    const float most = __uint_as_float(top_key & 0x80000000u ? top_key & 0x7fffffffu : ~top_key);
    if (most == kNegInf || temp == 0.f) {
      if (tid == 0 && all.rank == 0) {
        p.ids[r] = most == kNegInf ? -1 : (int64_t)(uint32_t)~(uint32_t)best;
        if (p.logprob) p.logprob[r] = most == kNegInf ? NAN : 0.f;
      }
      continue;
    }
    // 2 log2(e) / temperature in two floats: the quotient, and what its product with the temperature leaves
    const float tt = fmaxf(temp, 1e-30f);
    w.half = 0.5f * most;
    w.ch = 2.88539004f / tt;
    w.cl = w.ch > 0.f ? (fmaf(-w.ch, tt, 2.88539004f) + 3.85192598e-8f) / tt : 0.f;   // 0 inf is NaN
    w.shift = p.shift;
    Cut cut = {0, V, 1};
    if (min_p > 0.f) {   // a bound on the weights, rounded up
      const uint64_t one = 1ull << w.shift, f = min_p < 1.f ? fixed64(min_p) : 0;
      const uint64_t least = __umul64hi(f, one) + (f * one ? 1 : 0);
      cut.least = min_p < 1.f ? (least ? least : 1) : one;
    }
    auto kept = [&](int i, float x) -> uint64_t { return cut.keeps(key_of(x), i) ? cut.of(w(x)) : 0; };
    uint64_t total = 0;
    bool summed = false;
    const float inv = (float)kBins / 43.5f / tt * 2.f;   // of half distances; weights end at 2^-62.5 = e^-43.3
    if (top_k > 0 && top_k < V)
      cut = find_cut<false>(all, row, begin, end, V, w, inv, cut, (uint64_t)top_k, nullptr);
    if (by_sum) {
      cut = find_cut<true>(all, row, begin, end, V, w, inv, cut, fixed64(fmaxf(top_p, 0.f)), &total);
      summed = true;
    }
    // the draw: sums of the blocks, of 32 parts of the slice by warp, then the chosen part by the whole block.  Where no
    // order was needed, the sums are first taken of fp32 weights, whose error is known: 2^-22 by the special function; three
    // roundings of an exponent e make 2.1 e 2^-24, and the mean of e over the weights is at most log2 V = 20; 2^-24 for
    // each of a thread's additions.  Only where the number drawn is as near as that to a border between two tokens, exact
    // sums follow: of 50000 tokens in one block, with 9e-6 of the sum on either side, in a row of ten where a few dozen tokens
    // are likely (512 rows f32 in 75 us), but in nine of ten where all are about alike (125 us).
    const int len = ((end - begin + kWarps - 1) / kWarps + 7) / 8 * 8;
    const int from = min(end, begin + warp * len), to = min(end, from + len);
    const float u = __ldg(p.u + r);
    const uint64_t share = u >= 1.f ? ~0ull : u > 0.f ? fixed64(u) : 0;
    auto last_part = [&](int b0, int b1, uint64_t target, uint64_t total, uint64_t slack) {
      // a token a thread; whether one was found `slack` away from its borders
      bool clear = false;
      for (int i0 = b0; i0 < b1; i0 += kThreads) {
        const int i = i0 + tid;
        float x = i < b1 ? ld_f32(row + i) : kNegInf;
        if (x != x) x = kNegInf;
        const uint64_t own = i < b1 ? kept(i, x) : 0;
        uint64_t before;
        const int of = pick_warp(sm, own, target, &before);
        const uint64_t through = block_sum(sm, own);
        if (target >= through && i0 + kThreads < b1) {
          if (target - through < slack) return false;
          target -= through;
          continue;
        }
        uint64_t upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint64_t v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const uint64_t here = before + upto;
        const uint32_t past = __ballot_sync(0xffffffffu, here > target);
        const bool mine = warp == of && past && lane == __ffs(past) - 1;
        clear = __syncthreads_or(mine && here - target > slack && target - (here - own) >= slack);
        if (mine && clear) {
          p.ids[r] = i;
          if (p.logprob) {
            const float d = fmaf(x, -0.5f, w.half), z = d > 0.f ? -2.f * (d / tt) : 0.f;
            // the sum is at least the largest weight: its logarithm by that of its 24 leading bits
            p.logprob[r] = z - logf((float)total * __uint_as_float((uint32_t)(127 - w.shift) << 23));
          }
        }
        break;
      }
      return clear;
    };
    uint64_t s = 0, mine = 0, ahead = 0, before;
    if (!summed && cut.key == 0 && cut.last == V && cut.least == 1 && w.ch > 0.f) {   // (not at an infinite temperature)
      float f0 = 0.f, f1 = 0.f;
      for_tokens<4>(row, from, to, lane, 32, [&](int i, float x) {
        const float d = fmaf(x, 0.5f, -w.half), e = exp2f_fast(d * w.ch);
        if (i & 1) f1 += d < 0.f ? e : 1.f;
        else f0 += d < 0.f ? e : 1.f;
      });
      const float one = __uint_as_float((uint32_t)(127 + w.shift) << 23);
      s = __float2ull_rn((f0 + f1) * one);
      mine = block_sum(sm, s);
      total = mine;
      if constexpr (kMany) {
        const uint64_t* of = all.exchange(mine);
        total = 0;
        for (int b = 0; b < all.blocks; ++b) {
          if (b == all.rank) ahead = total;
          total += of[b];
        }
      }
      const uint64_t slack = (total >> 24) * (uint64_t)(2 * (len / 64 + 52));   // in the sum before and in the target
      uint64_t target = __umul64hi(share, total);
      bool clear = true;
      if (!kMany || (target >= ahead && target < ahead + mine)) {
        target -= ahead;
        const int part = pick_warp(sm, s, target, &before), b0 = min(end, begin + part * len), b1 = min(end, b0 + len);
        clear = last_part(b0, b1, target - before, total, slack);
      }
      bool all_clear = clear;
      if constexpr (kMany) {
        const uint64_t* of = all.exchange(clear);
        for (int b = 0; b < all.blocks; ++b) all_clear = all_clear && of[b];
      }
      if (all_clear) continue;
      ahead = 0;
      s = 0;
    }
    for_tokens<1>(row, from, to, lane, 32, [&](int i, float x) { s += kept(i, x); });
    if (kMany || !summed) {
      mine = block_sum(sm, s);
      total = mine;
      if constexpr (kMany) {
        const uint64_t* of = all.exchange(mine);
        total = 0;
        for (int b = 0; b < all.blocks; ++b) {
          if (b == all.rank) ahead = total;
          total += of[b];
        }
      }
    }
    uint64_t target = u >= 1.f ? total - 1 : __umul64hi(share, total);
    if (kMany && (target < ahead || target >= ahead + mine)) continue;   // another block's
    target -= ahead;
    const int part = pick_warp(sm, s, target, &before), b0 = min(end, begin + part * len), b1 = min(end, b0 + len);
    last_part(b0, b1, target - before, total, 0);
  }
  all.sync();   // no block ends while another may read or write its shared memory
}

template <typename T>
cudaError_t launch_sample(const SampleParams& p, cudaStream_t st) {
  // as many blocks a row as leave one block an SM
  unsigned blocks = 1;
  while (blocks < 8 && p.rows * (blocks * 2) <= 152) blocks *= 2;
  if (blocks == 1) {
    token_sample_kernel<T, false><<<(unsigned)(p.rows < (1 << 20) ? p.rows : 1 << 20), kThreads, 0, st>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = blocks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, token_sample_kernel<T, true>, p);
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
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t err = shape->io_dtype == SSD_BF16 ? launch_sample<__nv_bfloat16>(p, st) : launch_sample<float>(p, st);
  return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
