// Token embedding with scaling and the gradient of its table (declarations in include/ssdscan.h):
//   out[i] = scale * table[ids[i]],  dtable[v] = scale * sum_{ids[i] = v} dout[i].
#include <math.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>

#include "common.cuh"
#include "fp_helpers.cuh"
#include "launch.h"
#include "pack.cuh"

namespace ssd {
namespace {

constexpr int kThreads = 256;

template <typename Id>
__device__ __forceinline__ int64_t row_of(const Id* ids, int64_t i, int64_t V) {
  const int64_t v = (int64_t)__ldg(ids + i);
  return v >= 0 && v < V ? v : -1;
}

// V values as one load or store of up to 16 bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

// ------------------------------------------------------------------------------------------------
// Forward: a thread takes one vector column of U tokens at a time, all their loads in flight.  Bound by
// memory: the distinct rows once (repeated ones come from L2) and out once.  32768 tokens of a 50000 x
// 2048 bf16 table, frequencies as 1/rank: 33 us, 5.3 TB/s of 174 MB (78 % of the measured copy rate).
// ------------------------------------------------------------------------------------------------
template <typename T, typename Id, int V>
__global__ void __launch_bounds__(kThreads) embed_forward_kernel(const Id* ids, int64_t n, const T* table, int64_t rows,
                                                                 int64_t D, float scale, T* out, int cols,
                                                                 int tokens) {
  using Q = Pack<T, V>;
  constexpr int U = 4;   // tokens in flight
  const int col = threadIdx.x % cols, sub = threadIdx.x / cols;   // tokens: tokens a block takes at a time
  const int64_t d = ((int64_t)blockIdx.y * cols + col) * V;
  if (sub >= tokens || d >= D) return;
  const int64_t step = (int64_t)gridDim.x * tokens * U;
  int64_t next[U];   // the rows of the tokens after these
  auto fetch = [&](int64_t i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) next[u] = i0 + u * tokens < n ? row_of(ids, i0 + u * tokens, rows) : -1;
  };
  int64_t i0 = (int64_t)blockIdx.x * tokens * U + sub;
  T* o = out + i0 * D + d;
  fetch(i0);
  for (; i0 < n; i0 += step) {
    typename Q::Raw f[U];
    float times[U];   // padding is zeros whatever the scale
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f[u] = next[u] >= 0 ? Q::raw(table + next[u] * D + d) : Q::none();
      times[u] = next[u] >= 0 ? scale : 0.f;
    }
    fetch(i0 + step);
#pragma unroll
    for (int u = 0; u < U; ++u, o += tokens * D) {
      float2 v[Q::P];
      Q::unpack(f[u], v);
#pragma unroll
      for (int e = 0; e < Q::P; ++e) v[e] = fp::mul2(v[e], make_float2(times[u], times[u]));
      if (i0 + u * tokens < n) Q::store(o, v);
    }
    o += (step - U * tokens) * D;
  }
}

// ------------------------------------------------------------------------------------------------
// Backward.
//
// 1. The tokens are sorted by id, stably, so that a row's tokens stand together in their order: a radix
//    sort of 8 bits a pass, least significant digit first (Knuth, The Art of Computer Programming 3, 5.2.5),
//    the padding's key behind all rows.  It is short of work, so its launches,
//    like the others, take along the clearing of rows that no token has.
// 2. A subgroup of threads takes kPiece sorted tokens and adds their rows, writing each row's sum as its
//    run ends; a run that goes on over the ends of a piece leaves partial sums instead,
// 3. which the piece where the run starts joins, in order.
// Bound by memory: dout once, every row of dtable once.  32768 tokens, 50000 x 2048 bf16: 117 us, 4.6 TB/s
// of 544 MB (69 % of the measured copy rate): sorting takes 7 + 2 x 12 us beside 94 MB of clearing, the
// sums 60 us for 401 MB, the join 19 us beside 47 MB.  With few tokens and rows it is a chain of
// five short launches: 14824 tokens, 10335 x 324 f32 take 40 us.
// ------------------------------------------------------------------------------------------------
constexpr int kBins = 256;
constexpr int kKeys = 8;                        // keys of a thread
constexpr int kSortTile = kThreads * kKeys;     // keys of a block

struct EmbedParams {
  const void* ids;
  int64_t n, rows, D;
  const void* dout;
  float scale;
  float* dtable;
  uint8_t* used;                 // [rows] a token has this row
  uint32_t *key[2], *pos[2];     // sorted ping-pong; a key is the row, or `rows` for padding
  uint32_t *hist, *next_hist;    // [kBins, sort tiles] of this pass and of the next (NULL: the last)
  float *head, *tail;            // [pieces, D] partial sums
  int32_t sort_tiles, shift;
  int32_t in;                    // which of key/pos is read
  int32_t piece;                 // tokens of a piece
  int64_t pieces;
  int64_t fill0, fill1;          // rows that this launch clears where unused
  int32_t work_blocks;           // blocks (in x) that sort or add; the rest clear
  WsHeader* hdr;
};

// Rows [fill0, fill1) without tokens are zeros, by the warps of the blocks behind the working ones, four
// neighbouring rows a warp at a time with the flags of the next four on their way.
__device__ __forceinline__ void clear_rows(const EmbedParams& p) {
  constexpr int kRows = 4;
  const int lane = threadIdx.x % 32;
  const int64_t blocks = (int64_t)(gridDim.x - p.work_blocks) * gridDim.y;
  const int64_t first = (int64_t)(blockIdx.x - p.work_blocks) * gridDim.y + blockIdx.y;
  const int64_t step = blocks * (kThreads / 32) * kRows;
  const bool wide = p.D % 4 == 0 && (reinterpret_cast<uintptr_t>(p.dtable) & 15) == 0;
  auto flag = [&](int64_t r) { return lane < kRows && r + lane < p.fill1 ? (int)p.used[r + lane] : 1; };
  int64_t r = p.fill0 + (first * (kThreads / 32) + threadIdx.x / 32) * kRows;
  int next = flag(r);
  for (; r < p.fill1; r += step) {
    unsigned empty = __ballot_sync(0xffffffffu, next == 0);
    next = flag(r + step);
    for (; empty != 0; empty &= empty - 1) {
      const int64_t row = r + __ffs(empty) - 1;
      if (!SSD_INDEX_OK(p.hdr, (row + 1) * p.D - 1, p.rows * p.D, 80)) continue;
      float* to = p.dtable + row * p.D;
      if (wide) {
        for (int64_t d = lane; d < p.D / 4; d += 32) reinterpret_cast<float4*>(to)[d] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else {
        for (int64_t d = lane; d < p.D; d += 32) to[d] = 0.f;
      }
    }
  }
}

// Keys from ids, the rows that occur, and how many keys of a block have each lowest digit.
template <typename Id>
__global__ void __launch_bounds__(kThreads) embed_keys_kernel(EmbedParams p) {
  follow();
  __shared__ uint32_t bins[kBins];
  bins[threadIdx.x] = 0;
  __syncthreads();
  uint32_t key[kKeys];
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const int64_t i = (int64_t)blockIdx.x * kSortTile + k * kThreads + threadIdx.x;
    const int64_t r = i < p.n ? row_of(static_cast<const Id*>(p.ids), i, p.rows) : -1;
    key[k] = r < 0 ? (uint32_t)p.rows : (uint32_t)r;
  }
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const int64_t i = (int64_t)blockIdx.x * kSortTile + k * kThreads + threadIdx.x;
    if (i >= p.n) continue;
    if (key[k] != (uint32_t)p.rows) p.used[key[k]] = 1;
    p.key[p.in][i] = key[k];
    atomicAdd(&bins[key[k] & (kBins - 1)], 1u);
  }
  __syncthreads();
  p.hist[(int64_t)threadIdx.x * p.sort_tiles + blockIdx.x] = bins[threadIdx.x];
}
static_assert(kBins == kThreads, "a thread a bin");

// Few tokens: one block sorts them in shared memory, all passes in one launch.
template <typename Id>
__global__ void __launch_bounds__(kThreads) embed_small_sort_kernel(EmbedParams p, int passes) {
  constexpr int kW = kThreads / 32;
  __shared__ uint32_t keys[2][kSortTile], places[2][kSortTile], seen[kW][kBins], warps[kW];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, n = (int)p.n;
  follow();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int64_t r = row_of(static_cast<const Id*>(p.ids), i, p.rows);
    keys[0][i] = r < 0 ? (uint32_t)p.rows : (uint32_t)r;
    places[0][i] = (uint32_t)i;
    if (r >= 0) p.used[r] = 1;
  }
  for (int pass = 0; pass < passes; ++pass) {
    const uint32_t *key = keys[pass & 1], *pos = places[pass & 1];
    const int shift = 8 * pass;
    for (int k = threadIdx.x; k < kW * kBins; k += kThreads) (&seen[0][0])[k] = 0;
    __syncthreads();
    uint32_t rank[kKeys];
    const int i0 = warp * 32 * kKeys + lane;   // a warp takes neighbouring keys, 32 at a time
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      const bool in = i0 + k * 32 < n;
      const uint32_t digit = in ? (key[i0 + k * 32] >> shift) & (kBins - 1) : kBins;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      const uint32_t had = in ? seen[warp][digit] : 0u;
      rank[k] = had + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (in && lane == __ffs(same) - 1) seen[warp][digit] = had + __popc(same);
      __syncwarp();
    }
    __syncthreads();
    uint32_t all = 0;   // a thread a digit
#pragma unroll
    for (int k = 0; k < kW; ++k) all += seen[k][threadIdx.x];
    uint32_t inc = all;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warps[warp] = inc;
    __syncthreads();
    uint32_t base = inc - all;
    for (int k = 0; k < warp; ++k) base += warps[k];
#pragma unroll
    for (int k = 0; k < kW; ++k) {
      const uint32_t c = seen[k][threadIdx.x];
      seen[k][threadIdx.x] = base;
      base += c;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kKeys; ++k) {
      const int i = i0 + k * 32;
      if (i >= n) continue;
      const uint32_t at = seen[warp][(key[i] >> shift) & (kBins - 1)] + rank[k];
      keys[(pass & 1) ^ 1][at] = key[i];
      places[(pass & 1) ^ 1][at] = pos[i];
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += kThreads) {
    p.key[p.in][i] = keys[passes & 1][i];
    p.pos[p.in][i] = places[passes & 1][i];
  }
}

// hist becomes its exclusive prefix sum over digits, then tiles, by one block.
__global__ void __launch_bounds__(kThreads) embed_scan_kernel(EmbedParams p) {
  follow();
  if (blockIdx.x > 0) return clear_rows(p);
  __shared__ uint32_t warps[kThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t n = (int64_t)kBins * p.sort_tiles;
  uint32_t before = 0;
  constexpr int kPer = 8;   // neighbouring entries of a thread at a time
  for (int64_t at = 0; at < n; at += kThreads * kPer) {
    uint32_t v[kPer], sum = 0;
    const int64_t i0 = at + threadIdx.x * kPer;
#pragma unroll
    for (int k = 0; k < kPer; ++k) v[k] = i0 + k < n ? p.hist[i0 + k] : 0u;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const uint32_t x = v[k];
      v[k] = sum;
      sum += x;
    }
    uint32_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warps[warp] = inc;
    __syncthreads();
    uint32_t base = before + inc - sum;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < warp) base += warps[k];
      before += warps[k];
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (i0 + k < n) p.hist[i0 + k] = base + v[k];
    __syncthreads();
  }
}

// Keys and positions to their places by the pass's digit, equal digits in their order: a warp takes
// neighbouring keys, 32 at a time.  Counts the next pass's digits of the tiles that they go to (whole
// numbers: the order of the additions does not matter).  Where the tiles are few every block forms the
// prefix sums of the counts for itself, which spares the scan's launch.
constexpr int kFewTiles = 64;
template <bool kScanned>
__global__ void __launch_bounds__(kThreads) embed_scatter_kernel(EmbedParams p) {
  follow();
  if ((int)blockIdx.x >= p.work_blocks) return clear_rows(p);
  constexpr int kW = kThreads / 32;
  __shared__ uint32_t seen[kW][kBins];   // keys of the warp with this digit
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int k = threadIdx.x; k < kW * kBins; k += kThreads) (&seen[0][0])[k] = 0;
  __syncthreads();
  uint32_t key[kKeys], pos[kKeys], rank[kKeys];
  const int64_t i0 = (int64_t)blockIdx.x * kSortTile + warp * 32 * kKeys + lane;
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const int64_t i = i0 + k * 32;
    const bool in = i < p.n;
    key[k] = in ? p.key[p.in][i] : 0u;
    pos[k] = in && p.shift > 0 ? p.pos[p.in][i] : (uint32_t)i;
  }
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const bool in = i0 + k * 32 < p.n;
    const uint32_t digit = in ? (key[k] >> p.shift) & (kBins - 1) : kBins;
    const uint32_t same = __match_any_sync(0xffffffffu, digit);
    const uint32_t had = in ? seen[warp][digit] : 0u;
    rank[k] = had + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (in && lane == __ffs(same) - 1) seen[warp][digit] = had + __popc(same);
    __syncwarp();
  }
  __syncthreads();
  {   // a thread a digit: where the warps' keys of it start
    const uint32_t* row = p.hist + (int64_t)threadIdx.x * p.sort_tiles;
    uint32_t base;
    if (kScanned) {
      base = row[blockIdx.x];
    } else {
      __shared__ uint32_t warps[kW];
      uint32_t all = 0, mine = 0;
#pragma unroll 8
      for (int k = 0; k < p.sort_tiles; ++k) {
        const uint32_t c = row[k];
        all += c;
        mine += k < (int)blockIdx.x ? c : 0u;
      }
      uint32_t inc = all;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      if (lane == 31) warps[warp] = inc;
      __syncthreads();
      base = inc - all + mine;
      for (int k = 0; k < warp; ++k) base += warps[k];
    }
#pragma unroll
    for (int k = 0; k < kW; ++k) {
      const uint32_t c = seen[k][threadIdx.x];
      seen[k][threadIdx.x] = base;
      base += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kKeys; ++k) {
    const bool in = i0 + k * 32 < p.n;
    int64_t at = 0;
    if (in) {
      at = seen[warp][(key[k] >> p.shift) & (kBins - 1)] + rank[k];
      if (SSD_INDEX_OK(p.hdr, at, p.n, 81)) {
        p.key[p.in ^ 1][at] = key[k];
        p.pos[p.in ^ 1][at] = pos[k];
      }
    }
    if (p.next_hist) {   // lanes with the same count are added by one: the last pass may have two digits only
      const uint32_t bin =
          in ? ((key[k] >> (p.shift + 8)) & (kBins - 1)) * (uint32_t)p.sort_tiles + (uint32_t)(at / kSortTile) : ~0u;
      const uint32_t same = __match_any_sync(0xffffffffu, bin);
      if (in && lane == __ffs(same) - 1) atomicAdd(p.next_hist + bin, (uint32_t)__popc(same));
    }
  }
}

// A vector of fp32 values to `p`, in the widest stores its alignment takes.
template <int V>
__device__ __forceinline__ void store_sum(float* p, const float (&v)[V], float scale) {
  if (V % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
#pragma unroll
    for (int k = 0; k + 3 < V; k += 4)
      *reinterpret_cast<float4*>(p + k) = make_float4(scale * v[k], scale * v[k + 1], scale * v[k + 2], scale * v[k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) p[k] = scale * v[k];
  }
}

// A thread's vector of one row (4 bytes or more) to its own place in shared memory; it alone reads it there.
template <int kBytes>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else if constexpr (kBytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(d), "l"(src) : "memory");
  else if constexpr (kBytes == 4) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(d), "l"(src) : "memory");
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(EmbedParams p, int cols, int subs) {
  follow();
  constexpr int kRing = 12;   // rows in flight: 48 KB a block, four blocks an SM
  __shared__ Vec<T, V> ring[kRing][kThreads];
  if ((int)blockIdx.x >= p.work_blocks) return clear_rows(p);
  const int col = threadIdx.x % cols, sub = threadIdx.x / cols;
  const int64_t d = ((int64_t)blockIdx.y * cols + col) * V, piece = (int64_t)blockIdx.x * subs + sub;
  if (sub >= subs || d >= p.D || piece >= p.pieces) return;
  const uint32_t none = (uint32_t)p.rows;
  const int64_t j0 = piece * p.piece;
  const int n = (int)min((int64_t)p.piece, p.n - j0);
  const uint32_t *key = p.key[p.in] + j0, *pos = p.pos[p.in] + j0;
  const T* dout = static_cast<const T*>(p.dout) + d;
  uint32_t cur = *key;
  if (cur == none) return;
  bool open = j0 > 0 && key[-1] == cur;   // the run in hand started in an earlier piece
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  auto flush = [&](bool goes_on) {
    float* to = open ? p.head + piece * p.D : goes_on ? p.tail + piece * p.D : p.dtable + cur * p.D;
    const bool whole = !open && !goes_on;
    if (SSD_INDEX_OK(p.hdr, (whole ? cur : piece) * p.D + d + V - 1, (whole ? p.rows : p.pieces) * p.D, 82))
      store_sum<V>(to + d, acc, whole ? p.scale : 1.f);
  };
  auto request = [&](int j, int slot) {
    if (j < n) copy_async<V * (int)sizeof(T)>(&ring[slot][threadIdx.x], dout + (int64_t)pos[j] * p.D);
    cp_async_commit();
  };
  if constexpr (V * (int)sizeof(T) < 4) {   // single bf16 values: no asynchronous copy takes them
    constexpr int U = 16;
    for (int j = 0; j < n; j += U) {
      T f[U];
      uint32_t k[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        k[u] = j + u < n ? key[j + u] : none;
        if (k[u] != none) f[u] = dout[(int64_t)pos[j + u] * p.D];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (k[u] == none) continue;
        if (k[u] != cur) {
          flush(false);
          open = false;
          cur = k[u];
          acc[0] = 0.f;
        }
        acc[0] += (float)f[u];
      }
    }
    flush(j0 + n < p.n && key[n] == cur);
    return;
  }
  for (int j = 0; j < kRing; ++j) request(j, j);
  int slot = 0;
  for (int j = 0; j < n; ++j) {
    const uint32_t k = key[j];
    if (k == none) break;   // padding stands behind all rows
    if (k != cur) {
      flush(false);
      open = false;
      cur = k;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = 0.f;
    }
    cp_async_wait<kRing - 1>();
    const Vec<T, V> f = ring[slot][threadIdx.x];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] += (float)f.v[e];
    request(j + kRing, slot);
    slot = slot + 1 == kRing ? 0 : slot + 1;
  }
  cp_async_wait_all();
  flush(j0 + n < p.n && key[n] == cur);
}

// Runs over more than one piece: the piece where one starts adds the heads of those after it.  Keys and
// heads are asked for together (a head that is not the run's is not used), 32 values a thread at a time.
template <int V>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(EmbedParams p, int cols, int subs) {
  follow();
  constexpr int U = 32 / V;   // heads in flight
  if ((int)blockIdx.x >= p.work_blocks) return clear_rows(p);
  const int col = threadIdx.x % cols, sub = threadIdx.x / cols;
  const int64_t d = ((int64_t)blockIdx.y * cols + col) * V, piece = (int64_t)blockIdx.x * subs + sub;
  if (sub >= subs || d >= p.D || piece >= p.pieces) return;
  const uint32_t* key = p.key[p.in];
  const int64_t j0 = piece * p.piece, j1 = j0 + p.piece;
  if (j1 >= p.n) return;
  const uint32_t run = key[j1];   // the run that crosses the piece's end, if it is in this piece
  const uint32_t last = key[j1 - 1], early = j0 > 0 ? key[j0 - 1] : (uint32_t)p.rows;
  if (run == (uint32_t)p.rows || last != run || early == run) return;   // or it started earlier
  using F = Vec<float, V>;
  F acc = *reinterpret_cast<const F*>(p.tail + piece * p.D + d);
  for (int64_t q = piece + 1;; q += U) {
    F h[U];
    bool in[U];   // the run reaches piece q + u
#pragma unroll
    for (int u = 0; u < U; ++u) {
      in[u] = q + u < p.pieces;
      if (in[u]) {
        h[u] = *reinterpret_cast<const F*>(p.head + (q + u) * p.D + d);
        in[u] = key[(q + u) * p.piece] == run;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < V; ++e) acc.v[e] += in[u] ? h[u].v[e] : 0.f;
    if (!in[U - 1]) break;
  }
  if (SSD_INDEX_OK(p.hdr, run * p.D + d + V - 1, p.rows * p.D, 85)) store_sum<V>(p.dtable + run * p.D + d, acc.v, p.scale);
}

constexpr int64_t kMaxElems = (int64_t)1 << 40;

ssd_status check_sizes(int64_t n, int64_t V, int64_t D) {
  if (n < 0 || V < 1 || D < 1) return SSD_ERR_INVALID_ARG;
  if (n > 0x7fffffffLL || V >= 0x7fffffffLL || D > kMaxElems / V || (n > 0 && D > kMaxElems / n))
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

bool misaligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }
ssd_status done(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

// Vector width (values) that every row of the arrays is aligned to, 16 bytes at most.
int row_vec(size_t e, int64_t D, std::initializer_list<const void*> arrays) {
  uint64_t bits = (uint64_t)D * e;
  for (const void* a : arrays) bits |= reinterpret_cast<uintptr_t>(a);
  int v = (int)(16 / e);
  while (v > 1 && bits % (v * e) != 0) v /= 2;
  return v;
}

// Threads across a row of nv vectors, and how many rows a block takes side by side.
struct Split {
  int cols, subs;
  unsigned slices;
};
Split split_row(int64_t nv) {
  const int64_t slices = (nv + kThreads - 1) / kThreads;
  const int cols = (int)((nv + slices - 1) / slices);
  return {cols, kThreads / cols, (unsigned)slices};
}

// Rows are cut into slices of a block's vectors each, at most 65535 of them (a grid's second axis).
bool too_wide(int64_t D, int vec) { return (D + vec - 1) / vec > (int64_t)kThreads * 65535; }

template <typename T, typename Id, int V>
cudaError_t launch_forward_as(const void* ids, int64_t n, const void* table, int64_t rows, int64_t D, float scale,
                              void* out, cudaStream_t st) {
  const Split s = split_row((D + V - 1) / V);
  auto* kernel = embed_forward_kernel<T, Id, V>;
  int blocks = 0;
  const cudaError_t e = resident_blocks(kernel, kThreads, 0, &blocks);
  if (e != cudaSuccess) return e;
  const int64_t steps = (n + s.subs * 4 - 1) / (s.subs * 4);
  const unsigned bx = (unsigned)std::min<int64_t>(steps, std::max<int64_t>(1, blocks / s.slices));
  kernel<<<dim3(bx, s.slices), kThreads, 0, st>>>(static_cast<const Id*>(ids), n, static_cast<const T*>(table), rows, D,
                                                  scale, static_cast<T*>(out), s.cols, s.subs);
  return cudaGetLastError();
}

template <typename T, typename Id>
cudaError_t launch_forward(const void* ids, int64_t n, const void* table, int64_t rows, int64_t D, float scale,
                           void* out, cudaStream_t st) {
  switch (row_vec(sizeof(T), D, {table, out})) {
    case 8:
      if constexpr (sizeof(T) == 2) return launch_forward_as<T, Id, 8>(ids, n, table, rows, D, scale, out, st);
    case 4: return launch_forward_as<T, Id, 4>(ids, n, table, rows, D, scale, out, st);
    case 2: return launch_forward_as<T, Id, 2>(ids, n, table, rows, D, scale, out, st);
    default: return launch_forward_as<T, Id, 1>(ids, n, table, rows, D, scale, out, st);
  }
}

struct EmbedLayout {
  size_t used = 0, hist = 0, cleared = 0, key[2] = {0, 0}, pos[2] = {0, 0}, head = 0, tail = 0, total = 0;
  int64_t sort_tiles = 0, pieces = 0;
  int32_t piece = 0;
};
// Passes of 8 bits over keys up to `rows`.
int embed_passes(int64_t rows) {
  int passes = 1;
  while (passes < 4 && (rows >> (8 * passes)) != 0) passes += 1;
  return passes;
}
EmbedLayout embed_layout(int64_t n, int64_t rows, int64_t D) {
  EmbedLayout L;
  L.sort_tiles = (n + kSortTile - 1) / kSortTile;
  // short pieces while they do not fill the machine (four blocks an SM), then longer ones: they keep the
  // chain of partial sums that the join of a frequent row follows short
  L.piece = 32;
  while (L.piece < 256 && n / L.piece > 4 * 152) L.piece *= 2;
  L.pieces = (n + L.piece - 1) / L.piece;
  size_t off = sizeof(WsHeader);
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, kWsAlign);
    return at;
  };
  L.used = take((size_t)rows);   // cleared together with the counts behind it
  L.hist = take(sizeof(uint32_t) * kBins * (size_t)L.sort_tiles * embed_passes(rows));
  L.cleared = off - L.used;
  for (int k = 0; k < 2; ++k) L.key[k] = take(sizeof(uint32_t) * (size_t)n);
  for (int k = 0; k < 2; ++k) L.pos[k] = take(sizeof(uint32_t) * (size_t)n);
  L.head = take(sizeof(float) * (size_t)(L.pieces * D));
  L.tail = take(sizeof(float) * (size_t)(L.pieces * D));
  L.total = off;
  return L;
}

// The rows to clear, shared out to the launches behind the first: a sorting step and the join of long
// runs take a little of it in the time that they wait, the sums, bound by memory themselves, the rest.
constexpr int kSortShare = 2, kSumShare = 8, kJoinShare = 2;
struct Fill {
  int64_t done = 0, all = 0;
  unsigned take(EmbedParams& p, int share, int work) {
    p.work_blocks = work;
    p.fill0 = p.rows * done / all;
    done += share;
    p.fill1 = p.rows * done / all;
    const int64_t blocks = (p.fill1 - p.fill0 + 31) / 32;   // 8 warps of 4 rows each
    return (unsigned)(work + std::max<int64_t>(1, std::min<int64_t>(152 * 8, blocks)));
  }
};

template <typename T, int V>
cudaError_t launch_sum(EmbedParams p, Fill& fill, cudaStream_t st) {
  const Split s = split_row((p.D + V - 1) / V);
  const int work = (int)((p.pieces + s.subs - 1) / s.subs);
  const unsigned bx = fill.take(p, kSumShare, work);
  const cudaError_t e = launch_next(embed_sum_kernel<T, V>, dim3(bx, s.slices), kThreads, 0, st, p, s.cols, s.subs);
  if (e != cudaSuccess || p.pieces < 2) return e;   // one piece: no run crosses its end
  // the partial rows are aligned as the width is
  const int v = p.D % 4 == 0 ? 4 : p.D % 2 == 0 ? 2 : 1;
  const Split js = split_row(p.D / v);
  const unsigned jx = fill.take(p, kJoinShare, (int)((p.pieces + js.subs - 1) / js.subs));
  auto* join = v == 4 ? embed_join_kernel<4> : v == 2 ? embed_join_kernel<2> : embed_join_kernel<1>;
  return launch_next(join, dim3(jx, js.slices), kThreads, 0, st, p, js.cols, js.subs);
}

template <typename T, typename Id>
cudaError_t launch_backward(EmbedParams p, size_t cleared, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(p.used, 0, cleared, st);
  if (e != cudaSuccess) return e;
  const int passes = embed_passes(p.rows);
  const bool small = p.n <= kSortTile, scan = p.sort_tiles > kFewTiles;
  Fill fill;
  fill.all = (small ? 0 : passes * (scan ? 2 : 1) * kSortShare) + kSumShare + (p.pieces > 1 ? kJoinShare : 0);
  p.in = 0;
  if (small) embed_small_sort_kernel<Id><<<1, kThreads, 0, st>>>(p, passes);
  else embed_keys_kernel<Id><<<(unsigned)p.sort_tiles, kThreads, 0, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  for (int pass = 0; pass < passes && !small; ++pass) {
    p.shift = 8 * pass;
    p.next_hist = pass + 1 < passes ? p.hist + (int64_t)kBins * p.sort_tiles : nullptr;
    if (scan) {
      const unsigned grid = fill.take(p, kSortShare, 1);
      if ((e = launch_next(embed_scan_kernel, grid, kThreads, 0, st, p)) != cudaSuccess) return e;
    }
    const unsigned grid = fill.take(p, kSortShare, p.sort_tiles);
    auto* scatter = scan ? embed_scatter_kernel<true> : embed_scatter_kernel<false>;
    if ((e = launch_next(scatter, grid, kThreads, 0, st, p)) != cudaSuccess) return e;
    p.hist = p.next_hist;
    p.in ^= 1;
  }
  switch (row_vec(sizeof(T), p.D, {p.dout})) {
    case 8:
      if constexpr (sizeof(T) == 2) return launch_sum<T, 8>(p, fill, st);
    case 4: return launch_sum<T, 4>(p, fill, st);
    case 2: return launch_sum<T, 2>(p, fill, st);
    default: return launch_sum<T, 1>(p, fill, st);
  }
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status embedding_forward(const void* ids, int32_t ids_bits, int64_t n, const void* table,
                             int64_t vocab, int64_t dim, int32_t io_dtype, float scale, void* out,
                             void* stream) {
  const ssd_status bad = check_sizes(n, vocab, dim);
  if (bad != SSD_OK) return bad;
  if ((ids_bits != 32 && ids_bits != 64) || (io_dtype != SSD_F32 && io_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  const bool bf16 = io_dtype == SSD_BF16;
  const size_t e = bf16 ? 2 : 4;
  if (n > 0 && (!ids || !table || !out)) return SSD_ERR_INVALID_ARG;
  if (misaligned(ids, ids_bits / 8) || misaligned(table, e) || misaligned(out, e))
    return SSD_ERR_INVALID_ARG;
  if (n == 0) return SSD_OK;
  if (too_wide(dim, row_vec(e, dim, {table, out}))) return SSD_ERR_UNSUPPORTED;
  auto f = bf16 ? (ids_bits == 64 ? launch_forward<__nv_bfloat16, int64_t> : launch_forward<__nv_bfloat16, int32_t>)
                : (ids_bits == 64 ? launch_forward<float, int64_t> : launch_forward<float, int32_t>);
  return done(f(ids, n, table, vocab, dim, scale, out, static_cast<cudaStream_t>(stream)));
}

size_t embedding_backward_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  return check_sizes(n, vocab, dim) == SSD_OK ? embed_layout(n, vocab, dim).total : 0;
}

ssd_status embedding_backward(const void* ids, int32_t ids_bits, int64_t n, const void* dout,
                              int64_t vocab, int64_t dim, int32_t io_dtype, float scale,
                              float* dtable, void* workspace, size_t workspace_bytes,
                              void* stream) {
  const ssd_status bad = check_sizes(n, vocab, dim);
  if (bad != SSD_OK) return bad;
  if ((ids_bits != 32 && ids_bits != 64) || (io_dtype != SSD_F32 && io_dtype != SSD_BF16))
    return SSD_ERR_INVALID_ARG;
  const bool bf16 = io_dtype == SSD_BF16;
  if (!dtable || (n > 0 && (!ids || !dout))) return SSD_ERR_INVALID_ARG;
  if (misaligned(ids, ids_bits / 8) || misaligned(dout, bf16 ? 2 : 4) || misaligned(dtable, 4))
    return SSD_ERR_INVALID_ARG;
  // the join of partial f32 rows, of more than one piece, may have narrower vectors than the sums
  if (n > 0 && (too_wide(dim, row_vec(bf16 ? 2 : 4, dim, {dout})) ||
                (embed_layout(n, vocab, dim).pieces > 1 && too_wide(dim, row_vec(4, dim, {})))))
    return SSD_ERR_UNSUPPORTED;
  if (!workspace || misaligned(workspace, kWsAlign) ||
      workspace_bytes < embedding_backward_workspace_bytes(n, vocab, dim))
    return SSD_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n == 0)
    return done(cudaMemsetAsync(dtable, 0, sizeof(float) * (size_t)(vocab * dim), st));
  const EmbedLayout L = embed_layout(n, vocab, dim);
  char* ws = static_cast<char*>(workspace);
  EmbedParams p;
  memset(&p, 0, sizeof(p));
  p.ids = ids;
  p.n = n;
  p.rows = vocab;
  p.D = dim;
  p.dout = dout;
  p.scale = scale;
  p.dtable = dtable;
  p.used = reinterpret_cast<uint8_t*>(ws + L.used);
  for (int k = 0; k < 2; ++k) {
    p.key[k] = reinterpret_cast<uint32_t*>(ws + L.key[k]);
    p.pos[k] = reinterpret_cast<uint32_t*>(ws + L.pos[k]);
  }
  p.hist = reinterpret_cast<uint32_t*>(ws + L.hist);
  p.head = reinterpret_cast<float*>(ws + L.head);
  p.tail = reinterpret_cast<float*>(ws + L.tail);
  p.sort_tiles = (int32_t)L.sort_tiles;
  p.piece = L.piece;
  p.pieces = L.pieces;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  auto f = bf16 ? (ids_bits == 64 ? launch_backward<__nv_bfloat16, int64_t> : launch_backward<__nv_bfloat16, int32_t>)
                : (ids_bits == 64 ? launch_backward<float, int64_t> : launch_backward<float, int32_t>);
  return done(f(p, L.cleared, st));
}

}  // extern "C"
