// Gated delta rule on the tensor cores, bf16 inputs, chunk by chunk of 64 steps (declarations in include/ssdscan.h).
// With D_i the decay from the chunk's start to step i, E_i that behind it, M_ij between, S the state before the chunk:
//   A_ij = beta_i M_ij (k_i . k_j), j < i;   T = (I + A)^-1 diag(beta)
//   U = T (V - diag(D) K S^T)                          the writes of all steps: the triangular system solved
//   y = scale (diag(D) Q S^T + (M o Q K^T) U);   S' = D_last S + (diag(E) U)^T K
// Two kernels.  T and P = scale M o Q K^T do not depend on the state: delta_chunk_kernel makes them for all chunks in
// parallel.  delta_chain_kernel walks a sequence's chunks with its state on chip, one block a head and 128 values, in
// transposed form: values are the 128 lanes of TMEM, so that what one product leaves in an accumulator is, after
// scaling, the next product's A operand in TMEM, without a trip through shared memory.
// Operands that are computed (S, U, T, P and what lies between) enter a product as two bf16 terms, hi and lo: products
// with an input take two passes, between two computed ones three (lo lo is left out, 2^-18).  One term would leave
// states and outputs off by 3e-3.  States are kept in fp32 registers and products added to them there: the tensor
// core's own accumulation truncates, which over a long memory would show.
// Measured: 8 x 4096 x 16 heads of 128 x 128 with their states, 346 us; the chunk kernel takes 112 us of it, the walk 204
// to 232, 3.4 us a chunk; with 16 sequences alone on the machine a chunk takes 2.3.  The chunk kernel is bound by no unit
// (8 x 1024: issue slots 44 %, shared memory 49 %, DRAM 33 %) but by barriers and latencies.
#include <cudaTypedefs.h>
#include <string.h>

#include <algorithm>

#include "delta_tc.cuh"
#include "launch.h"
#include "tensor_map.h"

namespace ssd {
namespace {

using namespace delta;

// ---------------------------------------------------------------------------------------------------------------------
// T and P of every chunk and head.  One product stacks K on Q (128 rows) against K: rows 0..63 are K K^T, the others
// Q K^T; both are of the key head, the heads that share it take turns with their own decays and betas.
// ---------------------------------------------------------------------------------------------------------------------
constexpr int kPrepThreads = 128;
constexpr int kPitch = 72;   // rows of 16-by-8 fragments on different banks

template <int KB>
struct PrepSmem {
  union {
    uint8_t kq[KB * 2 * kTileBytes];   // blocks of 64 keys: 64 rows of K, 64 of Q; done with once the product is
    struct {
      float a[kChunk][kPitch], x[kChunk][kPitch];
    };
  };
  ChunkDecay c;
  uint64_t loaded, done;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

using Square = float[kChunk][kPitch];

// 16 x 8 of the product of a's rows from r, columns from k, with b's rows from m, columns from n, over 16 of them; a warp,
// in two bf16 terms.  These blocks are too small for a tcgen05 tile of 128 rows.
__device__ __forceinline__ void block_product(float (&acc)[4], const Square& a, int r, int k, const Square& b, int m, int n) {
  const int g = (threadIdx.x & 31) >> 2, t = (threadIdx.x & 3) * 2;
  uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = *reinterpret_cast<const float2*>(&a[r + g + (e & 1) * 8][k + t + (e >> 1) * 8]);
    split2(v.x, v.y, ah[e], al[e]);
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) split2(b[m + t + e * 8][n + g], b[m + t + 1 + e * 8][n + g], bh[e], bl[e]);
  mma16(acc, ah, bh);
  mma16(acc, ah, bl);
  mma16(acc, al, bh);
}
__device__ __forceinline__ void store_block(Square& to, int r, int n, const float (&v)[4], float sign) {
  const int g = (threadIdx.x & 31) >> 2, t = (threadIdx.x & 3) * 2;
  *reinterpret_cast<float2*>(&to[r + g][n + t]) = make_float2(sign * v[0], sign * v[1]);
  *reinterpret_cast<float2*>(&to[r + g + 8][n + t]) = make_float2(sign * v[2], sign * v[3]);
}

// (I + A)^-1 on and below the diagonal of `x`, for A strictly below the diagonal of `a`: the 16 x 16 blocks on the
// diagonal by forward substitution in fp32, a column a lane, then pairs of blocks by X21 = -X22 (A21 X11), whose inner
// product waits above the diagonal of `a`.  All four warps.  (Every column by forward substitution, 64 rows one after
// the other: the whole kernel took 298 us for 8 x 4096 x 16 heads; the pairs by fp32 loops 164 us.)
__device__ __forceinline__ void invert(Square& a, Square& x) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d0 = warp * 16;
  if (lane < 16) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
      for (int m = 0; m < i; m += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&a[d0 + i][d0 + m]);
        s0 = fmaf(-f.x, v[m], s0);
        if (m + 1 < i) s1 = fmaf(-f.y, v[m + 1], s1);
        if (m + 2 < i) s0 = fmaf(-f.z, v[m + 2], s0);
        if (m + 3 < i) s1 = fmaf(-f.w, v[m + 3], s1);
      }
      v[i] = s0 + s1;
      x[d0 + i][d0 + lane] = v[i];
    }
  } else if ((warp & 1) == 0) {   // above the diagonal, for the products to come
#pragma unroll
    for (int i = 0; i < 16; ++i) x[d0 + i][d0 + lane] = 0.f;
  }
  __syncthreads();
  {   // two pairs of blocks of 16, eight columns a warp
    const int r = (warp >> 1) * 32, n = (warp & 1) * 8;
    float y[4] = {}, z[4] = {};
    block_product(y, a, r + 16, r, x, r, r + n);
    store_block(a, r, r + 16 + n, y, 1.f);
    __syncwarp();   // a warp's product needs its own columns alone
    block_product(z, x, r + 16, r + 16, a, r, r + 16 + n);
    store_block(x, r + 16, r + n, z, -1.f);
  }
  __syncthreads();
  {   // one pair of blocks of 32, eight columns a warp; blocks that are zero above a diagonal are left out
    const int n = warp * 8;
#pragma unroll
    for (int r = 0; r < 32; r += 16) {
      float y[4] = {};
      if (n < 16) block_product(y, a, 32 + r, 0, x, 0, n);
      block_product(y, a, 32 + r, 16, x, 16, n);
      store_block(a, r, 32 + n, y, 1.f);
    }
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 32; r += 16) {
      float z[4] = {};
      block_product(z, x, 32 + r, 32, a, 0, 32 + n);
      if (r > 0) block_product(z, x, 32 + r, 48, a, 16, 32 + n);
      store_block(x, 32 + r, n, z, -1.f);
    }
  }
  __syncthreads();
}

__device__ __forceinline__ void store_split_row(uint8_t* hi, uint8_t* lo, int row, const float (&v)[8], int col) {
  uint4 h, l;
  split2(v[0], v[1], h.x, l.x);
  split2(v[2], v[3], h.y, l.y);
  split2(v[4], v[5], h.z, l.z);
  split2(v[6], v[7], h.w, l.w);
  *reinterpret_cast<uint4*>(hi + sw128_off16(row, col)) = h;
  *reinterpret_cast<uint4*>(lo + sw128_off16(row, col)) = l;
}

// Two tiles on their way from shared memory in one copy, read when this returns.  (Rows of 128 bytes straight from the
// registers, a lane a row, kept the memory pipe at 60 % with 20 % of instructions: 118 us instead of 110 for
// 8 x 4096 x 16 heads.)
__device__ __forceinline__ void send_tiles(uint8_t* to, const void* from) {
  fence_proxy_async_smem();
  __syncthreads();
  if (threadIdx.x == 0) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(smem_u32(from)),
                 "r"(2 * kTileBytes)
                 : "memory");
    bulk_commit_group();
    bulk_wait_group_read<0>();
  }
  __syncthreads();
}

template <int KB>
__global__ void __launch_bounds__(kPrepThreads, 6) delta_chunk_kernel(const __grid_constant__ Params p,
                                                                   const __grid_constant__ TcMaps m, TcBuffers buf) {
  extern __shared__ __align__(1024) uint8_t raw[];
  PrepSmem<KB>& sm = *reinterpret_cast<PrepSmem<KB>*>(raw);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x / 32), 0), lane = threadIdx.x % 32;
  int64_t id = blockIdx.x;
  const int64_t hk = id % p.Hk;
  id /= p.Hk;
  const int64_t chunk = id % p.nch, b = id / p.nch, t0 = chunk * kChunk, group = p.H / p.Hk;
  const int n = (int)min((int64_t)kChunk, p.T - t0);
  if (threadIdx.x == 0) {
    mbar_init(&sm.loaded, 1);
    mbar_init(&sm.done, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem, 64);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  bool ok = true;
  if (warp == 1) chunk_decay_warp(p, sm.c, b, t0, n, hk * group, lane);
  if (warp == 0) {
    mbar_arrive_expect_tx_elect(&sm.loaded, KB * 2 * kTileBytes);
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      tma_load_4d_elect(sm.kq + kb * 2 * kTileBytes, &m.k, &sm.loaded, kb * 64, (int)t0, (int)hk, (int)b);
      tma_load_4d_elect(sm.kq + (kb * 2 + 1) * kTileBytes, &m.q, &sm.loaded, kb * 64, (int)t0, (int)hk, (int)b);
    }
    ok = wait_bar(&sm.loaded, 0, &sm.abort, p.hdr, 1);
    if (ok) {
      const uint32_t lo = sdesc_sw128_lo(smem_u32(sm.kq), 0);
#pragma unroll
      for (int ks = 0; ks < KB * 4; ++ks) {
        const uint32_t at = lo + (((ks >> 2) * 2 * kTileBytes + (ks & 3) * 32) >> 4);
        mma_ss_we(tmem, at, kDHi, at, kDHi, idesc_bf16(128, 64, 0, 0), ks > 0);
      }
    }
    if (ok) mma_commit_elect(&sm.done);   // else every wait for it ends by the abort flag
  }
  // All warps go on, or none: one wait may give up as another one's barrier completes.
  const bool done = !__syncthreads_or(!wait_bar(&sm.done, 0, &sm.abort, p.hdr, 2));
  if (!done && warp == 0) {   // what this block has on its way
    mbar_wait_bounded(&sm.loaded, 0, kDrainNs);
    if (ok) mbar_wait_bounded(&sm.done, 0, kDrainNs);
  }
  tc_fence_after();
  const int row = (warp & 1) * 32 + lane;
  const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);
  for (int64_t h = hk * group; done && h < (hk + 1) * group; ++h) {
    const int64_t cell = (b * p.nch + chunk) * p.H + h;
    if (!SSD_INDEX_OK(p.hdr, cell, p.batch * p.nch * p.H, 2011)) break;
    uint8_t* out = buf.squares + cell * buf.square;
    __syncthreads();
    if (h > hk * group) {
      if (warp == 1) chunk_decay_warp(p, sm.c, b, t0, n, h, lane);
      __syncthreads();
    }
    float* decays = buf.decays + cell * kDecays;
    if (threadIdx.x < kChunk) {
      decays[threadIdx.x] = sm.c.from[threadIdx.x];
      decays[2 * kChunk + threadIdx.x] = sm.c.beta[threadIdx.x];
      decays[3 * kChunk + threadIdx.x] = sm.c.from[threadIdx.x] * p.scale;
    } else {
      decays[threadIdx.x] = sm.c.to[threadIdx.x - kChunk];
    }
    const float hi = sm.c.hi[row], lo = sm.c.lo[row];
    const float by = warp < 2 ? sm.c.beta[row] : p.scale, by_from = by * sm.c.from[row];
    const int last = warp < 2 ? row - 1 : row;   // the strict part of A, P with its diagonal
    const bool plain = sm.c.plain;
#pragma unroll 1
    for (int c0 = 0; c0 < kChunk; c0 += 16) {
      float v[16];
      if ((warp & 1) * 32 + 31 < c0) {   // above the diagonal
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
      } else {
        tmem_ld16(mine + c0, v);
        tmem_ld_wait();
        reg_tie(v);
        if (plain) {
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&sm.c.back[c0 + j]);
            v[j] = c0 + j <= last ? v[j] * (by_from * f.x) : 0.f;
            v[j + 1] = c0 + j + 1 <= last ? v[j + 1] * (by_from * f.y) : 0.f;
            v[j + 2] = c0 + j + 2 <= last ? v[j + 2] * (by_from * f.z) : 0.f;
            v[j + 3] = c0 + j + 3 <= last ? v[j + 3] * (by_from * f.w) : 0.f;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            v[j] = c0 + j <= last ? v[j] * by * expf((hi - sm.c.hi[c0 + j]) + (lo - sm.c.lo[c0 + j])) : 0.f;
        }
      }
      if (warp < 2) {
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          *reinterpret_cast<float4*>(&sm.a[row][c0 + j]) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      } else {
        uint8_t* to = reinterpret_cast<uint8_t*>(sm.x);   // P's place until it has left
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = v[half * 8 + j];
          store_split_row(to, to + kTileBytes, row, w, c0 + half * 8);
        }
      }
    }
    send_tiles(out + 2 * kTileBytes, sm.x);
    invert(sm.a, sm.x);
    // rows of T by two threads each, over A
    const int r = threadIdx.x & 63, first = threadIdx.x >> 6 << 5;
    uint8_t* to = reinterpret_cast<uint8_t*>(sm.a);
    for (int with_beta = 1; with_beta >= (buf.square > square_bytes(false) ? 0 : 1); --with_beta) {   // and without, for the walk back
#pragma unroll
      for (int c = first; c < first + 32; c += 8) {
        const float4 f = *reinterpret_cast<const float4*>(&sm.x[r][c]), g = *reinterpret_cast<const float4*>(&sm.x[r][c + 4]);
        float w[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = c + j <= r ? (with_beta ? w[j] * sm.c.beta[c + j] : w[j]) : 0.f;
        store_split_row(to, to + kTileBytes, r, w, c);
      }
      send_tiles(with_beta ? out : out + 4 * kTileBytes, sm.a);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 64);
}

// ---------------------------------------------------------------------------------------------------------------------
// The walk.  TMEM columns: the state's two terms, X = S K^T and after it -D X's two terms, U's accumulator and after it
// U's two terms, E U's two terms, (E U)^T K, y.  Every 16 columns keep hi then lo of themselves, so that a warp that
// has read them may write its terms over them.
// ---------------------------------------------------------------------------------------------------------------------
constexpr uint32_t kColS = 0, kColX = 128, kColU = 192, kColW = 256, kColD = 320, kColO = 448;

template <int KB>
struct Stage {
  uint8_t k[KB * kTileBytes], q[KB * kTileBytes], v[2 * kTileBytes], t[2 * kTileBytes], p[2 * kTileBytes];
  float from[kChunk], to[kChunk], beta[kChunk], scaled[kChunk];
};
struct ChainBars {
  uint64_t full[2], empty[2], s_ready[4], x_full, r_ready, u_full, w_ready, u_ready, d_full, o1_full, o_scaled, o2_full,
      o_free, drain;
};
template <int KB>
struct ChainSmem {
  Stage<KB> st[2];
  uint8_t y[2 * kTileBytes];
  uint8_t s[4][128 * 64];   // 128 rows of 16 keys of the state on their way out, for each quarter of the keys
  ChainBars bar;
  uint32_t tmem;
  int abort;
};

// kY: with the outputs; without them Q, P and the products with them are left out.
template <int KB, bool kY>
__global__ void __launch_bounds__(kWalkThreads, 1)
    delta_chain_kernel(const __grid_constant__ Params p, const __grid_constant__ TcMaps m, TcBuffers buf, int vtiles,
                       Segments seg) {
  extern __shared__ __align__(1024) uint8_t raw[];
  ChainSmem<KB>& sm = *reinterpret_cast<ChainSmem<KB>*>(raw);
  ChainBars& bar = sm.bar;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x / 32), 0), lane = threadIdx.x % 32;
  const int real = seg.pre ? seg.n - 1 : seg.n;   // segments with values of a sequence
  const int per = real * vtiles + (seg.pre ? seg.n - 2 : 0), seq = blockIdx.x / per, job = blockIdx.x % per;
  const bool identity = job >= real * vtiles;
  const int part_of = identity ? 1 + job - real * vtiles : job / vtiles, v0 = identity ? 0 : job % vtiles * 128;
  const int h = seq % (int)p.H, b = seq / (int)p.H, hk = h / (int)(p.H / p.Hk);
  const int first = part_of * seg.chunks, all_chunks = (int)p.nch, nch = min(seg.chunks, all_chunks - first);
  const int64_t seg_at = (int64_t)seq * seg.n + part_of;
  constexpr int Kp = KB * 64;
  volatile int* abort = &sm.abort;
  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], 1);
    }
    for (uint64_t* four : {&bar.s_ready[0], &bar.s_ready[1], &bar.s_ready[2], &bar.s_ready[3], &bar.o_scaled, &bar.o_free})
      mbar_init(four, 4);
    for (uint64_t* one : {&bar.x_full, &bar.u_full, &bar.d_full, &bar.o1_full, &bar.o2_full, &bar.drain}) mbar_init(one, 1);
    for (uint64_t* all : {&bar.r_ready, &bar.w_ready, &bar.u_ready}) mbar_init(all, kStateWarps);
    fence_mbar_init();
  }
  if (warp == 20) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;

  if (warp == 21) {   // loads
    int issued = 0;
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      if (c >= 2 && !wait_bar(&bar.empty[s], ((c >> 1) - 1) & 1, abort, p.hdr, 10)) break;
      Stage<KB>& st = sm.st[s];
      const int64_t cell = ((int64_t)b * all_chunks + first + c) * p.H + h;
      const int t0 = (first + c) * kChunk;
      mbar_arrive_expect_tx_elect(&bar.full[s], ((kY ? 2 * KB + 4 : KB + 2) + (identity ? 0 : 2)) * kTileBytes + kDecayBytes);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        tma_load_4d_elect(st.k + kb * kTileBytes, &m.k, &bar.full[s], kb * 64, t0, hk, b);
        if (kY) tma_load_4d_elect(st.q + kb * kTileBytes, &m.q, &bar.full[s], kb * 64, t0, hk, b);
      }
      if (!identity) {
        tma_load_4d_elect(st.v, &m.v, &bar.full[s], v0, t0, h, b);
        tma_load_4d_elect(st.v + kTileBytes, &m.v, &bar.full[s], v0 + 64, t0, h, b);
      }
      bulk_load_elect(st.t, buf.squares + cell * buf.square, (kY ? 4 : 2) * kTileBytes, &bar.full[s]);
      bulk_load_elect(st.from, buf.decays + cell * kDecays, kDecayBytes, &bar.full[s]);
      issued = c + 1;
    }
    bool drained = true;   // nothing may still be written to this block's shared memory when it ends
    for (int s = 0; s < 2; ++s) {
      const int loads = issued > s ? (issued - 1 - s) / 2 + 1 : 0;
      if (loads > 0) drained &= mbar_wait_bounded(&bar.full[s], (loads - 1) & 1, kDrainNs);
    }
    if (!drained && lane == 0) latch_error(p.hdr, SSD_ERR_TIMEOUT, 11);
  } else if (warp == 20) {   // products
    constexpr uint32_t id_k = idesc_bf16(128, 64, 0, 0), id_v = idesc_bf16(128, 64, 1, 0), id_d = idesc_bf16(128, Kp, 0, 1);
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      const uint32_t par = c & 1;
      Stage<KB>& st = sm.st[s];
      const uint32_t k_lo = sdesc_sw128_lo(smem_u32(st.k), 0), q_lo = sdesc_sw128_lo(smem_u32(st.q), 0);
      const uint32_t km_lo = sdesc_sw128_lo(smem_u32(st.k), kTileBytes), v_lo = sdesc_sw128_lo(smem_u32(st.v), kTileBytes);
      const uint32_t t_lo = sdesc_sw128_lo(smem_u32(st.t), 0), p_lo = sdesc_sw128_lo(smem_u32(st.p), 0);
      if (!wait_bar(&bar.full[s], (c >> 1) & 1, abort, p.hdr, 12)) break;
      // X = S K^T, a quarter of the keys as soon as its terms are there
      bool ready = true;
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        ready = ready && wait_bar(&bar.s_ready[part], par, abort, p.hdr, 13);
        if (!ready) break;
        tc_fence_after();
#pragma unroll
        for (int ks = part * KB; ks < (part + 1) * KB; ++ks) {
          const uint32_t at = k_lo + (((ks >> 2) * kTileBytes + (ks & 3) * 32) >> 4);
          mma_ts_we(tmem + kColX, tmem + kColS + ks * 8, at, kDHi, id_k, ks > 0);
          mma_ts_we(tmem + kColX, tmem + kColS + Kp / 2 + ks * 8, at, kDHi, id_k, 1);
        }
      }
      if (!ready) break;
      mma_commit_elect(&bar.x_full);
      // U = V T^T - (D X) T^T
      if (kY && c > 0 && !wait_bar(&bar.o2_full, (c - 1) & 1, abort, p.hdr, 14)) break;   // U's terms have been read
      if (!identity) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          mma_ss_we(tmem + kColU, v_lo + ks * (2048 >> 4), kDHi, t_lo + ks * 2, kDHi, id_v, ks > 0);
          mma_ss_we(tmem + kColU, v_lo + ks * (2048 >> 4), kDHi, t_lo + kLo + ks * 2, kDHi, id_v, 1);
        }
      }
      if (!wait_bar(&bar.r_ready, par, abort, p.hdr, 15)) break;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint32_t a = tmem + kColX + ks * 16;
        mma_ts_we(tmem + kColU, a, t_lo + ks * 2, kDHi, id_k, ks > 0 || !identity);
        mma_ts_we(tmem + kColU, a, t_lo + kLo + ks * 2, kDHi, id_k, 1);
        mma_ts_we(tmem + kColU, a + 8, t_lo + ks * 2, kDHi, id_k, 1);
      }
      mma_commit_elect(&bar.u_full);
      if constexpr (kY) {   // S Q^T, while U is turned into operands
        if (c > 0 && !wait_bar(&bar.o_free, (c - 1) & 1, abort, p.hdr, 16)) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < KB * 4; ++ks) {
          const uint32_t at = q_lo + (((ks >> 2) * kTileBytes + (ks & 3) * 32) >> 4);
          mma_ts_we(tmem + kColO, tmem + kColS + ks * 8, at, kDHi, id_k, ks > 0);
          mma_ts_we(tmem + kColO, tmem + kColS + Kp / 2 + ks * 8, at, kDHi, id_k, 1);
        }
        mma_commit_elect(&bar.o1_full);
      }
      // (E U)^T K
      if (!wait_bar(&bar.w_ready, par, abort, p.hdr, 17)) break;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint32_t a = tmem + kColW + ks * 16;
        mma_ts_we(tmem + kColD, a, km_lo + ks * (2048 >> 4), kDHi, id_d, ks > 0);
        mma_ts_we(tmem + kColD, a + 8, km_lo + ks * (2048 >> 4), kDHi, id_d, 1);
      }
      mma_commit_elect(&bar.d_full);
      if constexpr (kY) {   // y = scale D S Q^T + U P^T
        if (!wait_bar(&bar.u_ready, par, abort, p.hdr, 18)) break;
        if (!wait_bar(&bar.o_scaled, par, abort, p.hdr, 19)) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t a = tmem + kColU + ks * 16;
          mma_ts_we(tmem + kColO, a, p_lo + ks * 2, kDHi, id_k, 1);
          mma_ts_we(tmem + kColO, a, p_lo + kLo + ks * 2, kDHi, id_k, 1);
          mma_ts_we(tmem + kColO, a + 8, p_lo + ks * 2, kDHi, id_k, 1);
        }
        mma_commit_elect(&bar.o2_full);
      }
      mma_commit_elect(&bar.empty[s]);
    }
    mma_commit_elect(&bar.drain);
    if (!mbar_wait_bounded(&bar.drain, 0, kDrainNs) && lane == 0) latch_error(p.hdr, SSD_ERR_TIMEOUT, 20);
  } else if (warp < kStateWarps) {   // the state, and the operands on the way to the next one
    constexpr int KQ = Kp / 4;
    const int part = warp >> 2, row = v0 + (warp & 3) * 32 + lane, k0 = part * KQ, j0 = part * 16;
    const bool live = row < (identity ? p.K : p.V);
    const int64_t at = (int64_t)row * p.K + k0, KV = p.K * p.V;
    const float* init = identity ? nullptr : part_of == 0 ? (p.init ? p.init + seq * KV : nullptr)
                        : seg.pre ? nullptr : seg.start + seg_at * KV;
    float S[KQ];
    // By vectors, each chosen where it is loaded.  (Us for 8 x 4096, 1 x 32768 and 16 x 64 steps of 16 heads of 128 x 128:
    // 345, 513, 35; value by value 354, 536, 56; zeros first and loads over them 335, 551, 37.)
#pragma unroll
    for (int k = 0; k < KQ; k += 4) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (init && live && k0 + k < p.K) {
        if ((reinterpret_cast<uintptr_t>(init) & 15) == 0) f = *reinterpret_cast<const float4*>(init + at + k);
        else f = make_float4(init[at + k], init[at + k + 1], init[at + k + 2], init[at + k + 3]);
      } else if (identity) {
        const int one = row - k0 - k;
        f = make_float4(one == 0, one == 1, one == 2, one == 3);
      }
      S[k] = f.x;
      S[k + 1] = f.y;
      S[k + 2] = f.z;
      S[k + 3] = f.w;
    }
    const bool keep = p.states_out && !seg.pre;
    bool on = true;   // after a wait that gave up, without waiting: the quarter's warps meet at its barrier
    int cell = (b * all_chunks + first) * (int)p.H + h;
    for (int c = 0; c < nch; ++c, cell += (int)p.H) {
      const int s = c & 1;
      const uint32_t par = c & 1;
      const Stage<KB>& st = sm.st[s];
      store_state_terms(tmem + lanes + kColS + k0 / 2, Kp / 2, S);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.s_ready[part]);
      if (keep) send_state(sm.s[part], &m.states, S, part, 0, v0, cell, p.K);
      on = on && wait_bar(&bar.full[s], (c >> 1) & 1, abort, p.hdr, 21);   // the decays
      const float all = st.from[kChunk - 1];
      on = on && wait_bar(&bar.x_full, par, abort, p.hdr, 22);
      tc_fence_after();
      float x[16];
      tmem_ld16(tmem + lanes + kColX + j0, x);
      tmem_ld_wait();
      reg_tie(x);
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&st.from[j0 + j]);
        x[j] *= -f.x;
        x[j + 1] *= -f.y;
        x[j + 2] *= -f.z;
        x[j + 3] *= -f.w;
      }
      store_terms(tmem + lanes + kColX + j0, x);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.r_ready);
      if constexpr (KB == 2)
        if (keep) send_state(sm.s[part], &m.states, S, part, KQ / 2, v0, cell, p.K);
      on = on && wait_bar(&bar.u_full, par, abort, p.hdr, 23);
      tc_fence_after();
      tmem_ld16(tmem + lanes + kColU + j0, x);
      tmem_ld_wait();
      reg_tie(x);
      {
        uint32_t u[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&st.to[j0 + j]);
          split2(x[j] * f.x, x[j + 1] * f.y, u[j / 2], u[8 + j / 2]);
          split2(x[j + 2] * f.z, x[j + 3] * f.w, u[j / 2 + 1], u[8 + j / 2 + 1]);
        }
        tmem_st16u(tmem + lanes + kColW + j0, u);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.w_ready);
      if constexpr (kY) {
        store_terms(tmem + lanes + kColU + j0, x);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.u_ready);
      }
      on = on && wait_bar(&bar.d_full, par, abort, p.hdr, 24);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < KQ; k += 16) {
        tmem_ld16(tmem + lanes + kColD + k0 + k, x);
        tmem_ld_wait();
        reg_tie(x);
#pragma unroll
        for (int j = 0; j < 16; ++j) S[k + j] = fmaf(all, S[k + j], x[j]);
      }
    }
    if ((threadIdx.x & 127) == 0) bulk_wait_group<0>();
    float* end = seg.pre ? (identity ? seg.map + seg_at * p.K * p.K : seg.end + seg_at * KV)
                 : part_of == seg.n - 1 && p.final_state ? p.final_state + seq * KV : nullptr;
    if (end && live && on) {
      const bool wide = (reinterpret_cast<uintptr_t>(end) & 31) == 0;
#pragma unroll
      for (int k = 0; k < KQ; k += 8)
        if (k0 + k < p.K &&
            SSD_INDEX_OK(p.hdr, at + k + 7, identity ? p.K * p.K : KV, 2012) &&
            SSD_INDEX_OK(p.hdr, seg.pre ? seg_at : seq, p.batch * p.H * (seg.pre ? seg.n : 1), 2013))
          store8(end + at + k, S + k, wide);
    }
  } else if constexpr (kY) {   // y: a thread has a value
    const int v = (warp & 3) * 32 + lane;
    uint8_t* column = sm.y + (v >> 6) * kTileBytes;
    bool on = true;   // as above
    for (int c = 0; c < nch; ++c) {
      const int s = c & 1;
      const uint32_t par = c & 1;
      const Stage<KB>& st = sm.st[s];
      on = on && wait_bar(&bar.full[s], (c >> 1) & 1, abort, p.hdr, 25);
      on = on && wait_bar(&bar.o1_full, par, abort, p.hdr, 26);
      tc_fence_after();
      // 16 columns at a time: with more the kernel's 80 registers spill, and a reload from beyond the L1 stalls the walk
#pragma unroll 1
      for (int j0 = 0; j0 < kChunk; j0 += 16) {
        float o[16];
        tmem_ld16(tmem + lanes + kColO + j0, o);
        tmem_ld_wait();
        reg_tie(o);
        uint32_t u[16];
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&st.scaled[j0 + j]);
          u[j] = __float_as_uint(o[j] * f.x);
          u[j + 1] = __float_as_uint(o[j + 1] * f.y);
          u[j + 2] = __float_as_uint(o[j + 2] * f.z);
          u[j + 3] = __float_as_uint(o[j + 3] * f.w);
        }
        tmem_st16u(tmem + lanes + kColO + j0, u);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.o_scaled);
      if (warp == kStateWarps && lane == 0) bulk_wait_group_read<0>();   // the last chunk's rows have left
      named_barrier(1, 128);
      on = on && wait_bar(&bar.o2_full, par, abort, p.hdr, 27);
      tc_fence_after();
#pragma unroll 1
      for (int j0 = 0; j0 < kChunk; j0 += 16) {
        float o[16];
        tmem_ld16(tmem + lanes + kColO + j0, o);
        tmem_ld_wait();
        reg_tie(o);
#pragma unroll
        for (int j = 0; j < 16; j += 2)
          store_pair(column + sw128_off16(j0 + j, v & 63), column + sw128_off16(j0 + j + 1, v & 63), o[j], o[j + 1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.o_free);
      fence_proxy_async_smem();
      named_barrier(1, 128);
      if (warp == kStateWarps && lane == 0) {
        tma_store_4d(&m.y, sm.y, v0, (first + c) * kChunk, h, b);
        if (v0 + 64 < p.V) tma_store_4d(&m.y, sm.y + kTileBytes, v0 + 64, (first + c) * kChunk, h, b);
        bulk_commit_group();
      }
    }
    if (warp == kStateWarps && lane == 0) bulk_wait_group<0>();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 20) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The state before every segment: 16 rows of a sequence a block.  A thread has a key of four rows, and of the product with
// a segment's map the sum over 32 keys for all 16; the map's values, which do not wait for the rows, are loaded a segment
// ahead.  (128 threads, each with all keys: 10 us a segment instead of 3.)
constexpr int kCarryThreads = 512, kCarryRows = 16;
struct CarrySmem {
  float row[128][kCarryRows];       // by keys: four rows a load
  float part[4][kCarryRows][128];
};

__global__ void __launch_bounds__(kCarryThreads) delta_carry_kernel(const __grid_constant__ Params p, Segments seg, int tiles) {
  __shared__ __align__(16) CarrySmem sm;
  const int seq = blockIdx.x / tiles, v0 = blockIdx.x % tiles * kCarryRows, k = threadIdx.x & 127, part = threadIdx.x >> 7;
  const int64_t KV = p.K * p.V, at = (int64_t)seq * seg.n;
  const bool in = k < p.K;
  float s[4], f[32];
  auto own = [&](const float* base, int64_t i, int r) { return base + (at + i) * KV + (v0 + part * 4 + r) * p.K + k; };
  auto fetch = [&](int i) {   // the map of segment i
    const float* map = seg.map + (at + i) * p.K * p.K + k;
#pragma unroll
    for (int e = 0; e < 32; ++e) f[e] = in && part * 32 + e < p.K && i + 1 < seg.n ? map[(part * 32 + e) * p.K] : 0.f;
  };
  fetch(1);
#pragma unroll
  for (int r = 0; r < 4; ++r) s[r] = in && v0 + part * 4 + r < p.V ? *own(seg.end, 0, r) : 0.f;
  for (int i = 1; i < seg.n; ++i) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (in && v0 + part * 4 + r < p.V &&
          SSD_INDEX_OK(p.hdr, own(seg.start, i, r) - seg.start, p.batch * p.H * seg.n * KV, 2014))
        *const_cast<float*>(own(seg.start, i, r)) = s[r];
    if (i + 1 == seg.n) break;
    *reinterpret_cast<float4*>(&sm.row[k][part * 4]) = make_float4(s[0], s[1], s[2], s[3]);
#pragma unroll
    for (int r = 0; r < 4; ++r) s[r] = in && v0 + part * 4 + r < p.V ? *own(seg.end, i, r) : 0.f;
    __syncthreads();
    float sum[kCarryRows] = {};
#pragma unroll
    for (int e = 0; e < 32; ++e)
#pragma unroll
      for (int r = 0; r < kCarryRows; r += 4) {
        const float4 g = *reinterpret_cast<const float4*>(&sm.row[part * 32 + e][r]);
        sum[r] = fmaf(g.x, f[e], sum[r]);
        sum[r + 1] = fmaf(g.y, f[e], sum[r + 1]);
        sum[r + 2] = fmaf(g.z, f[e], sum[r + 2]);
        sum[r + 3] = fmaf(g.w, f[e], sum[r + 3]);
      }
    fetch(i + 1);
#pragma unroll
    for (int r = 0; r < kCarryRows; ++r) sm.part[part][r][k] = sum[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) s[r] += sm.part[q][part * 4 + r][k];
  }
}

// ------------------------------------------------------------------------------------------------ host
constexpr int kSms = 152, kMostSegments = 16;

// Segments of a sequence, by what the passes take: a chunk 2.5 us with outputs, 2.3 us without (2.4 and 2.2 measured at
// 86 chunks), blocks in rounds of one an SM, a segment's carry 3 us.  (1 x 32768 x 16 heads: 1261 us in one segment, 513
// us in six.)
int segments_for(int64_t batch, int64_t nch, int64_t H, int64_t V) {
  const int64_t vtiles = (V + 127) / 128, seqs = batch * H;
  int best = 1;
  double least = 0;
  for (int n = 1; n <= kMostSegments && (n == 1 || seqs * vtiles * n <= 2 * kSms); ++n) {
    const int64_t len = (nch + n - 1) / n;
    if ((n - 1) * len >= nch) continue;   // the last one would be empty
    auto rounds = [](int64_t blocks) { return (double)((blocks + kSms - 1) / kSms); };
    double us = rounds(seqs * vtiles * n) * len * 2.5;
    if (n > 1) us += rounds(seqs * ((n - 1) * vtiles + n - 2)) * len * 2.3 + 3.0 * n + 15;
    if (n == 1 || us < 0.9 * least) {
      best = n;
      least = us;
    }
  }
  return best;
}
size_t segment_bytes(int64_t batch, int64_t nch, int64_t H, int64_t V, int64_t K) {
  const int n = segments_for(batch, nch, H, V);
  return n == 1 ? 0 : (size_t)(batch * H * n) * (size_t)(2 * V * K + K * K) * 4;
}

bool rows_fit(const void* base, const int64_t* stride, int64_t batch, int64_t T, int64_t heads) {
  if (reinterpret_cast<uintptr_t>(base) % 16 != 0) return false;
  const int64_t n[3] = {batch, T, heads};
  for (int a = 0; a < 3; ++a)
    if (n[a] > 1 && (stride[a] <= 0 || stride[a] % 8 != 0 || stride[a] >= (int64_t)1 << 38)) return false;
  return true;
}

template <int KB>
cudaError_t chunks_as(const Params& p, const TcMaps& m, const TcBuffers& buf, cudaStream_t st) {
  constexpr int smem = sizeof(PrepSmem<KB>);
  const cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel<KB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  delta_chunk_kernel<KB><<<(unsigned)(p.batch * p.nch * p.Hk), kPrepThreads, smem, st>>>(p, m, buf);
  return cudaGetLastError();
}

template <int KB, bool kY>
cudaError_t walk_as(const Params& p, const TcMaps& m, const TcBuffers& buf, const Segments& seg, cudaStream_t st) {
  constexpr int smem = sizeof(ChainSmem<KB>);
  static_assert(smem <= 232448, "shared memory of a block");
  const auto kernel = delta_chain_kernel<KB, kY>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int vtiles = (int)((p.V + 127) / 128), per = seg.pre ? (seg.n - 1) * vtiles + seg.n - 2 : seg.n * vtiles;
  kernel<<<(unsigned)(p.batch * p.H * per), kWalkThreads, smem, st>>>(p, m, buf, vtiles, seg);
  return cudaGetLastError();
}

template <int KB>
cudaError_t chain_as(const Params& p, const TcMaps& m, const TcBuffers& buf, float* segments, cudaStream_t st) {
  Segments seg;
  memset(&seg, 0, sizeof(seg));
  seg.n = segments_for(p.batch, p.nch, p.H, p.V);
  seg.chunks = (int)((p.nch + seg.n - 1) / seg.n);
  if (seg.n > 1) {
    const int64_t states = p.batch * p.H * seg.n * p.V * p.K;
    seg.start = segments;
    seg.end = segments + states;
    seg.map = segments + 2 * states;
    seg.pre = 1;
    cudaError_t e = walk_as<KB, false>(p, m, buf, seg, st);
    if (e != cudaSuccess) return e;
    seg.pre = 0;
    const int tiles = (int)((p.V + kCarryRows - 1) / kCarryRows);
    delta_carry_kernel<<<(unsigned)(p.batch * p.H * tiles), kCarryThreads, 0, st>>>(p, seg, tiles);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return p.y ? walk_as<KB, true>(p, m, buf, seg, st) : walk_as<KB, false>(p, m, buf, seg, st);
}

TcBuffers buffers_in(void* at, const Params& p, bool backward) {
  const size_t cells = (size_t)(p.batch * p.nch * p.H);
  TcBuffers buf;
  buf.square = square_bytes(backward);
  buf.squares = static_cast<uint8_t*>(at);
  buf.decays = reinterpret_cast<float*>(buf.squares + cells * buf.square);
  buf.writes = reinterpret_cast<uint8_t*>(buf.decays) + align_up(cells * kDecayBytes, kWsAlign);
  return buf;
}
float* segments_in(const TcBuffers& buf, const Params& p, bool backward) {
  return reinterpret_cast<float*>(buf.writes + (backward ? (size_t)(p.batch * p.nch * p.H) * 4 * kTileBytes : 0));
}

}  // namespace

namespace delta {

// Map of [batch, steps, heads, cols] in boxes of 64 steps and 64 columns of one head.
bool head_map(CUtensorMap* m, const void* base, int64_t batch, int64_t T, int64_t heads, int64_t cols, const int64_t* stride) {
  const auto encode = tensor_map_encoder();
  if (!encode || !base) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)cols, (cuuint64_t)T, (cuuint64_t)heads, (cuuint64_t)batch};
  const int64_t of[3] = {T > 1 ? stride[1] : 8, heads > 1 ? stride[2] : 8, batch > 1 ? stride[0] : 8};
  cuuint64_t strides[3];
  for (int a = 0; a < 3; ++a) {
    if (of[a] <= 0 || of[a] % 8 != 0) return false;
    strides[a] = (cuuint64_t)of[a] * 2;
  }
  const cuuint32_t box[4] = {64, 64, 1, 1}, one[4] = {1, 1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Map of [cells, V, K] f32 states in boxes of 128 values and 16 keys.
bool state_map(CUtensorMap* m, const void* base, int64_t cells, int64_t V, int64_t K) {
  const auto encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)K, (cuuint64_t)V, (cuuint64_t)cells, 1};
  const cuuint64_t strides[3] = {(cuuint64_t)K * 4, (cuuint64_t)(K * V * 4), (cuuint64_t)(K * V * 4)};
  const cuuint32_t box[4] = {16, 128, 1, 1}, one[4] = {1, 1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void*>(base), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t tc_bytes(int64_t batch, int64_t nch, int64_t H, int64_t V, int64_t K, bool backward) {
  const size_t cells = (size_t)(batch * nch * H);
  return cells * square_bytes(backward) + align_up(cells * kDecayBytes, kWsAlign) + (backward ? cells * 4 * kTileBytes : 0) +
         segment_bytes(batch, nch, H, V, K);
}

// Forward, few sequences whose rows the walk on the CUDA cores has on the machine at once: from as many steps on as
// make up for two launches (us, walk and tensor cores: 16 heads of 128 x 128, 64 steps 21 and 23, 72 steps 25 and 25, 128
// steps 37 and 25; 16 of 64 x 64, 64 steps 17 and 17, 128 steps 29 and 19).  Many: from a quarter of a chunk on (256 of
// 128 x 128, 8 steps 39 and 37, 16 steps 39 and 37, 24 steps 62 and 37).  Backward: always (16 of 128 x 128, 8 steps 56
// and 36, 128 steps 111 and 39).
bool tc_takes(const Params& p, bool backward) {
  const int64_t most = INT32_MAX / 2;
  if (p.K % 8 != 0 || p.K > 128 || p.V % 8 != 0 || p.T > most || p.batch > most) return false;
  const bool few = p.batch * p.H * ((p.V + 15) / 16) <= 2 * kSms;
  if (!backward && p.T < (few ? 72 : kChunk / 4)) return false;
  if (p.batch * p.nch * p.H >= most) return false;
  if (!rows_fit(p.q, p.qs, p.batch, p.T, p.Hk) || !rows_fit(p.k, p.ks, p.batch, p.T, p.Hk) ||
      !rows_fit(p.v, p.vs, p.batch, p.T, p.H))
    return false;
  auto on16 = [](const void* a) { return reinterpret_cast<uintptr_t>(a) % 16 == 0; };
  if (!backward) return on16(p.y) && on16(p.states_out);
  return p.V <= 128 && rows_fit(p.dy, p.ds, p.batch, p.T, p.H) && on16(p.dq) && on16(p.dk) && on16(p.dv) &&
         on16(p.states_in) && on16(p.dfinal);
}

cudaError_t tc_forward(const Params& p, void* buffers, cudaStream_t st) {
  TcMaps m;
  memset(&m, 0, sizeof(m));
  const int64_t ys[3] = {p.T * p.H * p.V, p.H * p.V, p.V};
  if (!head_map(&m.q, p.q, p.batch, p.T, p.Hk, p.K, p.qs) || !head_map(&m.k, p.k, p.batch, p.T, p.Hk, p.K, p.ks) ||
      !head_map(&m.v, p.v, p.batch, p.T, p.H, p.V, p.vs) || (p.y && !head_map(&m.y, p.y, p.batch, p.T, p.H, p.V, ys)) ||
      (p.states_out && !state_map(&m.states, p.states_out, p.batch * p.nch * p.H, p.V, p.K)))
    return cudaErrorInvalidValue;
  const TcBuffers buf = buffers_in(buffers, p, false);
  const cudaError_t e = p.K <= 64 ? chunks_as<1>(p, m, buf, st) : chunks_as<2>(p, m, buf, st);
  if (e != cudaSuccess) return e;
  float* segments = segments_in(buf, p, false);
  return p.K <= 64 ? chain_as<1>(p, m, buf, segments, st) : chain_as<2>(p, m, buf, segments, st);
}

cudaError_t tc_backward(const Params& p, bool states_known, void* buffers, cudaStream_t st) {
  TcMaps m;
  memset(&m, 0, sizeof(m));
  const int64_t ks[3] = {p.T * p.Hk * p.K, p.Hk * p.K, p.K};
  const int64_t cells = p.batch * p.nch * p.H;
  if (!head_map(&m.q, p.q, p.batch, p.T, p.Hk, p.K, p.qs) || !head_map(&m.k, p.k, p.batch, p.T, p.Hk, p.K, p.ks) ||
      !head_map(&m.v, p.v, p.batch, p.T, p.H, p.V, p.vs) || !head_map(&m.dy, p.dy, p.batch, p.T, p.H, p.V, p.ds) ||
      !head_map(&m.dq, p.dq, p.batch, p.T, p.Hk, p.K, ks) || !head_map(&m.dk, p.dk, p.batch, p.T, p.Hk, p.K, ks))
    return cudaErrorInvalidValue;
  const TcBuffers buf = buffers_in(buffers, p, true);
  cudaError_t e = p.K <= 64 ? chunks_as<1>(p, m, buf, st) : chunks_as<2>(p, m, buf, st);
  if (e == cudaSuccess && !states_known) {
    Params f = p;
    f.y = nullptr;
    f.final_state = nullptr;
    f.states_out = const_cast<float*>(p.states_in);
    if (!state_map(&m.states, f.states_out, cells, p.V, p.K)) return cudaErrorInvalidValue;
    float* segments = segments_in(buf, p, true);
    e = p.K <= 64 ? chain_as<1>(f, m, buf, segments, st) : chain_as<2>(f, m, buf, segments, st);
  }
  if (e != cudaSuccess) return e;
  if (!state_map(&m.states, p.dstates, cells, p.V, p.K)) return cudaErrorInvalidValue;
  return tc_backward_kernels(p, m, buf, st);
}

}  // namespace delta
}  // namespace ssd
