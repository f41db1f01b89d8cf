// Gated delta rule on the tensor cores, backward (the forms and the notation are those of delta_rule_tc.cu).  With G the
// gradient of the state behind a chunk and I_ = (I + A)^-1:
//   dU = P^T dY + diag(E) K G^T;   dR = I_^T dU, the gradient of v - S k;   dV = beta dR
//   gradient of the state before the chunk = D_last G + scale (diag(D) dY)^T Q - (diag(D beta) dR)^T K
// is a walk from the last chunk to the first, of the forward walk's form (delta_chain_back_kernel); it leaves dR and G
// of every chunk.  From these, the states that the forward kept and U, formed anew, all else follows chunk by chunk in
// parallel (delta_grad_kernel), keys in the 128 lanes of TMEM:
//   dQ^T = scale S^T dY^T diag(D) + K^T Bm^T,               Bm = scale M o (dY U^T)
//   dK^T = G^T U^T diag(E) - S^T dR^T diag(D beta) + Q^T Bm + (K^T N'^T) diag(beta) + K^T diag(beta) N',
//                                                           N' = -M o (dR U^T) below the diagonal
//   dbeta_i = dR_i . v_i - k_i . (D_i S^T dR_i - (K^T N'^T)_i)
//   dg_i = D_last <G, S> + sum_{a >= i} (scale D_a q_a . S^T dy_a - beta_a D_a k_a . S^T dR_a) + sum_{b < i} E_b k_b . G^T u_b
//          + sum_{a >= i > b} (Bm_ab q_a . k_b + beta_a N'_ab k_a . k_b)
// that is, every product that the decay of step i is a factor of.  (The shorter sum of q . dq - dv . v over the steps
// behind i has the same value, but its terms cancel: with operands in two terms dg was off by 1e-5 to 3e-5.)
#include <string.h>

#include <algorithm>

#include "delta_tc.cuh"
#include "launch.h"

namespace ssd {
namespace {

using namespace delta;

// ---------------------------------------------------------------------------------------------------------------------
// The walk.  TMEM columns: G's two terms, P^T dY, K G^T and after it dU's two terms, dR, what of it enters G, the sum
// that G takes.  K and dY have two buffers, the others one: what is used early in a chunk is loaded again while the
// rest of it runs.
// ---------------------------------------------------------------------------------------------------------------------
constexpr uint32_t kColG = 0, kColY = 128, kColU = 192, kColR = 256, kColW = 320, kColD = 384;

template <int KB>
struct BackSmem {
  uint8_t k[2][KB * kTileBytes], dy[2][2 * kTileBytes];
  uint8_t q[KB * kTileBytes], t[2 * kTileBytes], p[2 * kTileBytes];
  uint8_t dys[2][2 * kTileBytes];   // scale D dY, hi and lo
  uint8_t r[4 * kTileBytes];        // dR on its way out: by 64 values, hi then lo
  uint8_t s[4][128 * 64];           // G on its way out
  float decays[2][kDecays];
  uint64_t kdy_full[2], kdy_empty[2], q_full, q_empty, t_full, t_empty, p_full, p_empty;
  uint64_t g_ready[4], y_full, u_ready, r_full, w_ready, r_free, dys_ready, d_full, drain;
  uint32_t tmem;
  int abort;
};

template <int KB>
__global__ void __launch_bounds__(kWalkThreads, 1)
    delta_chain_back_kernel(const __grid_constant__ Params p, const __grid_constant__ TcMaps m, TcBuffers buf) {
  extern __shared__ __align__(1024) uint8_t raw[];
  BackSmem<KB>& sm = *reinterpret_cast<BackSmem<KB>*>(raw);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x / 32), 0), lane = threadIdx.x % 32;
  const int h = blockIdx.x % (int)p.H, b = blockIdx.x / (int)p.H, hk = h / (int)(p.H / p.Hk), nch = (int)p.nch;
  constexpr int Kp = KB * 64;
  volatile int* abort = &sm.abort;
  if (threadIdx.x == 0) {
    sm.abort = 0;
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.kdy_full[s], 1);
      mbar_init(&sm.kdy_empty[s], 1);
    }
    for (uint64_t* four : {&sm.g_ready[0], &sm.g_ready[1], &sm.g_ready[2], &sm.g_ready[3], &sm.r_free, &sm.dys_ready})
      mbar_init(four, 4);
    for (uint64_t* one : {&sm.q_full, &sm.q_empty, &sm.t_full, &sm.t_empty, &sm.p_full, &sm.p_empty, &sm.y_full, &sm.r_full,
                          &sm.d_full, &sm.drain})
      mbar_init(one, 1);
    mbar_init(&sm.u_ready, kStateWarps);
    mbar_init(&sm.w_ready, kStateWarps);
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
  // n counts chunks done, c is the chunk: nch - 1 - n
  if (warp == 21) {   // loads
    int pairs = 0, ps = 0, ts = 0, qs = 0;   // loads issued
    for (int n = 0; n < nch; ++n) {
      const int s = n & 1, c = nch - 1 - n;
      const uint32_t par = (n - 1) & 1;
      const int64_t cell = ((int64_t)b * nch + c) * p.H + h;
      const uint8_t* sq = buf.squares + cell * buf.square;
      if (n >= 2 && !wait_bar(&sm.kdy_empty[s], ((n >> 1) - 1) & 1, abort, p.hdr, 40)) break;
      mbar_arrive_expect_tx_elect(&sm.kdy_full[s], (KB + 2) * kTileBytes + kDecayBytes);
      bulk_load_elect(sm.decays[s], buf.decays + cell * kDecays, kDecayBytes, &sm.kdy_full[s]);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        tma_load_4d_elect(sm.k[s] + kb * kTileBytes, &m.k, &sm.kdy_full[s], kb * 64, c * kChunk, hk, b);
      tma_load_4d_elect(sm.dy[s], &m.dy, &sm.kdy_full[s], 0, c * kChunk, h, b);
      tma_load_4d_elect(sm.dy[s] + kTileBytes, &m.dy, &sm.kdy_full[s], 64, c * kChunk, h, b);
      pairs = n + 1;
      if (n >= 1 && !wait_bar(&sm.p_empty, par, abort, p.hdr, 41)) break;
      mbar_arrive_expect_tx_elect(&sm.p_full, 2 * kTileBytes);
      bulk_load_elect(sm.p, sq + 2 * kTileBytes, 2 * kTileBytes, &sm.p_full);
      ps = n + 1;
      if (n >= 1 && !wait_bar(&sm.t_empty, par, abort, p.hdr, 42)) break;
      mbar_arrive_expect_tx_elect(&sm.t_full, 2 * kTileBytes);
      bulk_load_elect(sm.t, sq + 4 * kTileBytes, 2 * kTileBytes, &sm.t_full);
      ts = n + 1;
      if (n >= 1 && !wait_bar(&sm.q_empty, par, abort, p.hdr, 43)) break;
      mbar_arrive_expect_tx_elect(&sm.q_full, KB * kTileBytes);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
        tma_load_4d_elect(sm.q + kb * kTileBytes, &m.q, &sm.q_full, kb * 64, c * kChunk, hk, b);
      qs = n + 1;
    }
    bool drained = true;
    for (int s = 0; s < 2; ++s) {
      const int loads = pairs > s ? (pairs - 1 - s) / 2 + 1 : 0;
      if (loads > 0) drained &= mbar_wait_bounded(&sm.kdy_full[s], (loads - 1) & 1, kDrainNs);
    }
    if (ps > 0) drained &= mbar_wait_bounded(&sm.p_full, (ps - 1) & 1, kDrainNs);
    if (ts > 0) drained &= mbar_wait_bounded(&sm.t_full, (ts - 1) & 1, kDrainNs);
    if (qs > 0) drained &= mbar_wait_bounded(&sm.q_full, (qs - 1) & 1, kDrainNs);
    if (!drained && lane == 0) latch_error(p.hdr, SSD_ERR_TIMEOUT, 44);
  } else if (warp == 20) {   // products
    constexpr uint32_t id_k = idesc_bf16(128, 64, 0, 0), id_p = idesc_bf16(128, 64, 1, 1), id_t = idesc_bf16(128, 64, 0, 1);
    constexpr uint32_t id_q = idesc_bf16(128, Kp, 1, 1), id_d = idesc_bf16(128, Kp, 0, 1);
    const uint32_t p_lo = sdesc_sw128_lo(smem_u32(sm.p), 0), t_lo = sdesc_sw128_lo(smem_u32(sm.t), 0);
    const uint32_t q_lo = sdesc_sw128_lo(smem_u32(sm.q), kTileBytes);
    const uint32_t s_hi = sdesc_sw128_lo(smem_u32(sm.dys[0]), kTileBytes), s_lo = sdesc_sw128_lo(smem_u32(sm.dys[1]), kTileBytes);
    for (int n = 0; n < nch; ++n) {
      const int s = n & 1;
      const uint32_t par = n & 1;
      const uint32_t k_lo = sdesc_sw128_lo(smem_u32(sm.k[s]), 0), km_lo = sdesc_sw128_lo(smem_u32(sm.k[s]), kTileBytes);
      const uint32_t dy_lo = sdesc_sw128_lo(smem_u32(sm.dy[s]), kTileBytes);
      if (!wait_bar(&sm.kdy_full[s], (n >> 1) & 1, abort, p.hdr, 45)) break;
      if (!wait_bar(&sm.p_full, par, abort, p.hdr, 46)) break;
      // P^T dY (its accumulator was read before the chunk before this one was through)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        mma_ss_we(tmem + kColY, dy_lo + ks * (2048 >> 4), kDHi, p_lo + ks * (2048 >> 4), kDHi, id_p, ks > 0);
        mma_ss_we(tmem + kColY, dy_lo + ks * (2048 >> 4), kDHi, p_lo + kLo + ks * (2048 >> 4), kDHi, id_p, 1);
      }
      mma_commit_elect(&sm.p_empty);
      // K G^T
      bool ready = true;
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        ready = ready && wait_bar(&sm.g_ready[part], par, abort, p.hdr, 47);
        if (!ready) break;
        tc_fence_after();
#pragma unroll
        for (int ks = part * KB; ks < (part + 1) * KB; ++ks) {
          const uint32_t at = k_lo + (((ks >> 2) * kTileBytes + (ks & 3) * 32) >> 4);
          mma_ts_we(tmem + kColU, tmem + kColG + ks * 8, at, kDHi, id_k, ks > 0);
          mma_ts_we(tmem + kColU, tmem + kColG + Kp / 2 + ks * 8, at, kDHi, id_k, 1);
        }
      }
      if (!ready) break;
      mma_commit_elect(&sm.y_full);
      // scale (D dY)^T Q, while dU is made
      if (!wait_bar(&sm.q_full, par, abort, p.hdr, 48)) break;
      if (!wait_bar(&sm.dys_ready, par, abort, p.hdr, 49)) break;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        mma_ss_we(tmem + kColD, s_hi + ks * (2048 >> 4), kDHi, q_lo + ks * (2048 >> 4), kDHi, id_q, ks > 0);
        mma_ss_we(tmem + kColD, s_lo + ks * (2048 >> 4), kDHi, q_lo + ks * (2048 >> 4), kDHi, id_q, 1);
      }
      mma_commit_elect(&sm.q_empty);
      // dR^T = dU^T I_
      if (!wait_bar(&sm.t_full, par, abort, p.hdr, 50)) break;
      if (n > 0 && !wait_bar(&sm.r_free, (n - 1) & 1, abort, p.hdr, 51)) break;
      if (!wait_bar(&sm.u_ready, par, abort, p.hdr, 52)) break;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint32_t a = tmem + kColU + ks * 16;
        mma_ts_we(tmem + kColR, a, t_lo + ks * (2048 >> 4), kDHi, id_t, ks > 0);
        mma_ts_we(tmem + kColR, a, t_lo + kLo + ks * (2048 >> 4), kDHi, id_t, 1);
        mma_ts_we(tmem + kColR, a + 8, t_lo + ks * (2048 >> 4), kDHi, id_t, 1);
      }
      mma_commit_elect(&sm.r_full);
      mma_commit_elect(&sm.t_empty);
      // - (D beta dR)^T K
      if (!wait_bar(&sm.w_ready, par, abort, p.hdr, 53)) break;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint32_t a = tmem + kColW + ks * 16;
        mma_ts_we(tmem + kColD, a, km_lo + ks * (2048 >> 4), kDHi, id_d, 1);
        mma_ts_we(tmem + kColD, a + 8, km_lo + ks * (2048 >> 4), kDHi, id_d, 1);
      }
      mma_commit_elect(&sm.d_full);
      mma_commit_elect(&sm.kdy_empty[s]);
    }
    mma_commit_elect(&sm.drain);
    if (!mbar_wait_bounded(&sm.drain, 0, kDrainNs) && lane == 0) latch_error(p.hdr, SSD_ERR_TIMEOUT, 54);
  } else if (warp < kStateWarps) {   // G
    constexpr int KQ = Kp / 4;
    const int part = warp >> 2, row = (warp & 3) * 32 + lane, k0 = part * KQ, j0 = part * 16;
    const bool live = row < p.V;
    const int64_t at = (((int64_t)b * p.H + h) * p.V + row) * p.K + k0;
    bool on = true;   // after a wait that gave up, without waiting: the quarter's warps meet at its barrier
    float G[KQ];
#pragma unroll
    for (int k = 0; k < KQ; ++k) G[k] = 0.f;
    if (p.dfinal && live) load_row(G, p.dfinal + at, p.K - k0);
    int cell = (b * nch + nch - 1) * (int)p.H + h;
    for (int n = 0; n < nch; ++n, cell -= (int)p.H) {
      const int s = n & 1;
      const uint32_t par = n & 1;
      store_state_terms(tmem + lanes + kColG + k0 / 2, Kp / 2, G);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.g_ready[part]);
      send_state(sm.s[part], &m.states, G, part, 0, 0, cell, p.K);
      on = on && wait_bar(&sm.kdy_full[s], (n >> 1) & 1, abort, p.hdr, 55);   // the decays
      const float all = sm.decays[s][kChunk - 1];
      on = on && wait_bar(&sm.y_full, par, abort, p.hdr, 56);
      tc_fence_after();
      float x[16], y[16];
      tmem_ld16(tmem + lanes + kColY + j0, y);
      tmem_ld16(tmem + lanes + kColU + j0, x);
      tmem_ld_wait();
      reg_tie(x);
      reg_tie(y);
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&sm.decays[s][kChunk + j0 + j]);
        x[j] = fmaf(x[j], f.x, y[j]);
        x[j + 1] = fmaf(x[j + 1], f.y, y[j + 1]);
        x[j + 2] = fmaf(x[j + 2], f.z, y[j + 2]);
        x[j + 3] = fmaf(x[j + 3], f.w, y[j + 3]);
      }
      store_terms(tmem + lanes + kColU + j0, x);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.u_ready);
      if constexpr (KB == 2) send_state(sm.s[part], &m.states, G, part, KQ / 2, 0, cell, p.K);
      on = on && wait_bar(&sm.r_full, par, abort, p.hdr, 57);
      tc_fence_after();
      tmem_ld16(tmem + lanes + kColR + j0, x);
      tmem_ld_wait();
      reg_tie(x);
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&sm.decays[s][j0 + j]);
        x[j] *= -f.x;
        x[j + 1] *= -f.y;
        x[j + 2] *= -f.z;
        x[j + 3] *= -f.w;
      }
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&sm.decays[s][2 * kChunk + j0 + j]);
        x[j] *= f.x;
        x[j + 1] *= f.y;
        x[j + 2] *= f.z;
        x[j + 3] *= f.w;
      }
      store_terms(tmem + lanes + kColW + j0, x);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.w_ready);
      on = on && wait_bar(&sm.d_full, par, abort, p.hdr, 58);
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < KQ; k += 16) {
        tmem_ld16(tmem + lanes + kColD + k0 + k, x);
        tmem_ld_wait();
        reg_tie(x);
#pragma unroll
        for (int j = 0; j < 16; ++j) G[k + j] = fmaf(all, G[k + j], x[j]);
      }
    }
    if ((threadIdx.x & 127) == 0) bulk_wait_group<0>();
    if (p.dinit && live && on) {
      const bool wide = (reinterpret_cast<uintptr_t>(p.dinit) & 31) == 0;
#pragma unroll
      for (int k = 0; k < KQ; k += 8)
        if (k0 + k < p.K && SSD_INDEX_OK(p.hdr, at + k + 7, p.batch * p.H * p.V * p.K, 2015))
          store8(p.dinit + at + k, G + k, wide);
    }
  } else {   // scale D dY in two terms, and dR on its way out
    const int t = threadIdx.x - kStateWarps * 32, v = (warp & 3) * 32 + lane;
    bool on = true;   // as above
    for (int n = 0; n < nch; ++n) {
      const int s = n & 1, c = nch - 1 - n;
      const uint32_t par = n & 1;
      on = on && wait_bar(&sm.kdy_full[s], (n >> 1) & 1, abort, p.hdr, 59);
      if (n > 0) on = on && wait_bar(&sm.d_full, (n - 1) & 1, abort, p.hdr, 60);   // the last terms have been read
#pragma unroll 2
      for (int m8 = 0; m8 < 8; ++m8) {   // 16 bytes of a row
        const int at = m8 * 128 + t, blk = at >> 9, i = (at >> 3) & 63, col = (at & 7) * 8;
        const uint32_t off = blk * kTileBytes + sw128_off16(i, col);
        const uint4 d = *reinterpret_cast<const uint4*>(sm.dy[s] + off);
        const float f = sm.decays[s][3 * kChunk + i];
        uint4 hi, lo;
        split2(__uint_as_float(d.x << 16) * f, __uint_as_float(d.x & 0xffff0000u) * f, hi.x, lo.x);
        split2(__uint_as_float(d.y << 16) * f, __uint_as_float(d.y & 0xffff0000u) * f, hi.y, lo.y);
        split2(__uint_as_float(d.z << 16) * f, __uint_as_float(d.z & 0xffff0000u) * f, hi.z, lo.z);
        split2(__uint_as_float(d.w << 16) * f, __uint_as_float(d.w & 0xffff0000u) * f, hi.w, lo.w);
        *reinterpret_cast<uint4*>(sm.dys[0] + off) = hi;
        *reinterpret_cast<uint4*>(sm.dys[1] + off) = lo;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.dys_ready);
      on = on && wait_bar(&sm.r_full, par, abort, p.hdr, 61);
      tc_fence_after();
      if (warp == kStateWarps && lane == 0) bulk_wait_group_read<0>();
      named_barrier(1, 128);
      uint8_t* out = sm.r + (v >> 6) * 2 * kTileBytes;
#pragma unroll 1
      for (int j0 = 0; j0 < kChunk; j0 += 16) {
        float r[16];
        tmem_ld16(tmem + lanes + kColR + j0, r);
        tmem_ld_wait();
        reg_tie(r);
#pragma unroll
        for (int j = 0; j < 16; j += 2)
          store_pair_terms(out + sw128_off16(j0 + j, v & 63), out + sw128_off16(j0 + j + 1, v & 63), kTileBytes, r[j], r[j + 1]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.r_free);
      fence_proxy_async_smem();
      named_barrier(1, 128);
      if (warp == kStateWarps && lane == 0) {
        const int64_t cell = ((int64_t)b * nch + c) * p.H + h;
        if (SSD_INDEX_OK(p.hdr, cell, p.batch * p.nch * p.H, 2016))
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(buf.writes + cell * 4 * kTileBytes),
                       "r"(smem_u32(sm.r)), "r"(4 * kTileBytes)
                       : "memory");
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

// ---------------------------------------------------------------------------------------------------------------------
// A block an SM, which goes from chunk to chunk (of a key head; the heads that share the keys one after the other).  What
// the next head reads is loaded as soon as its place in shared memory is free: dY and dR once the products with them are
// through, the state, as it is in memory, into G's place, V, T, Q and K at the end.  (A block a chunk, loading when it
// begins: 415 us instead of 364 for 4 x 4096 x 16 heads.)
// ---------------------------------------------------------------------------------------------------------------------
constexpr int kGradThreads = 512;   // 16 columns of TMEM a warp (with 32 and 256 threads 473 us instead of 434: latency)
// TMEM: X and -D X, then [dY; dR hi] with U's first term; U, then with its second; S^T dY^T; S^T dR^T; G^T U^T; K^T Bm^T;
// [Q; K] K^T, then K^T N'^T; dR lo U^T, then Q^T Bm + K^T diag(beta) N'.  Operands that follow each other in shared
// memory enter one product of 128 columns: with 64 the reading of the operands (6 KB for 32 cycles' work) bounds it.
enum : uint32_t { kX = 0, kU = 64, kSY = 128, kSR = 192, kGU = 256, kKB = 320, kKN = 384, kQB = 448 };

struct GradSmem {
  uint8_t qk[2][2 * kTileBytes];      // by 64 keys: Q, K
  uint8_t dyr[2][3 * kTileBytes];     // by 64 values: dY, dR hi, dR lo
  uint8_t u[2][2 * kTileBytes];       // by 64 values: hi, lo
  uint8_t s[4][2 * kTileBytes];       // S, then G: hi by 64 keys, lo; 128 rows of values
  uint8_t v[2 * kTileBytes], t[2 * kTileBytes];   // then Bm hi, N' hi; Bm lo, N' lo
  uint8_t n2[2 * kTileBytes];         // diag(beta) N'
  ChunkDecay c;
  float dot[kChunk];                  // dR . v
  uint64_t loaded, done, shadow, drain;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(GradSmem) <= 232448, "shared memory of a block");

// A thread's 32 values of a state [V, K] f32: four times eight of a row; zeros around it.
__device__ __forceinline__ void read_state(float4 (&f)[8], const float* S, int64_t V, int64_t K) {
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int at = it * kGradThreads + threadIdx.x, row = at >> 4, col = (at & 15) * 8;
    f[2 * it] = f[2 * it + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (S && row < V && col < K) {
      f[2 * it] = *reinterpret_cast<const float4*>(S + row * K + col);
      f[2 * it + 1] = *reinterpret_cast<const float4*>(S + row * K + col + 4);
    }
  }
}
// As two terms to their place among the operands; with kInner the sum of the products with what stood there.
template <bool kInner>
__device__ __forceinline__ float stage_state(GradSmem& sm, const float4 (&f)[8]) {
  float inner = 0.f;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int at = it * kGradThreads + threadIdx.x, row = at >> 4, col = (at & 15) * 8;
    const float4 a = f[2 * it], b = f[2 * it + 1];
    uint8_t* hi_at = sm.s[col >> 6] + sw128_off16(row, col & 63);
    uint8_t* lo_at = hi_at + 4 * kTileBytes;
    if constexpr (kInner) {
      const uint4 h = *reinterpret_cast<const uint4*>(hi_at), l = *reinterpret_cast<const uint4*>(lo_at);
      auto pair = [&](uint32_t hh, uint32_t ll, float x, float y) {
        inner = fmaf(x, __uint_as_float(hh << 16) + __uint_as_float(ll << 16), inner);
        inner = fmaf(y, __uint_as_float(hh & 0xffff0000u) + __uint_as_float(ll & 0xffff0000u), inner);
      };
      pair(h.x, l.x, a.x, a.y);
      pair(h.y, l.y, a.z, a.w);
      pair(h.z, l.z, b.x, b.y);
      pair(h.w, l.w, b.z, b.w);
    }
    uint4 hi, lo;
    split2(a.x, a.y, hi.x, lo.x);
    split2(a.z, a.w, hi.y, lo.y);
    split2(b.x, b.y, hi.z, lo.z);
    split2(b.z, b.w, hi.w, lo.w);
    *reinterpret_cast<uint4*>(hi_at) = hi;
    *reinterpret_cast<uint4*>(lo_at) = lo;
  }
  return inner;
}

// 8 consecutive columns of TMEM.
__device__ __forceinline__ void tmem_ld8(uint32_t at, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

// Sums of N columns over a warp's lanes: lane l has that of column l % N.  Halving: N - 1 exchanges where sums column by
// column take 5 N.
template <int N>
__device__ __forceinline__ float sum_columns(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = N / 2; o; o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int j = 0; j < o; ++j) {
      const float keep = upper ? v[j + o] : v[j], give = upper ? v[j] : v[j + o];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (int o = N; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// Sums over the lanes before this one, and behind it.  Each adds up its own lanes: the sum of all less the others would leave
// the rounding of large values (of steps that a reset has cut off) on small ones.
__device__ __forceinline__ float sum_before(float v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  v = __shfl_up_sync(0xffffffffu, v, 1);
  return lane ? v : 0.f;
}
__device__ __forceinline__ float sum_behind(float v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_down_sync(0xffffffffu, v, o);
    if (lane + o < 32) v += u;
  }
  v = __shfl_down_sync(0xffffffffu, v, 1);
  return lane < 31 ? v : 0.f;
}

__global__ void __launch_bounds__(kGradThreads, 1)
    delta_grad_kernel(const __grid_constant__ Params p, const __grid_constant__ TcMaps m, TcBuffers buf) {
  extern __shared__ __align__(1024) uint8_t raw[];
  GradSmem& sm = *reinterpret_cast<GradSmem*>(raw);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid / 32, 0), lane = tid % 32;
  const int quarter = warp & 3, c0 = (warp >> 2) * 16, row = quarter * 32 + lane;   // lanes and columns of TMEM
  const int64_t group = p.H / p.Hk, KV = p.K * p.V, blocks = p.batch * p.nch * p.Hk;
  if (tid == 0) {
    mbar_init(&sm.loaded, 1);
    mbar_init(&sm.done, 1);
    mbar_init(&sm.shadow, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem, mine = tmem + ((uint32_t)(quarter * 32) << 16);
  volatile int* abort = &sm.abort;
  constexpr uint32_t kk = idesc_bf16(128, 64, 0, 0), mk = idesc_bf16(128, 64, 1, 0), mm = idesc_bf16(128, 64, 1, 1);
  constexpr uint32_t kk2 = idesc_bf16(128, 128, 0, 0), mk2 = idesc_bf16(128, 128, 1, 0);
  constexpr uint32_t kStep = 2048 >> 4, kStateLo = (4 * kTileBytes) >> 4;
  const uint32_t qk_lo = sdesc_sw128_lo(smem_u32(sm.qk[0]), 0), k_lo = qk_lo + kLo;
  const uint32_t qm_lo = sdesc_sw128_lo(smem_u32(sm.qk[0]), 2 * kTileBytes), km_lo = qm_lo + kLo;
  const uint32_t s_lo = sdesc_sw128_lo(smem_u32(sm.s[0]), 0), sm_lo = sdesc_sw128_lo(smem_u32(sm.s[0]), 2 * kTileBytes);
  const uint32_t dyr_lo = sdesc_sw128_lo(smem_u32(sm.dyr[0]), 0), u_lo = sdesc_sw128_lo(smem_u32(sm.u), 0);
  const uint32_t v_lo = sdesc_sw128_lo(smem_u32(sm.v), kTileBytes), t_lo = sdesc_sw128_lo(smem_u32(sm.t), 0);
  const uint32_t bm_lo = sdesc_sw128_lo(smem_u32(sm.v), 0), n2_lo = sdesc_sw128_lo(smem_u32(sm.n2), 0);
  // of 128 values in blocks of 64: step ks of 16
  auto by64 = [](int ks, uint32_t block) { return (ks >> 2) * (block >> 4) + (ks & 3) * 2; };
  uint32_t phase = 0, turn = 0, announced = 0;   // products waited for; loads waited for, and under way
  // The loads of a head's operands, in three parts (by warp 0); the first announces all.
  struct Item {
    int64_t id, h;   // of chunks and key heads; head
  };
  auto split = [&](int64_t id, int64_t& b, int64_t& chunk, int64_t& hk) {
    hk = id % p.Hk;
    chunk = id / p.Hk % p.nch;
    b = id / p.Hk / p.nch;
  };
  auto cell_of = [&](const Item& i) { return i.id / p.Hk * p.H + i.h; };   // (b nch + chunk) H + h
  auto load_gradients = [&](const Item& i) {
    int64_t b, chunk, hk;
    split(i.id, b, chunk, hk);
    ++announced;
    mbar_arrive_expect_tx_elect(&sm.loaded, (i.h == hk * group ? 14 : 10) * kTileBytes + (uint32_t)(KV * 4));
#pragma unroll
    for (int vb = 0; vb < 2; ++vb) {
      tma_load_4d_elect(sm.dyr[vb], &m.dy, &sm.loaded, vb * 64, (int)(chunk * kChunk), (int)i.h, (int)b);
      bulk_load_elect(sm.dyr[vb] + kTileBytes, buf.writes + (cell_of(i) * 4 + vb * 2) * kTileBytes, 2 * kTileBytes, &sm.loaded);
    }
  };
  auto load_state = [&](const Item& i) { bulk_load_elect(sm.s, p.states_in + cell_of(i) * KV, (uint32_t)(KV * 4), &sm.loaded); };
  auto load_rest = [&](const Item& i) {
    int64_t b, chunk, hk;
    split(i.id, b, chunk, hk);
    if (i.h == hk * group) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {   // keys past K are zeros
        tma_load_4d_elect(sm.qk[kb], &m.q, &sm.loaded, kb * 64, (int)(chunk * kChunk), (int)hk, (int)b);
        tma_load_4d_elect(sm.qk[kb] + kTileBytes, &m.k, &sm.loaded, kb * 64, (int)(chunk * kChunk), (int)hk, (int)b);
      }
    }
#pragma unroll
    for (int vb = 0; vb < 2; ++vb)
      tma_load_4d_elect(sm.v + vb * kTileBytes, &m.v, &sm.loaded, vb * 64, (int)(chunk * kChunk), (int)i.h, (int)b);
    bulk_load_elect(sm.t, buf.squares + cell_of(i) * buf.square, 2 * kTileBytes, &sm.loaded);
  };
  Item item = {(int64_t)blockIdx.x, (int64_t)blockIdx.x % p.Hk * group};
  if (warp == 0) {
    load_gradients(item);
    load_state(item);
    load_rest(item);
  }
  float dq[16] = {}, dk[16] = {};
  bool ok = true;
  while (item.id < blocks) {
    int64_t b, chunk, hk;
    split(item.id, b, chunk, hk);
    const int64_t h = item.h, cell = cell_of(item), t0 = chunk * kChunk;
    const int n = (int)min((int64_t)kChunk, p.T - t0);
    const bool last_head = h + 1 == (hk + 1) * group;
    const Item next = last_head ? Item{item.id + gridDim.x, (item.id + gridDim.x) % p.Hk * group} : Item{item.id, h + 1};
    const bool more = next.id < blocks;
    if (warp == 1) chunk_decay_warp(p, sm.c, b, t0, n, h, lane);
    ok = wait_bar(&sm.loaded, turn++ & 1, abort, p.hdr, 70);
    {
      float4 f[8];   // from where the copy put it, then over it
      read_state(f, reinterpret_cast<const float*>(sm.s), p.V, p.K);
      __syncthreads();
      stage_state<false>(sm, f);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    ok = !__syncthreads_or(!ok);   // all warps go on, or none
    tc_fence_after();
    if (!ok) break;
    if (warp == 0) {
      // X = S K^T and V T^T
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        mma_ss_we(tmem + kX, s_lo + by64(ks, 2 * kTileBytes), kDHi, k_lo + by64(ks, 2 * kTileBytes), kDHi, kk, ks > 0);
        mma_ss_we(tmem + kX, s_lo + kStateLo + by64(ks, 2 * kTileBytes), kDHi, k_lo + by64(ks, 2 * kTileBytes), kDHi, kk, 1);
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        mma_ss_we(tmem + kU, v_lo + ks * kStep, kDHi, t_lo + ks * 2, kDHi, mk, ks > 0);
        mma_ss_we(tmem + kU, v_lo + ks * kStep, kDHi, t_lo + kLo + ks * 2, kDHi, mk, 1);
      }
      mma_commit_elect(&sm.done);
    }
    // dv = beta dR, and dR . v: eight threads a step, 16 bytes at a time
    {
      const int i = tid >> 3, part = tid & 7;
      const float beta = sm.c.beta[i];
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = (e * 8 + part) * 8, vb = col >> 6;
        const uint32_t off = sw128_off16(i, col & 63);
        const uint4 hi = *reinterpret_cast<const uint4*>(sm.dyr[vb] + kTileBytes + off);
        const uint4 lo = *reinterpret_cast<const uint4*>(sm.dyr[vb] + 2 * kTileBytes + off);
        const uint4 v = *reinterpret_cast<const uint4*>(sm.v + vb * kTileBytes + off);
        uint32_t out[4];
        auto pair = [&](uint32_t a, uint32_t l, uint32_t w, uint32_t& o) {
          const float x = __uint_as_float(a << 16) + __uint_as_float(l << 16);
          const float y = __uint_as_float(a & 0xffff0000u) + __uint_as_float(l & 0xffff0000u);
          dot = fmaf(x, __uint_as_float(w << 16), dot);
          dot = fmaf(y, __uint_as_float(w & 0xffff0000u), dot);
          const __nv_bfloat162 r = __floats2bfloat162_rn(beta * x, beta * y);
          o = *reinterpret_cast<const uint32_t*>(&r);
        };
        pair(hi.x, lo.x, v.x, out[0]);
        pair(hi.y, lo.y, v.y, out[1]);
        pair(hi.z, lo.z, v.z, out[2]);
        pair(hi.w, lo.w, v.w, out[3]);
        const int64_t to = ((b * p.T + t0 + i) * p.H + h) * p.V + col;
        if (i < n && col < p.V && SSD_INDEX_OK(p.hdr, to + 7, p.batch * p.T * p.H * p.V, 2017))
          *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dv) + to) = make_uint4(out[0], out[1], out[2], out[3]);
      }
      dot += __shfl_xor_sync(0xffffffffu, dot, 1);
      dot += __shfl_xor_sync(0xffffffffu, dot, 2);
      dot += __shfl_xor_sync(0xffffffffu, dot, 4);
      if (part == 0) sm.dot[i] = dot;
    }
    // the gradient of the state behind this chunk, on its way until the state is through
    float4 gs[8];
    read_state(gs, p.dstates + cell * KV, p.V, p.K);
    ok = wait_bar(&sm.done, phase++ & 1, abort, p.hdr, 71);
    tc_fence_after();
    float x[16];
    if (ok) {   // -D X: hi over its first 8 columns, lo over the others
      tmem_ld16(mine + kX + c0, x);
      tmem_ld_wait();
      reg_tie(x);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] *= -sm.c.from[c0 + j];
      uint32_t terms[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) split2(x[2 * j], x[2 * j + 1], terms[j], terms[8 + j]);
      tmem_st16u(mine + kX + c0, terms);
      tmem_st_wait();
    }
    if (tid == 0) bulk_wait_group_read<0>();   // dq and dk have left U's place
    tc_fence_before();
    ok = !__syncthreads_or(!ok);
    tc_fence_after();
    if (!ok) break;
    if (warp == 0) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint32_t a = tmem + kX + ks * 16;
        mma_ts_we(tmem + kU, a, t_lo + ks * 2, kDHi, kk, 1);
        mma_ts_we(tmem + kU, a, t_lo + kLo + ks * 2, kDHi, kk, 1);
        mma_ts_we(tmem + kU, a + 8, t_lo + ks * 2, kDHi, kk, 1);
      }
      mma_commit_elect(&sm.done);
      // S^T [dY; dR]^T
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t a = sm_lo + ks * kStep, at = dyr_lo + by64(ks, 3 * kTileBytes);
        mma_ss_we(tmem + kSY, a, kDHi, at, kDHi, mk2, ks > 0);
        mma_ss_we(tmem + kSY, a + kStateLo, kDHi, at, kDHi, mk2, 1);
        mma_ss_we(tmem + kSR, a, kDHi, at + 2 * kLo, kDHi, mk, 1);
      }
      // [Q; K] K^T, where K^T N'^T will be
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        mma_ss_we(tmem + kKN, qk_lo + by64(ks, 2 * kTileBytes), kDHi, k_lo + by64(ks, 2 * kTileBytes), kDHi, kk, ks > 0);
      mma_commit_elect(&sm.shadow);
    }
    ok = wait_bar(&sm.done, phase++ & 1, abort, p.hdr, 72);
    tc_fence_after();
    if (ok) {   // U's rows, by steps
      tmem_ld16(mine + kU + c0, x);
      tmem_ld_wait();
      reg_tie(x);
      uint8_t* at = sm.u[row >> 6];
#pragma unroll
      for (int j = 0; j < 16; j += 2)
        store_pair_terms(at + sw128_off16(c0 + j, row & 63), at + sw128_off16(c0 + j + 1, row & 63), kTileBytes, x[j], x[j + 1]);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    ok = !__syncthreads_or(!ok);
    tc_fence_after();
    if (!ok) break;
    if (warp == 0) {
      // [dY; dR hi] U^T, and (rows 64..127) dR lo U^T
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t a = dyr_lo + by64(ks, 3 * kTileBytes), at = u_lo + by64(ks, 2 * kTileBytes);
        mma_ss_we(tmem + kX, a, kDHi, at, kDHi, kk2, ks > 0);
        mma_ss_we(tmem + kQB, a + kLo, kDHi, at, kDHi, kk, ks > 0);
      }
      mma_commit_elect(&sm.done);
    }
    // G takes the state's place
    ok = wait_bar(&sm.shadow, (turn - 1) & 1, abort, p.hdr, 73);
    float inner = 0.f;
    if (ok) inner = stage_state<true>(sm, gs) * sm.c.from[kChunk - 1];
    fence_proxy_async_smem();
    ok = !__syncthreads_or(!ok);
    if (!ok) break;
    if (warp == 0) {
      // G^T U^T
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const uint32_t a = sm_lo + ks * kStep, at = u_lo + by64(ks, 2 * kTileBytes);
        mma_ss_we(tmem + kGU, a, kDHi, at, kDHi, mk, ks > 0);
        mma_ss_we(tmem + kGU, a, kDHi, at + kLo, kDHi, mk, 1);
        mma_ss_we(tmem + kGU, a + kStateLo, kDHi, at, kDHi, mk, 1);
      }
    }
    ok = wait_bar(&sm.done, phase++ & 1, abort, p.hdr, 74);
    tc_fence_after();
    if (ok && warp == 0 && more) load_gradients(next);
    float across = 0.f, row_sum = 0.f;   // sum over the pairs of steps around the lane's; of this row
    if (ok) {
      // lanes 0..63: Bm's rows; 64..127: N's
      const int i = row & 63;
      const bool lower = quarter >= 2;
      float y[16], z[16];
      tmem_ld16(mine + kX + c0, x);
      tmem_ld16(mine + kU + c0, y);
      tmem_ld16(mine + kQB + c0, z);
      tmem_ld_wait();
      reg_tie(x);
      reg_tie(y);
      reg_tie(z);
      const float ch = sm.c.hi[i], cl = sm.c.lo[i], beta = sm.c.beta[i], by = lower ? -1.f : p.scale;
      const int last = lower ? i - 1 : i;
      const bool plain = sm.c.plain;
      const float mine_from = sm.c.from[i];
      uint8_t* to = lower ? sm.v + kTileBytes : sm.v;   // lo: in t, at the same place
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int c = c0 + j;
        const float f = lower ? (x[j] + y[j]) + z[j] : x[j] + y[j];
        const float decay = plain ? mine_from * sm.c.back[c] : expf((ch - sm.c.hi[c]) + (cl - sm.c.lo[c]));
        x[j] = c <= last ? f * by * decay : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 16; j += 8) {
        const uint32_t off = sw128_off16(i, c0 + j);
        uint4 hi, lo;
        split2(x[j], x[j + 1], hi.x, lo.x);
        split2(x[j + 2], x[j + 3], hi.y, lo.y);
        split2(x[j + 4], x[j + 5], hi.z, lo.z);
        split2(x[j + 6], x[j + 7], hi.w, lo.w);
        *reinterpret_cast<uint4*>(to + off) = hi;
        *reinterpret_cast<uint4*>(to + 2 * kTileBytes + off) = lo;
        if (lower) {
          split2(beta * x[j], beta * x[j + 1], hi.x, lo.x);
          split2(beta * x[j + 2], beta * x[j + 3], hi.y, lo.y);
          split2(beta * x[j + 4], beta * x[j + 5], hi.z, lo.z);
          split2(beta * x[j + 6], beta * x[j + 7], hi.w, lo.w);
          *reinterpret_cast<uint4*>(sm.n2 + off) = hi;
          *reinterpret_cast<uint4*>(sm.n2 + kTileBytes + off) = lo;
        }
      }
      // products of pairs a > b, summed along this row (a) over this warp's columns before each, then over the rows from
      // it on
      tmem_ld16(mine + kKN + c0, y);
      tmem_ld_wait();
      reg_tie(y);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float w = lower ? beta * y[j] : y[j];
        y[j] = i >= c0 + j ? row_sum : 0.f;
        row_sum = fmaf(x[j], w, row_sum);
      }
      across = sum_columns(y);
    }
    fence_proxy_async_smem();
    tc_fence_before();
    ok = !__syncthreads_or(!ok);
    tc_fence_after();
    if (!ok) break;
    if (warp == 0) {
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint32_t k = km_lo + ks * kStep, q = qm_lo + ks * kStep;
        mma_ss_we(tmem + kKB, k, kDHi, bm_lo + ks * 2, kDHi, mk2, ks > 0);   // with N' beside Bm
        mma_ss_we(tmem + kKB, k, kDHi, bm_lo + 2 * kLo + ks * 2, kDHi, mk2, 1);
        mma_ss_we(tmem + kQB, q, kDHi, bm_lo + ks * kStep, kDHi, mm, ks > 0);
        mma_ss_we(tmem + kQB, q, kDHi, bm_lo + 2 * kLo + ks * kStep, kDHi, mm, 1);
        mma_ss_we(tmem + kQB, k, kDHi, n2_lo + ks * kStep, kDHi, mm, 1);
        mma_ss_we(tmem + kQB, k, kDHi, n2_lo + kLo + ks * kStep, kDHi, mm, 1);
      }
      mma_commit_elect(&sm.done);
    }
    ok = wait_bar(&sm.done, phase++ & 1, abort, p.hdr, 75);
    tc_fence_after();
    if (ok && warp == 0 && more) load_state(next);
    // this thread's key, 16 steps: dq, dk, and three sums over the keys, by quarters of the lanes
    float* sums = reinterpret_cast<float*>(sm.n2);   // (which has been read) [3][4][64]; across [4][64], row_sum [4][128], inner [16]
    if (ok) {
      const uint8_t *qt = sm.qk[row >> 6], *kt = qt + kTileBytes;
#pragma unroll
      for (int j0 = 0; j0 < 16; j0 += 8) {
        float sy[8], sr[8], gu[8], kb[8], qb[8], kn[8];
        tmem_ld8(mine + kSY + c0 + j0, sy);
        tmem_ld8(mine + kSR + c0 + j0, sr);
        tmem_ld8(mine + kGU + c0 + j0, gu);
        tmem_ld8(mine + kKB + c0 + j0, kb);
        tmem_ld8(mine + kQB + c0 + j0, qb);
        tmem_ld8(mine + kKN + c0 + j0, kn);
        tmem_ld_wait();
        reg_tie(sy);
        reg_tie(sr);
        reg_tie(gu);
        reg_tie(kb);
        reg_tie(qb);
        reg_tie(kn);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = c0 + j0 + j;
          const float from = sm.c.from[i], to = sm.c.to[i], beta = sm.c.beta[i];
          const float kv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(kt + sw128_off16(i, row & 63)));
          const float qv = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(qt + sw128_off16(i, row & 63)));
          const float q1 = p.scale * from * sy[j], r1 = from * sr[j], wrote = to * gu[j];
          dq[j0 + j] += q1 + kb[j];
          dk[j0 + j] += wrote - beta * (r1 - kn[j]) + qb[j];
          sy[j] = kv * (r1 - kn[j]);
          sr[j] = fmaf(qv, q1, -beta * kv * r1);
          gu[j] = kv * wrote;
        }
        const float s0 = sum_columns(sy), s1 = sum_columns(sr), s2 = sum_columns(gu);
        if (lane < 8) {
          sums[quarter * kChunk + c0 + j0 + lane] = s0;
          sums[(4 + quarter) * kChunk + c0 + j0 + lane] = s1;
          sums[(8 + quarter) * kChunk + c0 + j0 + lane] = s2;
        }
      }
      if (lane < 16) sums[(12 + quarter) * kChunk + c0 + lane] = across;
      sums[16 * kChunk + (c0 >> 4) * 128 + row] = row_sum;
#pragma unroll
      for (int o = 16; o; o >>= 1) inner += __shfl_xor_sync(0xffffffffu, inner, o);
      if (lane == 0) sums[24 * kChunk + warp] = inner;
    }
    ok = !__syncthreads_or(!ok);
    if (!ok) break;
    if (warp == 0 && more) load_rest(next);
    if (last_head) {   // dq, dk by steps: through U's place
      uint8_t* to = sm.u[0] + (row >> 6) * kTileBytes;
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        uint8_t *first = to + sw128_off16(c0 + j, row & 63), *second = to + sw128_off16(c0 + j + 1, row & 63);
        store_pair(first, second, dq[j], dq[j + 1]);
        store_pair(first + 2 * kTileBytes, second + 2 * kTileBytes, dk[j], dk[j + 1]);
        dq[j] = dq[j + 1] = dk[j] = dk[j + 1] = 0.f;
      }
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0) {
        for (int kb = 0; kb < (p.K > 64 ? 2 : 1); ++kb) {
          tma_store_4d(&m.dq, sm.u[0] + kb * kTileBytes, kb * 64, (int)t0, (int)hk, (int)b);
          tma_store_4d(&m.dk, sm.u[1] + kb * kTileBytes, kb * 64, (int)t0, (int)hk, (int)b);
        }
        bulk_commit_group();
      }
    }
    if (warp == 2) {   // a lane has steps 2 l and 2 l + 1
      float z[2], rho[2], sigma[2], g[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        z[e] = rho[e] = sigma[e] = g[e] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          z[e] += sums[w * kChunk + i];
          rho[e] += sums[(4 + w) * kChunk + i];
          sigma[e] += sums[(8 + w) * kChunk + i];
          g[e] += sums[(12 + w) * kChunk + i];
        }
      }
      // pairs whose earlier step is in an earlier warp's columns: rows from a step on
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const float* of = sums + 16 * kChunk + c * 128;
        const float p0 = of[2 * lane] + of[64 + 2 * lane], p1 = of[2 * lane + 1] + of[65 + 2 * lane];
        const float rest = sum_behind(p0 + p1, lane) + p1;
        if (2 * lane >= 16 * (c + 1)) {
          g[0] += rest + p0;
          g[1] += rest;
        }
      }
      float all = lane < 16 ? sums[24 * kChunk + lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      // from a step to the chunk's end; the sums before it
      const float after = sum_behind(rho[0] + rho[1], lane), before = sum_before(sigma[0] + sigma[1], lane);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * lane + e;
        g[e] += all + after + rho[1] + (e ? 0.f : rho[0]) + before + (e ? sigma[0] : 0.f);
        const int64_t at = (b * p.T + t0 + i) * p.H + h;
        if (i < n && SSD_INDEX_OK(p.hdr, at, p.batch * p.T * p.H, 2018)) {
          p.dbeta[at] = sm.dot[i] - z[e];
          if (p.dg) p.dg[at] = g[e];
        }
      }
    }
    item = next;
  }
  if (tid == 0) bulk_wait_group<0>();
  if (!ok && warp == 0) {   // a load or a product may be on its way
    mma_commit_elect(&sm.drain);
    mbar_wait_bounded(&sm.drain, 0, kDrainNs);
    mbar_wait_bounded(&sm.loaded, (announced - 1) & 1, kDrainNs);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int KB>
cudaError_t walk_as(const Params& p, const TcMaps& m, const TcBuffers& buf, cudaStream_t st) {
  constexpr int smem = sizeof(BackSmem<KB>);
  static_assert(smem <= 232448, "shared memory of a block");
  const cudaError_t e = cudaFuncSetAttribute(delta_chain_back_kernel<KB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  delta_chain_back_kernel<KB><<<(unsigned)(p.batch * p.H), kWalkThreads, smem, st>>>(p, m, buf);
  return cudaGetLastError();
}

}  // namespace

namespace delta {

cudaError_t tc_backward_kernels(const Params& p, const TcMaps& m, const TcBuffers& buf, cudaStream_t st) {
  cudaError_t e = p.K <= 64 ? walk_as<1>(p, m, buf, st) : walk_as<2>(p, m, buf, st);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(delta_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(GradSmem));
  if (e != cudaSuccess) return e;
  int most = 0;   // blocks that run at once
  e = resident_blocks(delta_grad_kernel, kGradThreads, (int)sizeof(GradSmem), &most);
  if (e != cudaSuccess) return e;
  delta_grad_kernel<<<(unsigned)std::min<int64_t>(p.batch * p.nch * p.Hk, most), kGradThreads, sizeof(GradSmem), st>>>(p, m, buf);
  return cudaGetLastError();
}

}  // namespace delta
}  // namespace ssd
