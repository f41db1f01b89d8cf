// What the tensor-core kernels of the gated delta rule share: bounded waits, operands in two bf16 terms, the tiles that
// the chunk kernel leaves for the walks, and tensor maps.
#pragma once

#include <cuda.h>

#include "delta_rule.cuh"
#include "fp_helpers.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace delta {

using namespace tc;

// A square of chunk steps as the tensor core reads it: 64 rows of 64 bf16, 128-byte swizzled, hi term then lo.
constexpr uint32_t kTileBytes = kChunk * kChunk * 2;
// Of every chunk and head in the workspace: T = (I + A)^-1 diag(beta) hi and lo, P hi and lo, for the backward pass
// (I + A)^-1 hi and lo; and e^(sum of g up to a step), e^(sum behind it), beta, the first times the output's scale.
constexpr int kDecays = 4 * kChunk;
constexpr uint32_t kDecayBytes = kDecays * 4;
constexpr uint32_t square_bytes(bool backward) { return (backward ? 6 : 4) * kTileBytes; }

struct TcMaps {
  CUtensorMap q, k, v, y, dy, dq, dk, states;   // states: kept by the forward walk, or the backward's gradients
};

struct TcBuffers {
  uint8_t* squares;    // [b*nch*H][square]
  float* decays;       // [b*nch*H][4][kChunk]
  uint8_t* writes;     // backward: gradients of v - S k, [b*nch*H][2 blocks of 64 values][hi, lo][kTileBytes]
  uint32_t square;
};

// A sequence cut into segments that are walked at once, where there are fewer sequences than SMs.  A row s of the state
// becomes s M + n over a segment: a first pass (pre) walks every segment but the last from zero (the first from the
// initial state) for its n, and every one but the first and last from the rows of the identity, without values, for its M;
// a carry makes of them the state before every segment, and the full pass starts there.
struct Segments {
  int n, chunks, pre;   // segments of a sequence, chunks of a segment (the last may have fewer)
  float *start, *end, *map;   // [b*H*n][V][K]: states before and behind segments; [b*H*n][K][K]: M
};

constexpr long long kWaitCycles = 4000000000ll;   // a wait gives up after about 2 s

static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, WsHeader* hdr, int site) {
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitCycles) {
      *abort = 1;
      if (hdr) latch_error(hdr, SSD_ERR_TIMEOUT, site);
      return false;
    }
  }
}
// A wait that gave up has set the flag, which ends all others of the block.  Its warp must still meet every barrier that it
// shares with warps whose waits came through: it goes on without waiting, or all settle it at a barrier.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, WsHeader* hdr, int site) {
#ifdef SSD_INDEX_CHECKS
  // How a test comes to what is behind a wait that ran out: the workspace names the site and the warps.
  if (hdr && hdr->give_up_site == (uint32_t)site && (hdr->give_up_warps >> (threadIdx.x / 32) & 1)) {
    *abort = 1;
    latch_error(hdr, SSD_ERR_TIMEOUT, site);
    return false;
  }
#endif
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, hdr, site);
}
constexpr uint64_t kDrainNs = 2000000000ull;   // that a block waits at its end for its own copies and products

// v = hi + lo, two bf16 terms with 16 bits of mantissa between them, for a pair of values (the first in the low half).
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// A pair of values as bf16 to two rows of a tile, two bytes each.  (Converted together: a single conversion takes four
// times a pair's.)
__device__ __forceinline__ void store_pair(uint8_t* first, uint8_t* second, float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  *reinterpret_cast<__nv_bfloat16*>(first) = __low2bfloat16(h);
  *reinterpret_cast<__nv_bfloat16*>(second) = __high2bfloat16(h);
}
// Both terms: hi there, lo `lo` bytes further.
__device__ __forceinline__ void store_pair_terms(uint8_t* first, uint8_t* second, uint32_t lo, float a, float b) {
  uint32_t h, l;
  split2(a, b, h, l);
  *reinterpret_cast<uint16_t*>(first) = (uint16_t)h;
  *reinterpret_cast<uint16_t*>(second) = (uint16_t)(h >> 16);
  *reinterpret_cast<uint16_t*>(first + lo) = (uint16_t)l;
  *reinterpret_cast<uint16_t*>(second + lo) = (uint16_t)(l >> 16);
}

// 1-D copy global -> shared by one elected lane; addresses and size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load_elect(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// 32 bytes at once where the row starts on such a border (`wide`), else value by value.
__device__ __forceinline__ void store8(float* p, const float* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = v[i];
  }
}

// N values of a row, zeros behind its end; rows are multiples of eight values.
template <int N>
__device__ __forceinline__ void load_row(float (&v)[N], const float* p, int64_t left) {
  const bool wide = (reinterpret_cast<uintptr_t>(p) & 15) == 0;
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (k < left) {
      if (wide) f = *reinterpret_cast<const float4*>(p + k);
      else f = make_float4(p[k], p[k + 1], p[k + 2], p[k + 3]);
    }
    v[k] = f.x;
    v[k + 1] = f.y;
    v[k + 2] = f.z;
    v[k + 3] = f.w;
  }
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// 8 consecutive columns of TMEM.
__device__ __forceinline__ void tmem_st8u(uint32_t at, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

constexpr uint32_t kDHi = sdesc_sw128_hi(1024);
constexpr uint32_t kLo = kTileBytes >> 4;   // from a square's hi to its lo, in a descriptor's units

// Two terms of 16 columns, written over the 16 columns' place: hi in the first 8, lo in the others; as an operand this is
// one k-step of hi and one of lo.
__device__ __forceinline__ void store_terms(uint32_t at, const float (&v)[16]) {
  uint32_t u[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) split2(v[2 * j], v[2 * j + 1], u[j], u[8 + j]);
  tmem_st16u(at, u);
}

// The walks' 16 state warps, four to each quarter of the lanes: a thread has a value's quarter of the keys, and 16 steps
// of a chunk.  (Eight warps with halves: 2.44 us a chunk instead of 2.24; what they do between two products is a
// chain of latencies.)
constexpr int kStateWarps = 16, kWalkThreads = 22 * 32;   // and four at the output, one for products, one for loads

// The two terms of a thread's keys: hi at `at`, lo `lo` columns further.
template <int N>
__device__ __forceinline__ void store_state_terms(uint32_t at, uint32_t lo_at, const float (&S)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 16) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) split2(S[k + 2 * j], S[k + 2 * j + 1], hi[j], lo[j]);
    tmem_st8u(at + k / 2, hi);
    tmem_st8u(at + lo_at + k / 2, lo);
  }
}

// 16 of a thread's keys (from `first` of its quarter) of the state at a chunk's border, through shared memory: rows of 64
// bytes, swizzled, leave as one tile of `map`.  By the four warps of a quarter of the keys.  (Straight from the
// registers, 32 bytes of 32 rows an instruction, the forward walk took a third longer.)
template <int KQ>
__device__ __forceinline__ void send_state(uint8_t* to, const CUtensorMap* map, const float (&S)[KQ], int quarter, int first,
                                           int v0, int cell, int64_t K) {
  const int t = threadIdx.x & 127;
  if (t == 0) bulk_wait_group_read<0>();   // the tile before has left
  named_barrier(2 + quarter, 128);
  const uint32_t at = smem_u32(to) + t * 64 + (((t >> 1) & 3) << 4);
#pragma unroll
  for (int k = 0; k < 16; k += 4)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (k << 2)), "f"(S[first + k]), "f"(S[first + k + 1]),
                 "f"(S[first + k + 2]), "f"(S[first + k + 3])
                 : "memory");
  fence_proxy_async_smem();
  named_barrier(2 + quarter, 128);
  if (t == 0 && quarter * KQ + first < K) {
    tma_store_4d(map, to, quarter * KQ + first, v0, cell, 0);
    bulk_commit_group();
  }
}

// Whether the tensor-core kernels take a call, its workspace, and the call itself (delta_rule_tc.cu).
bool tc_takes(const Params& p, bool backward);
size_t tc_bytes(int64_t batch, int64_t nch, int64_t H, int64_t V, int64_t K, bool backward);
cudaError_t tc_forward(const Params& p, void* buffers, cudaStream_t st);
cudaError_t tc_backward(const Params& p, bool states_known, void* buffers, cudaStream_t st);   // fills states_in where not
// The backward walk and the chunks' gradients (delta_rule_tc_back.cu).
cudaError_t tc_backward_kernels(const Params& p, const TcMaps& m, const TcBuffers& buf, cudaStream_t st);
bool head_map(CUtensorMap* m, const void* base, int64_t batch, int64_t T, int64_t heads, int64_t cols, const int64_t* stride);
bool state_map(CUtensorMap* m, const void* base, int64_t cells, int64_t V, int64_t K);

}  // namespace delta
}  // namespace ssd
