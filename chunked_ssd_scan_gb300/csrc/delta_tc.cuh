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
// Of every chunk and head in the workspace: T = (I + A)^-1 diag(beta) hi and lo, P hi and lo, then e^(sum of g up to a
// step) and e^(sum behind it).
constexpr uint32_t kSquareBytes = 4 * kTileBytes, kDecayBytes = 2 * kChunk * 4;

struct TcMaps {
  CUtensorMap q, k, v, y, dy, dv, dq, dk, states;
};

struct TcBuffers {
  uint8_t* squares;   // [b*nch*H][kSquareBytes]
  float* decays;      // [b*nch*H][2][kChunk]
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
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort, WsHeader* hdr, int site) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort, hdr, site);
}

// v = hi + lo, two bf16 terms with 16 bits of mantissa between them, for a pair of values (the first in the low half).
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
  lo = *reinterpret_cast<const uint32_t*>(&l);
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

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Whether the tensor-core kernels take a call, its workspace, and the call itself (delta_rule_tc.cu).
bool tc_takes(const Params& p, bool backward);
size_t tc_forward_bytes(int64_t batch, int64_t nch, int64_t H);
cudaError_t tc_forward(const Params& p, void* buffers, cudaStream_t st);

}  // namespace delta
}  // namespace ssd
