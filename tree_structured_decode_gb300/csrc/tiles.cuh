// What the kernels of 128-row attention tiles on tcgen05 share: bounded waits, the
// weights' rounding, the accumulator's rescaling.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "batch.h"
#include "ptx.cuh"

namespace ta {
namespace tiles {

constexpr long long kWaitLimitNs = 2000000000ll, kDrainLimitNs = 200000000ll;

// Out of line, once per register split: a call must match its caller's.
template <int kRole>
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                       int32_t* status) {
  if (*abort_flag) return false;
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t n = 1;; ++n) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((n & 15) == 0) {
      if (*abort_flag) return false;
      if ((long long)(ptx::globaltimer() - t0) > kWaitLimitNs) {
        *abort_flag = 1;
        if (status) atomicOr(status, kBatchTimeout);
        return false;
      }
    }
  }
}
// True once the phase is complete; false when the CTA has given up.  The same in
// all lanes of the warp.
template <int kRole>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* status) {
  bool ok = ptx::mbar_try_wait(bar, parity);
  if (!ok) ok = wait_slow<kRole>(bar, parity, abort_flag, status);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity))
    if ((long long)(ptx::globaltimer() - t0) > kDrainLimitNs) return;
}

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kHalf) return ptx::pack_f16(lo, hi);
  return ptx::pack_bf16(lo, hi);
}

template <int D>
__device__ __noinline__ void rescale_o(uint32_t o, float alpha) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float v[32];
    ptx::tmem_ld32(o + c * 32, v);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] *= alpha;
    ptx::tmem_st32(o + c * 32, v);
  }
  ptx::tmem_wait_st();
}

}  // namespace tiles
}  // namespace ta
