// Log probabilities of given tokens, entropy and the likeliest tokens of rows of
// logits (sm_103a): the plain form.  A CTA a row; a pass for the largest logit,
// one for the sums, and one for each alternative.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "drafts.h"

namespace ta {
namespace {

constexpr int kThreads = 256;
typedef unsigned long long u64;

template <class T>
__device__ __forceinline__ float value(const T* row, int i) { return (float)row[i]; }

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}

template <class F>
__device__ __forceinline__ u64 block_max(u64 x, u64* s, F) {
  for (int o = 16; o; o >>= 1) {
    const u64 y = __shfl_xor_sync(0xffffffffu, x, o);
    x = y > x ? y : x;
  }
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = s[0];
  for (int w = 1; w < kThreads / 32; ++w) x = s[w] > x ? s[w] : x;
  __syncthreads();
  return x;
}

__device__ __forceinline__ float block_sum(float x, float* s) {
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0;
  for (int w = 0; w < kThreads / 32; ++w) x += s[w];
  __syncthreads();
  return x;
}

template <class T>
__global__ void __launch_bounds__(kThreads) scores_kernel(const ScoreParams p) {
  __shared__ u64 s_max[32];
  __shared__ float s_sum[32];
  const T* row = static_cast<const T*>(p.logits) + blockIdx.x * p.stride;
  const int tid = threadIdx.x, r = blockIdx.x;
  auto id = [] {};
  u64 best = 0;
  bool nan = false;
  for (int i = tid; i < p.vocab; i += kThreads) {
    const float x = value(row, i);
    nan |= x != x;
    const u64 k = ((u64)key_of(x) << 32) | (uint32_t)~i;
    best = k > best ? k : best;
  }
  nan = __syncthreads_or(nan);
  best = block_max(best, s_max, id);
  const int at = (int)~(uint32_t)best;
  const float top = value(row, at);
  const bool broken = nan || top == -INFINITY;
  const float T0 = p.temperature ? p.temperature[r] : p.temperature_all;
  const bool greedy = !(T0 > 0);
  const float inv = greedy ? 1.f : 1.f / T0;
  // (max - x) / T of a logit: 0 for the largest, also where it is infinite
  auto below = [&](float x, int i) -> float {
    if (greedy) return i == at ? 0.f : INFINITY;
    return x == top ? 0.f : (top - x) * inv;
  };
  float sum = 0, dot = 0;
  for (int i = tid; i < p.vocab; i += kThreads) {
    const float y = below(value(row, i), i), w = expf(-y);
    sum += w;
    if (w > 0) dot += w * y;
  }
  sum = block_sum(sum, s_sum);
  dot = block_sum(dot, s_sum);
  const float ln = logf(sum);
  if (tid == 0 && p.entropy) p.entropy[r] = broken ? NAN : ln + dot / sum;
  for (int g = tid; g < p.n_given; g += kThreads) {
    const int i = p.given[(long long)r * p.n_given + g];
    const bool in = i >= 0 && i < p.vocab;
    p.given_logprobs[(long long)r * p.n_given + g] = broken || !in ? NAN : -below(value(row, i), i) - ln;
  }
  u64 last = ~0ull;
  for (int k = 0; k < p.top; ++k) {
    u64 most = 0;
    for (int i = tid; !broken && i < p.vocab; i += kThreads) {
      const float x = value(row, i);
      const u64 key = ((u64)key_of(x) << 32) | (uint32_t)~i;
      if (x > -INFINITY && key < last && key > most) most = key;
    }
    most = block_max(most, s_max, id);
    last = most;
    if (tid == 0) {
      const int i = (int)~(uint32_t)most;
      const long long to = (long long)r * p.top + k;
      p.top_tokens[to] = most ? i : -1;
      p.top_logprobs[to] = broken ? NAN : most ? -below(value(row, i), i) - ln : -INFINITY;
    }
  }
}

}  // namespace

cudaError_t launch_token_logprobs(const ScoreParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.rows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  if (p.dtype == kFp32) return cudaLaunchKernelEx(&cfg, scores_kernel<float>, p);
  return p.dtype == kFp16 ? cudaLaunchKernelEx(&cfg, scores_kernel<__half>, p)
                          : cudaLaunchKernelEx(&cfg, scores_kernel<__nv_bfloat16>, p);
}

}  // namespace ta
