// Attention of several new tokens of each request over its pages (sm_103a): the
// plain form.  A warp a (token, q head): 32 keys a step, one a lane, with a
// running maximum and sum, then V's rows with the weights handed round.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "drafts.h"

namespace ta {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kBadOffsets = 256;

struct Chunk {
  int len, n, tok0;
};
__device__ __forceinline__ Chunk checked(const ChunkParams& p, int b, int& bad) {
  Chunk r;
  const int len = p.lens[b];
  int first = b, last = b + 1;
  if (p.cu) first = p.cu[b], last = p.cu[b + 1];
  if (len < 0 || len > p.width * kPage) bad |= kBatchBadInput;
  if (first < 0 || last < first || last > p.n_tokens) bad |= kBatchBadInput | kBadOffsets;
  r.len = min(max(len, 0), p.width * kPage);
  r.tok0 = min(max(first, 0), p.n_tokens);
  r.n = min(max(last, r.tok0), p.n_tokens) - r.tok0;
  if (p.parents && r.n > kMaxNodes) bad |= kBatchBadInput, r.n = 0;
  return r;
}

template <class T, int D>
__global__ void __launch_bounds__(256) chunk_rows_kernel(const ChunkParams p) {
  __shared__ float s_q[8][D];
  __shared__ Chunk s_r;
  __shared__ int s_b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tok = blockIdx.x;
  if (tid == 0) s_b = -1;
  __syncthreads();
  int bad = 0;
  for (int b = tid; b < p.n_req; b += 256) {
    const Chunk r = checked(p, b, bad);
    if (tok >= r.tok0 && tok < r.tok0 + r.n) s_b = b, s_r = r;
  }
  const bool broken = __syncthreads_or(bad & kBadOffsets);
  if (tok == 0 && bad && p.status) atomicOr(p.status, bad & ~kBadOffsets);
  const int b = broken ? -1 : s_b;
  const Chunk r = s_r;
  const T* K = reinterpret_cast<const T*>(p.k_pages);
  const T* V = reinterpret_cast<const T*>(p.v_pages);
  for (int h = warp; h < p.hq; h += 8) {
    const long long row = (long long)tok * p.hq + h;
    T* out = reinterpret_cast<T*>(p.out) + row * D;
    float m = -INFINITY, l = 0, o[D / 32] = {};
    if (b >= 0) {
      const T* q = reinterpret_cast<const T*>(p.q) + tok * p.q_stride + h * D;
      __syncwarp();
      for (int c = lane; c < D; c += 32) s_q[warp][c] = (float)q[c] * p.scale_log2;
      __syncwarp();
      const int i = tok - r.tok0, base = r.len - r.n;
      unsigned sees[kMaxNodes / 32] = {};
      if (p.parents) {
        int at = i;
        while (at >= 0) {
          sees[at >> 5] |= 1u << (at & 31);
          const int up = p.parents[r.tok0 + at];
          if ((up < -1 || up >= at) && p.status && lane == 0) atomicOr(p.status, kBatchBadInput);
          at = up >= at ? -1 : up;
        }
      }
      const int end = max(min(base + i + 1, r.len), 0);
      const int32_t* table = p.table + b * p.table_stride;
      for (int k0 = 0; k0 < end; k0 += 32) {
        const int key = k0 + lane, node = key - base;
        const bool in = key < end && (!p.parents || node < 0 || (sees[node >> 5] >> (node & 31) & 1));
        int page = key < end ? table[key / kPage] : 0;
        if ((unsigned)page >= (unsigned)p.num_pages) {
          if (p.status) atomicOr(p.status, kBatchBadSlot);
          page = -1;
        }
        const long long at = (((long long)page * p.hkv + h / p.gqa) * kPage + key % kPage) * D;
        float x = in ? 0.f : -INFINITY;
        if (in && page >= 0)
          for (int c = 0; c < D; ++c) x = fmaf((float)K[at + c], s_q[warp][c], x);
        float top = x;
        for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        top = fmaxf(top, m);
        if (top == -INFINITY) continue;
        const float alpha = exp2f(m - top), w = exp2f(x - top);
        m = top;
        l = l * alpha + w;
        for (int e = 0; e < D / 32; ++e) o[e] *= alpha;
        for (int s = 0; s < 32; ++s) {
          const float ws = __shfl_sync(0xffffffffu, w, s);
          const long long as = __shfl_sync(0xffffffffu, at, s);
          const int ps = __shfl_sync(0xffffffffu, page, s);
          if (ws > 0 && ps >= 0)
            for (int e = 0; e < D / 32; ++e) o[e] = fmaf(ws, (float)V[as + e * 32 + lane], o[e]);
        }
      }
      for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    }
    const float inv = l > 0 ? 1 / l : l == 0 ? 0 : l;
    for (int e = 0; e < D / 32; ++e) out[e * 32 + lane] = (T)(o[e] * inv);
    if (lane == 0 && p.lse) p.lse[row] = l == 0 ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <class T>
cudaError_t run(const ChunkParams& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_tokens);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  return p.d == 128 ? cudaLaunchKernelEx(&cfg, chunk_rows_kernel<T, 128>, p)
                    : cudaLaunchKernelEx(&cfg, chunk_rows_kernel<T, 64>, p);
}

}  // namespace

size_t chunk_workspace(const ChunkParams& p) { return 0; }

cudaError_t launch_chunk_attention(const ChunkParams& p, void* workspace, cudaStream_t s) {
  if (p.n_tokens == 0) return cudaSuccess;
  return p.dtype == kFp16 ? run<__half>(p, s) : run<__nv_bfloat16>(p, s);
}

}  // namespace ta
