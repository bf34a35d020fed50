// Which drafts of a verified tree stand, and their keys and values moved together
// (sm_103a).  Both are a few words a request: bound by the launch and the loads
// that depend on one another.  In a graph, both kernels: 4.3 us for 4 trees of 8
// nodes, 6.6 for 64 of up to 60 with 16 layers' keys and values (8 x 128), whose
// bytes take 2.5.
#include <cuda_runtime.h>

#include <cstdint>

#include "drafts.h"

namespace ta {
namespace {

// A request's nodes [tok0, tok0 + n), if its offsets lie in the batch.
struct Nodes {
  int tok0, n;
  bool ok;
};
__device__ __forceinline__ Nodes nodes_of(const int32_t* cu, int b, int n_tokens) {
  int first = b, last = b + 1;
  if (cu) first = cu[b], last = cu[b + 1];
  const bool ok = first >= 0 && last >= first && last <= n_tokens;
  return Nodes{ok ? first : 0, ok ? last - first : 0, ok};
}

// A warp a request; lane i holds nodes i, i + 32, ...: whether a node's token is
// what was drawn above it needs no walk, so a level of the path is four ballots.
constexpr int kAcceptThreads = 256;
constexpr int kPerLane = kMaxNodes / 32;

__global__ void __launch_bounds__(kAcceptThreads) accept_drafts_kernel(const AcceptParams p) {
  constexpr int kWarps = kAcceptThreads / 32;
  __shared__ int32_t s_drawn[kWarps][kMaxNodes], s_path[kWarps][kMaxNodes];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // offsets out of order could give a token to many requests: then none has nodes
  bool broken = false;
  for (int b = threadIdx.x; p.cu && b < p.n_req; b += kAcceptThreads) broken |= !nodes_of(p.cu, b, p.n_tokens).ok;
  broken = __syncthreads_or(broken);
  const int b = blockIdx.x * kWarps + warp;
  int bad = broken ? kBatchBadInput : 0;

  // tokens of no request
  const int end = broken ? 0 : p.cu ? (p.n_req > 0 ? p.cu[p.n_req] : 0) : p.n_tokens;
  for (long long t = (broken ? 0 : (long long)end) + (long long)blockIdx.x * kAcceptThreads + threadIdx.x; t < p.n_tokens;
       t += (long long)gridDim.x * kAcceptThreads)
    p.path[t] = -1;
  const int before = !broken && p.cu && p.n_req > 0 ? p.cu[0] : 0;
  for (int t = blockIdx.x * kAcceptThreads + threadIdx.x; t < before; t += gridDim.x * kAcceptThreads) p.path[t] = -1;

  if (b < p.n_req) {
    const Nodes r = broken ? Nodes{0, 0, true} : nodes_of(p.cu, b, p.n_tokens);
    int kept = 0, next = -1;
    if (r.n > kMaxNodes) {
      bad |= kBatchBadInput;
      for (int i = lane; i < r.n; i += 32) p.path[r.tok0 + i] = -1;
    } else if (r.n > 0) {
      int parent[kPerLane], drafted[kPerLane];
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        const int i = k * 32 + lane;
        const bool in = i < r.n;
        parent[k] = in ? p.parents[r.tok0 + i] : -1;
        drafted[k] = in ? p.drafted[r.tok0 + i] : -1;
        s_drawn[warp][i] = in ? p.sampled[r.tok0 + i] : -1;
        s_path[warp][i] = -1;
        if (parent[k] < -1 || parent[k] >= i) {
          if (in) bad |= kBatchBadInput;
          parent[k] = -1;
        }
      }
      __syncwarp();
      // parent[k] = the node above that drew this one's token, or -1
#pragma unroll
      for (int k = 0; k < kPerLane; ++k)
        if (parent[k] >= 0 && (drafted[k] < 0 || drafted[k] != s_drawn[warp][parent[k]])) parent[k] = -1;
      int at = 0;
      while (true) {  // nodes rise along the path, so this ends
        if (lane == 0) s_path[warp][kept] = at;
        ++kept;
        int child = -1;
#pragma unroll
        for (int k = kPerLane - 1; k >= 0; --k) {
          const unsigned hit = __ballot_sync(0xffffffffu, parent[k] == at);
          if (hit) child = k * 32 + __ffs(hit) - 1;
        }
        if (child < 0) break;
        at = child;
      }
      next = s_drawn[warp][at];
      __syncwarp();
      for (int i = lane; i < r.n; i += 32) p.path[r.tok0 + i] = s_path[warp][i];
    }
    if (lane == 0) {
      p.kept[b] = kept;
      p.next[b] = next;
      if (p.back) p.back[b] = kept - r.n;
    }
  }
  if (bad && p.status) atomicOr(p.status, bad);
}

// A block a request and layer.  Its threads own 16-byte columns of a token's row
// and walk the path upwards, kAtOnce moves loaded before any of them is stored:
// place i is written after node path[i] >= i has been read, and later nodes lie
// above it.  (One at a time: 6.9 us for the 64 trees above, eight 7.1.)
constexpr int kKeepThreads = 128, kAtOnce = 4, kListed = 128;

__global__ void __launch_bounds__(kKeepThreads) keep_drafts_kernel(const KeepParams p) {
  __shared__ long long s_from[kListed], s_to[kListed];  // elements, of head 0
  __shared__ int s_moves, s_more;
  const int b = blockIdx.x, tid = threadIdx.x;
  const Nodes r = nodes_of(p.cu, b, p.n_tokens);
  const int len = p.lens[b];
  const long long base = (long long)len - r.n;  // (any 32 bits may stand in lens)
  if (tid == 0 && !r.ok && p.status) atomicOr(p.status, kBatchBadInput);
  const int chunks = p.d / 8, pieces = p.hkv * chunks;
  uint16_t* const k = p.k_pages + (long long)blockIdx.y * p.layer_stride;
  uint16_t* const v = p.v_pages + (long long)blockIdx.y * p.layer_stride;
  const int32_t* table = p.table + (long long)b * p.table_stride;
  for (int i0 = 0; i0 < r.n; i0 += kListed) {
    if (tid < 32) {  // the first warp lists the next moves
      int moves = 0, bad = 0;
      bool more = true;
      for (int i1 = i0; more && i1 < min(i0 + kListed, r.n); i1 += 32) {
        const int i = i1 + tid;
        const int from = i < r.n ? p.path[r.tok0 + i] : -1;
        const int prev = i < r.n && i > 0 ? p.path[r.tok0 + i - 1] : -1;
        const bool ends = from == -1;
        const long long at = base + from, to = base + i;
        bool fine = from >= 0 && from > prev && from < r.n && base >= 0 && len <= (long long)p.width * kPage;
        long long source = 0, target = 0;
        if (fine && from != i) {
          const int a = table[at / kPage], z = table[to / kPage];
          fine = (unsigned)a < (unsigned)p.num_pages && (unsigned)z < (unsigned)p.num_pages;
          if (!fine) bad |= kBatchBadSlot;
          source = ((long long)a * p.hkv * kPage + at % kPage) * p.d;
          target = ((long long)z * p.hkv * kPage + to % kPage) * p.d;
        } else if (!ends && !fine) {
          bad |= kBatchBadInput;
        }
        const unsigned stop = ~__ballot_sync(0xffffffffu, fine);
        const int count = stop ? __ffs(stop) - 1 : 32;  // path entries before the first that ends it
        if (tid > count) bad = 0;                      // what lies behind it is not looked at
        const unsigned listed = __ballot_sync(0xffffffffu, tid < count && from != i);
        if (tid < count && from != i) {
          const int n = moves + __popc(listed & ((1u << tid) - 1));
          s_from[n] = source;
          s_to[n] = target;
        }
        moves += __popc(listed);
        more = count == 32;
      }
      if (bad && p.status) atomicOr(p.status, bad);
      if (tid == 0) s_moves = moves, s_more = more;
    }
    __syncthreads();
    const int moves = s_moves;
    for (int c = tid; c < pieces; c += kKeepThreads) {
      const long long in = (long long)(c / chunks) * kPage * p.d + (c % chunks) * 8;
      for (int m = 0; m < moves; m += kAtOnce) {
        uint4 kk[kAtOnce], vv[kAtOnce];
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
          if (m + e < moves) {
            kk[e] = *reinterpret_cast<const uint4*>(k + s_from[m + e] + in);
            vv[e] = *reinterpret_cast<const uint4*>(v + s_from[m + e] + in);
          }
#pragma unroll
        for (int e = 0; e < kAtOnce; ++e)
          if (m + e < moves) {
            *reinterpret_cast<uint4*>(k + s_to[m + e] + in) = kk[e];
            *reinterpret_cast<uint4*>(v + s_to[m + e] + in) = vv[e];
          }
      }
    }
    if (!s_more) break;
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_accept_drafts(const AcceptParams& p, cudaStream_t s) {
  if (p.n_req == 0 && p.n_tokens == 0) return cudaSuccess;
  constexpr int kWarps = kAcceptThreads / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.n_req / kWarps + 1));
  cfg.blockDim = dim3(kAcceptThreads);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, accept_drafts_kernel, p);
}

cudaError_t launch_keep_drafts(const KeepParams& p, cudaStream_t s) {
  if (p.n_req == 0 || p.n_tokens == 0 || p.layers == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_req, p.layers);
  cfg.blockDim = dim3(kKeepThreads);
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, keep_drafts_kernel, p);
}

}  // namespace ta
