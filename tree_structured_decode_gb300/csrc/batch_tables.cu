// Page tables and slot maps built on the GPU, and the append by slot.
#include <cuda_runtime.h>
#include <cooperative_groups.h>

#include <cstdint>

#include "batch.h"

namespace ta {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;

// Inclusive scan of three sums over the block (32 warps), 64 bits: lengths
// come from the device and their sums may pass 32 bits before they are checked.
struct Sum3 {
  long long a, b, c;
};
__device__ __forceinline__ Sum3 add(const Sum3& x, const Sum3& y) {
  return {x.a + y.a, x.b + y.b, x.c + y.c};
}
__device__ __forceinline__ Sum3 scan_warp(Sum3 v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Sum3 o{__shfl_up_sync(0xffffffffu, v.a, off), __shfl_up_sync(0xffffffffu, v.b, off),
                 __shfl_up_sync(0xffffffffu, v.c, off)};
    if (lane >= off) v = add(v, o);
  }
  return v;
}

// Last index i in [0, n) with off[i] <= x (off ascending, off[0] = 0 <= x).
__device__ __forceinline__ int find_owner(const int32_t* off, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Per request: tokens to add, pages to take, pages to give back.
struct Step {
  int add, need, back;
};
__device__ __forceinline__ Step step_of(int len, int n) {
  const int after = max(len + n, 0);
  const int old = (len + kPage - 1) / kPage, now = (after + kPage - 1) / kPage;
  return {max(n, 0), max(now - old, 0), max(old - now, 0)};
}

// One cluster (of one or eight CTAs) does the whole operator: every CTA scans
// all requests (a few loads a thread, from L2), then takes its share of new
// pages and tokens; cluster barriers stand between the phases that read a
// state and the ones that change it.  What is read and written is two ints a
// new token, so the time is launch, one scan and two barriers' latency: 4 us for
// 256 requests with a token each, 12 us for 100000 tokens.
//
//   need_b = pages(len_b + n_b) - pages(len_b)      (n_b > 0)
//   page j of the request's new ones = free[n_free - 1 - (sum of need before b + j)]
//   slot(pos) = table[b][pos / 16] * 16 + pos % 16
__global__ void __launch_bounds__(kThreads, 1) extend_tables_kernel(const ExtendParams p) {
  extern __shared__ int32_t smem[];
  int32_t* s_cu = smem;                     // new tokens before request b
  int32_t* s_need = s_cu + p.n_req + 1;     // pages taken before
  int32_t* s_back = s_need + p.n_req + 1;   // pages given back before
  __shared__ Sum3 s_warp[32];
  __shared__ int s_bad;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_bad = 0;
  __syncthreads();

  // ---- scan: a run of consecutive requests per thread
  const int per = (p.n_req + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.n_req), b1 = min(b0 + per, p.n_req);
  const long long room = (long long)p.width * kPage;
  Sum3 mine{0, 0, 0};
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = p.lens[b], n = p.n_new[b];
    if (len < 0 || len > room)
      bad |= kBatchBadInput;
    else if (n > 0 && (long long)len + n > room)
      bad |= kBatchTableFull;
    else {
      const Step s = step_of(len, max(n, -len));
      mine = add(mine, {s.add, s.need, s.back});
    }
  }
  if (bad) atomicOr(&s_bad, bad);
  Sum3 v = scan_warp(mine, lane);
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    const Sum3 w = scan_warp(s_warp[lane], lane);
    s_warp[lane] = w;
  }
  __syncthreads();
  const Sum3 total = s_warp[31];
  const int n_free = *p.n_free;
  bad = s_bad;
  if (n_free < 0 || n_free > p.free_cap)
    bad |= kBatchBadInput;
  else if (total.b > n_free)
    bad |= kBatchNoPages;
  else if (n_free - total.b + total.c > p.free_cap)
    bad |= kBatchBadInput;
  if (total.a > p.max_new) bad |= kBatchTableFull;
  if (bad) {
    // all or nothing: no token has a slot, the state stays as it is
    for (int t = rank * kThreads + tid; t < p.max_new; t += ranks * kThreads)
      p.slots[t] = p.positions[t] = -1;
    if (p.cu_new)
      for (int b = rank * kThreads + tid; b <= p.n_req; b += ranks * kThreads) p.cu_new[b] = 0;
    if (rank == 0 && tid == 0 && p.status) atomicOr(p.status, bad);
    return;  // every CTA of the cluster alike
  }
  {
    Sum3 at{v.a - mine.a, v.b - mine.b, v.c - mine.c};  // before this thread, in its warp
    if (warp > 0) at = add(at, s_warp[warp - 1]);
    for (int b = b0; b < b1; ++b) {
      const int len = p.lens[b];
      const Step s = step_of(len, max(p.n_new[b], -len));
      s_cu[b] = (int32_t)at.a;
      s_need[b] = (int32_t)at.b;
      s_back[b] = (int32_t)at.c;
      at = add(at, {s.add, s.need, s.back});
    }
  }
  const int n_add = (int)total.a, n_need = (int)total.b, n_back = (int)total.c;
  if (tid == 0) {
    s_cu[p.n_req] = n_add;
    s_need[p.n_req] = n_need;
    s_back[p.n_req] = n_back;
  }
  __syncthreads();

  // ---- the state is read; new table entries and the outputs are written
  if (p.cu_new)
    for (int b = rank * kThreads + tid; b <= p.n_req; b += ranks * kThreads) p.cu_new[b] = s_cu[b];
  for (int e = rank * kThreads + tid; e < n_need; e += ranks * kThreads) {
    const int b = find_owner(s_need, p.n_req, e);
    const int old = (p.lens[b] + kPage - 1) / kPage;
    p.table[(long long)b * p.table_stride + old + (e - s_need[b])] = p.free_pages[n_free - 1 - e];
  }
  for (int t = rank * kThreads + tid; t < p.max_new; t += ranks * kThreads) {
    int slot = -1, position = -1;
    if (t < n_add) {
      const int b = find_owner(s_cu, p.n_req, t);
      const int len = p.lens[b], pos = len + (t - s_cu[b]);
      const int old = (len + kPage - 1) / kPage, j = pos / kPage;
      const int page = j < old ? p.table[(long long)b * p.table_stride + j]
                               : p.free_pages[n_free - 1 - (s_need[b] + j - old)];
      if ((unsigned)page < kMaxPages)
        slot = page * kPage + pos % kPage;
      else if (p.status)
        atomicOr(p.status, kBatchBadSlot);
      position = p.position_base + pos;
    }
    p.slots[t] = slot;
    p.positions[t] = position;
  }
  cluster.sync();
  // ---- pages given back, the last one lowest: an extension taken back
  // leaves the stack bit for bit as it was
  if (n_back > 0) {
    for (int e = rank * kThreads + tid; e < n_back; e += ranks * kThreads) {
      const int b = find_owner(s_back, p.n_req, e);
      const int len = p.lens[b];
      const int now = (len + max(p.n_new[b], -len) + kPage - 1) / kPage;
      p.free_pages[n_free - n_need + n_back - 1 - e] =
          p.table[(long long)b * p.table_stride + now + (e - s_back[b])];
    }
    cluster.sync();
  }
  for (int b = rank * kThreads + tid; b < p.n_req; b += ranks * kThreads) {
    const int len = p.lens[b];
    p.lens[b] = len + max(p.n_new[b], -len);
  }
  if (rank == 0 && tid == 0) *p.n_free = n_free - n_need + n_back;
}

// A warp copies up to 128 16-byte pieces (2 KB) of a token's K and the same of
// its V: eight loads in flight a lane.  A piece's head and place follow by
// shifts (d / 8 pieces a head).  Reads and writes each byte once: bound by DRAM
// (131 MB in 20 us, 6.5 TB/s) or, for a few tokens, by the launch (2.5 us).
template <int kShift>  // log2(d / 8)
__global__ void __launch_bounds__(256) append_slots_kernel(const AppendSlotsParams p, int parts) {
  const int lane = threadIdx.x & 31;
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int t = (int)(w / parts), part = (int)(w % parts);
  if (t >= p.n_tokens) return;
  const int slot = __ldg(p.slots + t);
  if (slot < 0 || slot >= p.n_slots) {
    if (slot != -1 && lane == 0 && part == 0 && p.status) atomicOr(p.status, kBatchBadSlot);
    return;
  }
  const int pieces = p.hkv << kShift;
  const uint4* ks = reinterpret_cast<const uint4*>(p.k_new + t * p.k_stride);
  const uint4* vs = reinterpret_cast<const uint4*>(p.v_new + t * p.v_stride);
  uint4 kv[4], vv[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = part * 128 + i * 32 + lane;
    if (c < pieces) {
      kv[i] = __ldg(ks + c);
      vv[i] = __ldg(vs + c);
    }
  }
  uint4* kd = reinterpret_cast<uint4*>(p.k_pages);
  uint4* vd = reinterpret_cast<uint4*>(p.v_pages);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = part * 128 + i * 32 + lane;
    if (c < pieces) {
      const int h = c >> kShift, in = c & ((1 << kShift) - 1);
      const long long at =
          ((((long long)(slot >> 4) * p.hkv + h) * kPage + (slot & 15)) << kShift) + in;
      kd[at] = kv[i];
      vd[at] = vv[i];
    }
  }
}

}  // namespace

cudaError_t launch_extend_tables(const ExtendParams& p, cudaStream_t s) {
  const size_t smem = 3 * sizeof(int32_t) * ((size_t)p.n_req + 1);
  constexpr size_t kMost = 3 * sizeof(int32_t) * (kMaxRequests + 1);
  static_assert(kMost + 2048 <= 227 * 1024, "the scans of the largest batch fit a CTA");
  if (smem > 40 * 1024) {  // more than any kernel may have unasked
    // The limit is the kernel's, for all threads of the process: always the
    // largest batch's, not this call's, which would fail another's launch.
    const cudaError_t e = cudaFuncSetAttribute(
        extend_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  // two calls with 256, 4096, 8192 and 65536 tokens: 7, 10, 13 and 63 us in one
  // CTA, 9, 10, 9 and 16 us in eight.  What is taken back is on the GPU alone, so a
  // call that only takes back is one CTA however many pages return: 256 pages 4 us,
  // 8192 9 to 20 (with the requests), 32768 32.
  const int ranks = p.max_new > 4 * kThreads ? 8 : 1;
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, extend_tables_kernel, p);
}

cudaError_t launch_append_slots(const AppendSlotsParams& p, cudaStream_t s) {
  if (p.n_tokens == 0) return cudaSuccess;
  const int parts = (p.hkv * (p.d / 8) + 127) / 128;
  const long long warps = (long long)p.n_tokens * parts;
  // The launch's own error: cudaGetLastError() would give one that another call left.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  return p.d == 128 ? cudaLaunchKernelEx(&cfg, append_slots_kernel<4>, p, parts)
                    : cudaLaunchKernelEx(&cfg, append_slots_kernel<3>, p, parts);
}

}  // namespace ta
