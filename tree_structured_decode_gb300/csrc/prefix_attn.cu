// Attention of a batch whose requests share a prefix (sm_103a).
//
// A query row (token, q head) sees the prefix's keys and its own request's.
// Both spans are computed apart, each with one pass and an online softmax, and
// joined: with m_i, l_i, O_i the running maximum, sum and accumulator of span
// i (or of a piece of it),
//   m = max m_i, out = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i,
//   lse = ln2 (m + log2 sum 2^(m_i - m) l_i).
//
// Lengths are device data, so the work is cut up on the device: the pages of
// all (request, kv head, row tile) segments stand in one line, and every warp
// takes an equal, contiguous run of it.  A segment that lies in several runs
// gives several pieces; a warp has at most one that began before its run and
// one that goes on after it, so pieces need two slots a warp, whatever the
// lengths are.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "batch.h"
#include "kernels.h"
#include "prefix_attn.h"
#include "ptx.cuh"

namespace ta {
namespace {

constexpr float kGrowLog2 = 8.f;  // the running maximum is raised when a score passes it by 2^8
constexpr float kLn2 = 0.69314718055994530942f;
constexpr long long kWaitLimitNs = 2000000000ll;

// (The line kernel's) All SMs without tensor-core tiles.
__device__ __forceinline__ Split split_for_line(const Args& a, long long total) {
  if (a.tiles) return split_of(a, prefix_cuts(a), total);
  return Split{a.p.num_sms, Runs{1, 0, 1}};
}

// Batches of more requests than a CTA of the line kernel has threads.
__global__ void __launch_bounds__(1024) prefix_schedule_kernel(const Args a) {
  __shared__ long long s_warp[32];
  const PrefixParams& p = a.p;
  asm volatile("griddepcontrol.launch_dependents;");
  const int per = (p.n_req + 1023) / 1024;
  const int b0 = min((int)threadIdx.x * per, p.n_req), b1 = min(b0 + per, p.n_req);
  int bad = 0;
  long long mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += steps_of(a, checked(p, b, bad));
  const bool broken = __syncthreads_or(bad & kBadOffsets);
  if (broken) mine = 0;
  const long long base = a.mixed ? prefix_cuts(a).total : 0;
  long long at = base + scan_block(mine, s_warp, total) - mine;
  for (int b = b0; b < b1; ++b) {
    Request r = checked(p, b, bad);
    if (broken) r.n = 0;
    r.p0 = at;
    at += steps_of(a, r);
    publish(a, b, r);
  }
  if (bad && p.status) atomicOr(p.status, bad & ~kBadOffsets);
  if (threadIdx.x == 0) publish_sizes(a, base + total, split_for_line(a, base + total));
}

// ------------------------------------------------------------- attention
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kHalf)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kHalf) return ptx::pack_f16(lo, hi);
  return ptx::pack_bf16(lo, hi);
}

// The transpose of an 8 x 8 matrix of 16-bit values held two a lane.
__device__ __forceinline__ uint32_t turn(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// A page-head in shared memory: [64-column half][16 tokens][128 B], 128-byte swizzle.
__device__ __forceinline__ uint32_t page_at(uint32_t base, int row, int chunk) {
  return base + (chunk >> 3) * 2048 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

constexpr int kMaxPlaces = 2048;  // requests whose places are searched in shared memory

// 12 warps an SM hide one another's latencies; each has two pages (four at d =
// 64) in flight or in use.
constexpr int kMaxSelf = kLineWarps * 32;  // requests that a CTA checks by itself, one a thread
template <int D>
struct Ring {
  static constexpr int kWarps = kLineWarps;
  static constexpr int kHead = kPage * D * 2;           // bytes of a page-head
  static constexpr int kStages = 2 * (128 / D);  // K and V of one page each
  static constexpr int kBytes = kWarps * kStages * 2 * kHead;
  // barriers, the scan's sums, the requests (or their places in the line)
  static constexpr int kSum = kBytes + kWarps * kStages * 8;
  static constexpr int kPlaces = kSum + kWarps * 8;
  static constexpr int kSmem = kPlaces + kMaxPlaces * 8;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(kMaxSelf * sizeof(Request) <= kMaxPlaces * 8, "the requests fit where places would");
};

// NT: tiles of 8 query rows.
// Each warp streams its run of pages through its own ring of shared-memory
// stages (K and V of one page, by TMA) and never waits for another warp.  Query
// rows are the N of mma.m16n8k16, a page's 16 tokens its M and then its K:
//   S^T = K Q^T (16 x 8 NT),  O^T += V^T P^T (d x 8 NT),
// with P^T turned by movmatrix, in the queries' type (see kFp16Base).  (Rows as M want 16 of them: twice the products
// and accumulators for the eight or fewer rows of one query.)  The running
// maximum grows only when a score passes it by 2^8, so most pages need no
// reduction across lanes.  Bound by reading K and V once: 64000 page-heads of 16
// x 128 (527 MB) in 103 us, 5.1 TB/s; while its SMs are busy 6.4 TB/s, but runs of
// equal length do not end together.  (The pages by cp.async instead of TMA: 6 %
// slower.  A CTA that joins its warps' pieces: three times as slow.)
// The line is the requests' own pages, with the prefix's before them where it
// has at most 16 query rows a kv head (b < 0 below).  Every CTA sums up the
// requests by itself, which costs less than a kernel before this one.
template <int D, bool kHalf, int NT>
__global__ void __launch_bounds__(Ring<D>::kWarps * 32, 1)
    prefix_line_kernel(const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const Args a) {
  using R = Ring<D>;
  constexpr float kBase = kHalf ? kFp16Base : 0.f;  // m is that much below the largest score
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const PrefixParams& p = a.p;
  const Line& L = a.line[0];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = ptx::smem_u32(smem_raw) + warp * R::kStages * 2 * R::kHead;
  const uint32_t bars = ptx::smem_u32(smem_raw) + R::kBytes + warp * R::kStages * 8;
  if (ptx::smem_u32(smem_raw) & 1023) {  // the swizzled pages need it
    if (threadIdx.x == 0 && p.status) atomicOr(p.status, kBatchTimeout);
    return;
  }
  if (lane == 0) {
    for (int s = 0; s < R::kStages; ++s) ptx::mbar_init(bars + 8 * s, 1);
    ptx::fence_mbar_init();
  }
  __syncwarp();
  // the next kernel may set itself up while this one runs
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the schedule, if there is one

  Request* requests = reinterpret_cast<Request*>(smem_raw + R::kPlaces);
  long long* places = reinterpret_cast<long long*>(smem_raw + R::kPlaces);
  const bool near = p.n_req <= kMaxPlaces;
  Cuts prefix{};
  if (a.mixed) prefix = prefix_cuts(a);
  const long long base = prefix.total;  // the prefix's pages in the line
  long long total, run;
  int ctas;  // that have a part of the line
  if (a.self) {
    const int b = threadIdx.x;
    int bad = 0;
    Request r{};
    if (b < p.n_req) r = checked(p, b, bad);
    if (__syncthreads_or(bad & kBadOffsets)) r.n = 0;
    const long long mine = b < p.n_req ? steps_of(a, r) : 0;
    r.p0 = base + scan_block(mine, reinterpret_cast<long long*>(smem_raw + R::kSum), total) - mine;
    total += base;
    const Split split = split_for_line(a, total);
    ctas = split.line_ctas;
    run = own_run(a, total, ctas);
    if (b < p.n_req) requests[b] = r;
    if (blockIdx.x == 0) {  // for the merge
      if (b < p.n_req) publish(a, b, r);
      if (bad && p.status) atomicOr(p.status, bad & ~kBadOffsets);
      if (b == 0) publish_sizes(a, total, split);
    }
    __syncthreads();
  } else {
    if (near) {
      for (int b = threadIdx.x; b < p.n_req; b += R::kWarps * 32) places[b] = __ldcg(&L.req[b].p0);
      __syncthreads();
    }
    total = __ldcg(L.sizes);
    run = __ldcg(L.sizes + 1);
    ctas = split_for_line(a, total).line_ctas;
  }
  auto request = [&](int b) {  // (past L1: see above)
    if (b < 0) return prefix.one;
    if (a.self) return requests[b];
    const long long* src = reinterpret_cast<const long long*>(L.req + b);
    Request r;
    const long long w[3] = {__ldcg(src), __ldcg(src + 1), __ldcg(src + 2)};
    memcpy(&r, w, sizeof r);
    return r;
  };
  if ((int)blockIdx.x >= ctas) return;
  const int w = warp * ctas + blockIdx.x;
  const long long x0 = min((long long)w * run, total);
  const int count = (int)(min(x0 + run, total) - x0);

  // Coordinates of 32 positions of the run at a time, one a lane: position
  // x0 + 32 k + lane.  The next 32 are looked up while these are used.
  struct Where {
    int b, head, tile, pg, np, page;
  };
  auto look_up = [&](int from) {
    Where r{0, 0, 0, 0, 1, 0};
    const int i = from + lane;
    if (i < count) {
      const long long x = x0 + i;
      int lo = 0, hi = p.n_req;
      if (x < base) lo = -1, hi = 0;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((a.self ? requests[mid].p0 : near ? places[mid] : __ldcg(&L.req[mid].p0)) <= x)
          lo = mid;
        else
          hi = mid;
      }
      const Request q = request(lo);
      const long long in = x - q.p0;
      const long long seg = quotient(in, q.np);
      const int tiles = tiles_of(q, p.gqa, L);
      r.b = lo;
      r.head = (int)quotient(seg, tiles);
      r.tile = (int)(seg - (long long)r.head * tiles);
      r.pg = (int)(in - seg * q.np);
      r.np = q.np;
      r.page = lo < 0 ? p.prefix_pages[r.pg] : p.table[(long long)lo * p.table_stride + r.pg];
      if ((unsigned)r.page >= (unsigned)p.num_pages) {
        r.page = p.num_pages;  // outside the tensor map: read as zeros
        if (p.status) atomicOr(p.status, kBatchBadSlot);
      }
    }
    return r;
  };
  Where cur = look_up(0), nxt = count > 32 ? look_up(32) : cur;
  auto copy = [&](int i, int page, int head) {
    const int s = i % R::kStages;
    if (lane == 0) {
      const uint32_t bar = bars + 8 * s, dst = ring + s * 2 * R::kHead;
      ptx::mbar_arrive_expect_tx(bar, 2 * R::kHead);
      if constexpr (D == 128) {
        ptx::tma_load_5d(dst, &tmk, 0, 0, 0, head, page, bar);
        ptx::tma_load_5d(dst + R::kHead, &tmv, 0, 0, 0, head, page, bar);
      } else {
        ptx::tma_load_4d(dst, &tmk, 0, 0, head, page, bar);
        ptx::tma_load_4d(dst + R::kHead, &tmv, 0, 0, head, page, bar);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < R::kStages; ++i) {
    const int page = __shfl_sync(0xffffffffu, cur.page, i), head = __shfl_sync(0xffffffffu, cur.head, i);
    if (i < count) copy(i, page, head);
  }

  uint32_t qf[D / 16][NT][2];
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2];  // rows 8 nt + 2 t + e
  int vis[NT][2], len = 0, b = 0, head = 0, tile = 0, pg0 = 0, rows = 0, tok0 = 0;
  for (int i = 0; i < count; ++i) {
    const int at = i & 31;
    if (i > 0 && at == 0) {
      cur = nxt;
      if (i + 32 < count) nxt = look_up(i + 32);
    }
    const int pg = __shfl_sync(0xffffffffu, cur.pg, at), np = __shfl_sync(0xffffffffu, cur.np, at);
    if (i == 0 || pg == 0) {  // a segment begins (or goes on from the warp before)
      b = __shfl_sync(0xffffffffu, cur.b, at);
      head = __shfl_sync(0xffffffffu, cur.head, at);
      tile = __shfl_sync(0xffffffffu, cur.tile, at);
      pg0 = pg;
      const Request r = request(b);
      len = r.len;
      tok0 = r.tok0;
      rows = min(8 * NT, r.n * p.gqa - tile * 8 * NT);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = tile * 8 * NT + 8 * n + g;
        const bool there = 8 * n + g < rows;
        const uint16_t* src =
            p.q + (tok0 + row / p.gqa) * p.q_stride + (head * p.gqa + row % p.gqa) * D + 2 * t;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][n][0] = there ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
          qf[k][n][1] = there ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r2 = 8 * n + 2 * t + e, j = (tile * 8 * NT + r2) / p.gqa;
          vis[n][e] = r2 >= rows ? 0 : b >= 0 ? max(r.len - r.n + j + 1, 0) : r.len;
          m[n][e] = -INFINITY;
          l[n][e] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][n][e] = 0.f;
      }
    }
    const int s = i % R::kStages;
    const uint32_t kb = ring + s * 2 * R::kHead, vb = kb + R::kHead;
    {
      const uint32_t bar = bars + 8 * s, par = (i / R::kStages) & 1;
      bool ok = ptx::mbar_try_wait(bar, par);
      if (!ok) {
        const uint64_t t0 = ptx::globaltimer();
        while (!(ok = ptx::mbar_try_wait(bar, par)))
          if ((long long)(ptx::globaltimer() - t0) > kWaitLimitNs) break;
      }
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0 && p.status) atomicOr(p.status, kBatchTimeout);
        // the other copies in flight land before the CTA may end
        const uint64_t t0 = ptx::globaltimer();
        for (int j = i; j < min(i + R::kStages, count); ++j)
          while (!ptx::mbar_try_wait(bars + 8 * (j % R::kStages), (j / R::kStages) & 1) &&
                 (long long)(ptx::globaltimer() - t0) < kWaitLimitNs) {
          }
        break;
      }
    }
    float sc[NT][4] = {};  // tokens g, g + 8; rows 2 t, 2 t + 1
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t kf[4];
      ldsm4(kf, page_at(kb, (lane & 7) + (((lane >> 3) & 1) << 3), 2 * k + (lane >> 4)));
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16816<kHalf>(sc[n], kf, qf[k][n][0], qf[k][n][1]);
    }
    const int tk0 = pg * kPage;
    bool grow = false;
    float mx[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (tk0 + kPage > vis[n][e]) {
          if (tk0 + g >= vis[n][e]) sc[n][e] = -INFINITY;
          if (tk0 + g + 8 >= vis[n][e]) sc[n][2 + e] = -INFINITY;
        }
        mx[n][e] = fmaxf(sc[n][e], sc[n][2 + e]) * p.scale_log2;
        grow |= mx[n][e] > m[n][e] + (kBase + kGrowLog2);
      }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = mx[n][e];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x - kBase, m[n][e]);
          alpha[e] = x == m[n][e] ? 1.f : ptx::ex2(m[n][e] - x);
          m[n][e] = x;
          l[n][e] *= alpha[e];
        }
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][n][e] *= alpha[e & 1];
      }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float off = m[n][e] == -INFINITY ? 0.f : m[n][e];  // nothing seen yet
        sc[n][e] = ptx::ex2(fmaf(sc[n][e], p.scale_log2, -off));
        sc[n][2 + e] = ptx::ex2(fmaf(sc[n][2 + e], p.scale_log2, -off));
        l[n][e] += sc[n][e] + sc[n][2 + e];
      }
      pf[n][0] = turn(pack2<kHalf>(sc[n][0], sc[n][1]));
      pf[n][1] = turn(pack2<kHalf>(sc[n][2], sc[n][3]));
    }
    const int left = len - tk0;
    if (left >= kPage) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t vf[4];
        ldsm4t(vf, page_at(vb, (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<kHalf>(o[k][n], vf, pf[n][0], pf[n][1]);
      }
    } else {
      // V rows past the request's end may hold anything: their weight is 0, but
      // 0 * NaN is not 0
      const uint32_t keep0 = (2 * t < left ? 0xffffu : 0u) | (2 * t + 1 < left ? 0xffff0000u : 0u);
      const uint32_t keep1 = (2 * t + 8 < left ? 0xffffu : 0u) | (2 * t + 9 < left ? 0xffff0000u : 0u);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t vf[4];
        ldsm4t(vf, page_at(vb, (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
        vf[0] &= keep0, vf[1] &= keep0, vf[2] &= keep1, vf[3] &= keep1;
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816<kHalf>(o[k][n], vf, pf[n][0], pf[n][1]);
      }
    }
    __syncwarp();  // the stage is read by every lane
    {
      const int j = i + R::kStages, in = j & 31;
      const bool from_next = (j >> 5) != (i >> 5);
      const int page = __shfl_sync(0xffffffffu, from_next ? nxt.page : cur.page, in);
      const int hd = __shfl_sync(0xffffffffu, from_next ? nxt.head : cur.head, in);
      if (j < count) copy(j, page, hd);
    }
    if (pg + 1 == np || i + 1 == count) {  // the segment, or this warp's part of it, ends
      const bool whole = pg0 == 0 && pg + 1 == np;
      const long long slot = (2ll * w + (pg0 == 0 ? 1 : 0)) * (8 * NT);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float den = l[n][e];
          den += __shfl_xor_sync(0xffffffffu, den, 4);
          den += __shfl_xor_sync(0xffffffffu, den, 8);
          den += __shfl_xor_sync(0xffffffffu, den, 16);
          const int r = 8 * n + 2 * t + e;
          if (r >= rows) continue;
          const int row = tile * 8 * NT + r;
          const long long at_row = (long long)(tok0 + row / p.gqa) * p.hq + head * p.gqa + row % p.gqa;
          if (whole && a.join) {  // there is no prefix: the row is done
            const float inv = den > 0.f ? 1.f / den : den == 0.f ? 0.f : den;
            uint16_t* dst = p.out + at_row * D + g;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t two = pack2<kHalf>(o[k][n][e] * inv, o[k][n][2 + e] * inv);
              dst[16 * k] = (uint16_t)two;
              dst[16 * k + 8] = (uint16_t)(two >> 16);
            }
            if (g == 0 && p.lse) p.lse[at_row] = den == 0.f ? -INFINITY : (m[n][e] + log2f(den)) * kLn2;
          } else {
            const Line& M = a.line[b < 0 ? 1 : 0];
            float* dst = (whole ? M.row_o + at_row * D : L.piece_o + (slot + r) * D) + g;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              dst[16 * k] = o[k][n][e];
              dst[16 * k + 8] = o[k][n][2 + e];
            }
            if (g == 0) (whole ? M.row_ml[at_row] : L.piece_ml[slot + r]) = make_float2(m[n][e], den);
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------- merge
// Folds up to 16 pieces' {m, l} (one a lane of half a warp) into a row's running
// maximum and sum; returns this lane's piece's factor, a0 what was there before's.
__device__ __forceinline__ float fold_ml(const float2 ml, float& M, float& den, float& a0) {
  float m_new = ml.x;
#pragma unroll
  for (int off = 8; off; off >>= 1) m_new = fmaxf(m_new, __shfl_xor_sync(0xffffffffu, m_new, off));
  m_new = fmaxf(M, m_new);
  const float base = m_new == -INFINITY ? 0.f : m_new;
  a0 = ptx::ex2(M - base);
  const float w = ptx::ex2(ml.x - base);
  float sum = w * ml.y;
#pragma unroll
  for (int off = 8; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  den = den * a0 + sum;
  M = m_new;
  return w;
}
// Adds the O rows of `all` pieces (lane i of half a warp holds piece i's address,
// 0 for none, and factor), four loads in flight.
template <int E>
__device__ __forceinline__ void fold_o(unsigned long long at, float w, int all, float (&acc)[E]) {
  const int lane = threadIdx.x & 31, in = lane & 15;
  for (int j = 0; j < all; j += 4) {
    float4 v[4][E / 4];
    float wj[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4* s = reinterpret_cast<const float4*>(__shfl_sync(0xffffffffu, at, (lane & 16) + min(j + i, 15)));
      wj[i] = __shfl_sync(0xffffffffu, w, (lane & 16) + min(j + i, 15));
      const bool mine = j + i < 16 && s != nullptr;
      if (!mine) wj[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E / 4; ++e) v[i][e] = mine ? __ldcg(s + 16 * e + in) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        acc[4 * e] = fmaf(v[i][e].x, wj[i], acc[4 * e]);
        acc[4 * e + 1] = fmaf(v[i][e].y, wj[i], acc[4 * e + 1]);
        acc[4 * e + 2] = fmaf(v[i][e].z, wj[i], acc[4 * e + 2]);
        acc[4 * e + 3] = fmaf(v[i][e].w, wj[i], acc[4 * e + 3]);
      }
  }
}
__device__ __forceinline__ float inverse(float den) {
  return den > 0.f ? 1.f / den : den == 0.f ? 0.f : den;  // a NaN stays one
}

// Joins a row's (token, q head) pieces of both lines, where the line kernel has
// not: half a warp a row, a block 16 rows of a kv head, whose pieces one warp
// looks up, a row a lane.  What bounds it is the chain of loads: request, then
// {m, l} and O of two pieces at once (four, with the registers for three blocks an
// SM instead of four, is as fast; four with four blocks 8 us slower at 32768 rows).
constexpr int kMergeRows = 16;
constexpr int kAtOnce = 2;  // pieces
template <int D, bool kHalf>
__global__ void __launch_bounds__(256, 4) prefix_merge_kernel(const Args a) {
  const PrefixParams& p = a.p;
  constexpr int E = D / 16;  // columns of a lane
  const int in = threadIdx.x & 15, half = threadIdx.x >> 4;
  const int rows = p.n_tokens * p.gqa;  // of a kv head
  const int chunks = (rows + kMergeRows - 1) / kMergeRows;
  const int kvh = blockIdx.x / chunks, first = (blockIdx.x - kvh * chunks) * kMergeRows;
  struct Place {
    long long w0, row;
    int n, in;
  };
  __shared__ Place s_own[kMergeRows], s_prefix[kMergeRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x < kMergeRows) {
    const int row = min(first + (int)threadIdx.x, rows - 1);
    const int tok = row / p.gqa, in_head = row - tok * p.gqa;
    const long long at_row = (long long)tok * p.hq + kvh * p.gqa + in_head;
    const Cuts cuts = prefix_cuts(a);
    int b = tok;
    if (p.cu) b = tok < cuts.one.n ? a.request_of[tok] : -1;
    Request own{};
    if ((unsigned)b < (unsigned)p.n_req) own = a.line[0].req[b];
    Pieces po{&a.line[0], 0, at_row, 0, 0}, pp{&a.line[1], 0, at_row, 0, 0};
    if (tok >= own.tok0 && tok < own.tok0 + own.n) {
      if (tok < cuts.one.n) pp = pieces_of(a.line[1], cuts.one, prefix_runs(a), p, tok, kvh, in_head);  // else cu is broken
      po = pieces_of(a.line[0], own, own_runs(a), p, tok, kvh, in_head);
    }
    s_own[threadIdx.x] = Place{po.w0, po.row, po.n, po.in};
    s_prefix[threadIdx.x] = Place{pp.w0, pp.row, pp.n, pp.in};
  }
  __syncthreads();
  if (first + half >= rows) return;
  const Place own = s_own[half], pre = s_prefix[half];
  const long long at_row = own.row;
  const Pieces po{&a.line[0], own.w0, at_row, own.n, own.in}, pp{&a.line[1], pre.w0, at_row, pre.n, pre.in};
  if (a.join && po.n == 1) return;  // done by the line kernel
  const int n = po.n + pp.n;
  float M = -INFINITY, den = 0.f, acc[E] = {};
  for (int k0 = 0; k0 < n; k0 += kAtOnce) {
    float2 ml[kAtOnce];
    float4 v[kAtOnce][E / 4];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int k = k0 + i;
      ml[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E / 4; ++e) v[i][e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < n) {
        const bool mine = k < po.n;
        ml[i] = mine ? po.ml(k) : pp.ml(k - po.n);
        const float4* src = reinterpret_cast<const float4*>(mine ? po.o(k, D) : pp.o(k - po.n, D));
#pragma unroll
        for (int e = 0; e < E / 4; ++e) v[i][e] = __ldcg(src + 16 * e + in);
      }
    }
    float m_new = M;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) m_new = fmaxf(m_new, ml[i].x);
    const float base = m_new == -INFINITY ? 0.f : m_new;
    const float a0 = ptx::ex2(M - base);
    M = m_new;
    den *= a0;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= a0;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float w = ptx::ex2(ml[i].x - base);
      den = fmaf(w, ml[i].y, den);
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        acc[4 * e] = fmaf(v[i][e].x, w, acc[4 * e]);
        acc[4 * e + 1] = fmaf(v[i][e].y, w, acc[4 * e + 1]);
        acc[4 * e + 2] = fmaf(v[i][e].z, w, acc[4 * e + 2]);
        acc[4 * e + 3] = fmaf(v[i][e].w, w, acc[4 * e + 3]);
      }
    }
  }
  const float inv = inverse(den);
#pragma unroll
  for (int e = 0; e < E / 4; ++e)
    *reinterpret_cast<uint2*>(p.out + at_row * D + 64 * e + 4 * in) =
        make_uint2(pack2<kHalf>(acc[4 * e] * inv, acc[4 * e + 1] * inv),
                   pack2<kHalf>(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv));
  if (in == 0 && p.lse) p.lse[at_row] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
}

// The same for few rows, which have many pieces: a block a row, its half-warps
// every 16th piece.
template <int D, bool kHalf>
__global__ void __launch_bounds__(256) prefix_merge_row_kernel(const Args a) {
  const PrefixParams& p = a.p;
  constexpr int E = D / 16;
  const int lane = threadIdx.x & 31, in = lane & 15, half = threadIdx.x >> 4;
  const long long row = blockIdx.x;
  const int tok = (int)((uint32_t)row / (uint32_t)p.hq), h = (int)((uint32_t)row % (uint32_t)p.hq);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Pieces po{}, pp{};
  const Cuts cuts = p.prefix_len > 0 || p.cu ? prefix_cuts(a) : Cuts{};
  int b = tok;
  if (p.cu) b = tok < cuts.one.n ? a.request_of[tok] : -1;
  Request own{};
  if ((unsigned)b < (unsigned)p.n_req) own = a.line[0].req[b];
  if (tok >= own.tok0 && tok < own.tok0 + own.n) {
    const int kvh = h / p.gqa;
    if (p.prefix_len > 0 && tok < cuts.one.n)
      pp = pieces_of(a.line[1], cuts.one, prefix_runs(a), p, tok, kvh, h - kvh * p.gqa);
    po = pieces_of(a.line[0], own, own_runs(a), p, tok, kvh, h - kvh * p.gqa);
  }
  const int n = po.n + pp.n;
  if (a.join && po.n == 1) return;  // done by the line kernel (the whole block)
  float M = -INFINITY, den = 0.f, acc[E] = {};
  for (int k0 = 0; k0 < n; k0 += 256) {
    // this half-warp's pieces are k0 + half + 16 i; lane i reads its {m, l}
    const int k = k0 + half + 16 * in;
    float2 x = make_float2(-INFINITY, 0.f);
    unsigned long long at = 0;
    if (k < n) {
      x = k < po.n ? po.ml(k) : pp.ml(k - po.n);
      at = reinterpret_cast<unsigned long long>(k < po.n ? po.o(k, D) : pp.o(k - po.n, D));
    }
    float a0;
    const float w = fold_ml(x, M, den, a0);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= a0;
    fold_o<E>(at, w, min(16, (n - k0 + 15) / 16), acc);
  }
  __shared__ float2 s_ml[16];
  __shared__ float s_o[16][D];
  if (in == 0) s_ml[half] = make_float2(M, den);
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[half][64 * (e / 4) + 4 * in + e % 4] = acc[e];
  __syncthreads();
  if (threadIdx.x >= 32) return;
  M = -INFINITY;
  for (int k = 0; k < 16; ++k) M = fmaxf(M, s_ml[k].x);
  const float base = M == -INFINITY ? 0.f : M;
  den = 0.f;
  float o[D / 32] = {};
  for (int k = 0; k < 16; ++k) {
    const float w = ptx::ex2(s_ml[k].x - base);
    den += w * s_ml[k].y;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) o[e] = fmaf(w, s_o[k][lane * (D / 32) + e], o[e]);
  }
  const float inv = inverse(den);
#pragma unroll
  for (int e = 0; e < D / 32; e += 2)
    *reinterpret_cast<uint32_t*>(p.out + row * D + lane * (D / 32) + e) = pack2<kHalf>(o[e] * inv, o[e + 1] * inv);
  if (lane == 0 && p.lse) p.lse[row] = den == 0.f ? -INFINITY : (M + log2f(den)) * kLn2;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Query rows (of a kv head) from which the prefix goes to the tensor-core tiles.
// The line's tiles have up to 16, and read the prefix once each: 24 rows behind
// 4000 tokens take 19 us by tensor-core tiles, 52 by the line; 16 rows 19 and 16
// (64 rows behind 200 tokens 15 and 20, 16 rows 13 and 14).
constexpr int kTileMinRows = 17;
bool by_tiles(const PrefixParams& p) { return (long long)p.n_tokens * p.gqa >= kTileMinRows; }

// Rows an SM up to which the merge takes a block a row: 512 rows with prefixes
// of 8000 24 us (half a warp a row: 47), 1216 rows 33 (32), of 500 26 (22).
constexpr int kBlockRows = 4;

// Lays the workspace out; returns its size.
size_t lay_out(const PrefixParams& p, uint8_t* base, Args* a) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = base + at;
    at += up(bytes);
    return q;
  };
  const size_t rows = (size_t)p.n_tokens * p.hq;
  a->tiles = p.prefix_len > 0 && by_tiles(p);
  a->mixed = p.prefix_len > 0 && !a->tiles;
  a->self = p.n_req <= kMaxSelf;
  // (Joining a segment with the prefix's pieces as well, in the line kernel's
  // epilogue, was slower: its warps wait for those loads, 105 to 168 us at 512
  // requests of 64 heads, against 9 us less in the merge.)
  a->join = p.prefix_len == 0;
  a->request_of = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * (size_t)p.n_tokens));
  auto rows_of = [&](Line& L) {
    L.row_o = reinterpret_cast<float*>(take(rows * p.d * 4));
    L.row_ml = reinterpret_cast<float2*>(take(rows * 8));
  };
  auto pieces_of_runs = [&](Line& L) {
    for (L.tile_shift = 0; (1 << L.tile_shift) < L.tile_rows;) ++L.tile_shift;
    const size_t pieces = 2 * (size_t)L.runs * L.tile_rows;
    L.piece_o = reinterpret_cast<float*>(take(pieces * p.d * 4));
    L.piece_ml = reinterpret_cast<float2*>(take(pieces * 8));
  };
  Line& own = a->line[0];
  Line& pre = a->line[1];
  own = Line{};
  // query rows of a tile: 8, or 16 where a request has more on average (the
  // prefix by lines has at most 16).  32 were slower, with the registers they
  // take: 62 us against 37 at 128 requests of up to four drafts, 16 rows each.
  const long long queries = a->mixed || p.n_req == 0 ? p.n_tokens : (p.n_tokens + p.n_req - 1) / p.n_req;
  own.tile_rows = queries * p.gqa <= 8 ? 8 : 16;
  own.step = kPage;
  own.runs = p.num_sms * kLineWarps;
  own.req = reinterpret_cast<Request*>(take(sizeof(Request) * (size_t)(p.n_req + 1)));
  own.sizes = reinterpret_cast<long long*>(take(5 * sizeof(long long)));
  pieces_of_runs(own);
  rows_of(own);
  pre = own;  // mixed: the same line, pieces and all
  if (a->tiles) {
    pre.tile_rows = kTileRows;
    pre.step = kTileTokens;
    pre.runs = p.num_sms;
    pieces_of_runs(pre);
  }
  if (p.prefix_len > 0) rows_of(pre);
  return at;
}

template <int D, bool kHalf, int NT>
cudaError_t launch_line(const Args& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  using R = Ring<D>;
  cudaError_t e = cudaFuncSetAttribute(prefix_line_kernel<D, kHalf, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.p.num_sms);
  cfg.blockDim = dim3(R::kWarps * 32);
  cfg.dynamicSmemBytes = R::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = a.self ? 0 : 1;  // (the schedule comes before it)
  return cudaLaunchKernelEx(&cfg, prefix_line_kernel<D, kHalf, NT>, mk, mv, a);
}

template <int D, bool kHalf>
cudaError_t run(const Args& a, cudaStream_t s) {
  const PrefixParams& p = a.p;
  CUtensorMap mk, mv;
  cudaError_t e = make_page_map(&mk, p.k_pages, D, p.hkv, p.num_pages, true);
  if (e != cudaSuccess) return e;
  e = make_page_map(&mv, p.v_pages, D, p.hkv, p.num_pages, true);
  if (e != cudaSuccess) return e;
  if (!a.self) {
    cudaLaunchConfig_t one = {};  // (not by cudaGetLastError(), which gives what another call left)
    one.gridDim = dim3(1);
    one.blockDim = dim3(1024);
    one.stream = s;
    e = cudaLaunchKernelEx(&one, prefix_schedule_kernel, a);
    if (e != cudaSuccess) return e;
  }
  e = a.line[0].tile_rows == 8 ? launch_line<D, kHalf, 1>(a, mk, mv, s) : launch_line<D, kHalf, 2>(a, mk, mv, s);
  if (e != cudaSuccess) return e;
  if (a.tiles) {
    CUtensorMap half;  // one 64-column half of a page-head
    e = make_page_map(&half, p.k_pages, D, p.hkv, p.num_pages, false);
    if (e != cudaSuccess) return e;
    e = launch_prefix_tiles(a, half, mv, s);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const long long rows = (long long)p.n_tokens * p.hq;
  const bool block = rows <= (long long)kBlockRows * p.num_sms;
  const long long chunks = ((long long)p.n_tokens * p.gqa + kMergeRows - 1) / kMergeRows;
  cfg.gridDim = dim3((unsigned)(block ? rows : chunks * p.hkv));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return block ? cudaLaunchKernelEx(&cfg, prefix_merge_row_kernel<D, kHalf>, a)
               : cudaLaunchKernelEx(&cfg, prefix_merge_kernel<D, kHalf>, a);
}

}  // namespace

size_t prefix_workspace(const PrefixParams& p) {
  Args a{};
  return p.n_tokens ? lay_out(p, nullptr, &a) : 0;
}

cudaError_t launch_prefix_attention(const PrefixParams& p, void* workspace, cudaStream_t s) {
  if (p.n_tokens == 0) return cudaSuccess;
  Args a{};
  a.p = p;
  lay_out(p, static_cast<uint8_t*>(workspace), &a);
  if (p.d == 128) return p.dtype == kFp16 ? run<128, true>(a, s) : run<128, false>(a, s);
  return p.dtype == kFp16 ? run<64, true>(a, s) : run<64, false>(a, s);
}

}  // namespace ta
