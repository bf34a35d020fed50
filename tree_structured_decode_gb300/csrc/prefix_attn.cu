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

constexpr int kRows = 16;       // query rows of a tile (the M of mma.m16n8k16)
constexpr int kWarps = 8;       // per CTA, each on its own
constexpr int kMinPages = 4;    // shortest run of a warp
constexpr float kLn2 = 0.69314718055994530942f;
constexpr long long kWaitLimitNs = 2000000000ll;

__device__ __forceinline__ int tiles_of(const Request& r, int gqa, int tile_rows = kRows) {
  return (r.n * gqa + tile_rows - 1) / tile_rows;
}

// Last i in [0, n) with key(i) <= x, 32 probes a step (key ascending, key(0) <= x).
template <class Key>
__device__ __forceinline__ int find_warp(int n, long long x, int lane, Key key) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, i < hi && key(i) <= x);
    lo += (__popc(below) - 1) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// ------------------------------------------------------------- schedule
// One block: checks lengths and offsets, sums up the line of own pages.
__global__ void __launch_bounds__(1024) prefix_schedule_kernel(const Args a) {
  const PrefixParams& p = a.p;
  __shared__ long long s_warp[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.n_req + 1023) / 1024;
  const int b0 = min(tid * per, p.n_req), b1 = min(b0 + per, p.n_req);
  int bad = 0;
  auto request = [&](int b) {
    Request r;
    int len = p.lens[b], first = b, last = b + 1;
    if (p.cu) first = p.cu[b], last = p.cu[b + 1];
    if (len < 0 || len > p.width * kPage || first < 0 || last < first || last > p.n_tokens)
      bad |= kBatchBadInput;
    r.len = min(max(len, 0), p.width * kPage);
    r.tok0 = min(max(first, 0), p.n_tokens);
    r.n = min(max(last, r.tok0), p.n_tokens) - r.tok0;
    r.np = (r.len + kPage - 1) / kPage;
    r.p0 = 0;
    return r;
  };
  auto work = [&](const Request& r) {
    return (long long)tiles_of(r, p.gqa) * r.np * p.hkv;
  };
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += work(request(b));
  long long v = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += o;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  long long at = v - mine + (warp > 0 ? s_warp[warp - 1] : 0);
  for (int b = b0; b < b1; ++b) {
    Request r = request(b);
    r.p0 = at;
    a.line[0].req[b] = r;
    at += work(r);
  }
  if (bad && p.status) atomicOr(p.status, bad);
  if (tid == 0) {
    const long long nw = (long long)p.num_sms * kWarps;
    const long long total = s_warp[31];
    a.line[0].sizes[0] = total;
    a.line[0].sizes[1] = max((total + nw - 1) / nw, (long long)kMinPages);
  }
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

// A page-head in shared memory: [64-column half][16 tokens][128 B], 128-byte swizzle.
__device__ __forceinline__ uint32_t page_at(uint32_t base, int row, int chunk) {
  return base + (chunk >> 3) * 2048 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int D>
struct Ring {
  static constexpr int kHead = kPage * D * 2;           // bytes of a page-head
  static constexpr int kStages = D == 128 ? 3 : 6;      // K and V of one page each
  static constexpr int kBytes = kWarps * kStages * 2 * kHead;
  static constexpr int kSmem = kBytes + kWarps * kStages * 8;
};

// Each warp streams its run of pages through its own ring of shared-memory
// stages (K and V of one page, by TMA) and never waits for another warp.
// S = Q K^T and O += P V on mma.m16n8k16 with 16 tokens a page; the kernel is
// bound by reading K and V once, where the query rows of a request are few.
template <int D, bool kHalf>
__global__ void __launch_bounds__(kWarps * 32, 1)
    prefix_line_kernel(const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const Args a, const int which) {
  using R = Ring<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const PrefixParams& p = a.p;
  const Line& L = a.line[which];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = ptx::smem_u32(smem_raw) + warp * R::kStages * 2 * R::kHead;
  const uint32_t bars = ptx::smem_u32(smem_raw) + R::kBytes + warp * R::kStages * 8;
  if (lane == 0) {
    for (int s = 0; s < R::kStages; ++s) ptx::mbar_init(bars + 8 * s, 1);
    ptx::fence_mbar_init();
  }
  __syncwarp();

  const long long total = L.steps(), run = L.length();
  const int w = warp * gridDim.x + blockIdx.x;
  const long long x0 = min((long long)w * run, total);
  const int count = (int)(min(x0 + run, total) - x0);
  if (count <= 0) return;

  // Coordinates of 32 positions of the run at a time, one a lane: position
  // x0 + 32 k + lane.  The next 32 are looked up while these are used.
  struct Where {
    int b, head, tile, pg, np, page;
  };
  auto look_up = [&](int base) {
    Where r{0, 0, 0, 0, 1, 0};
    const int i = base + lane;
    if (i < count) {
      const long long x = x0 + i;
      int lo = 0, hi = L.n_req;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (L.req[mid].p0 <= x)
          lo = mid;
        else
          hi = mid;
      }
      const Request q = L.request(lo);
      const long long in = x - q.p0;
      const long long seg = in / q.np;
      const int tiles = tiles_of(q, p.gqa);
      r.b = lo;
      r.head = (int)(seg / tiles);
      r.tile = (int)(seg % tiles);
      r.pg = (int)(in - seg * q.np);
      r.np = q.np;
      r.page = L.table[(long long)lo * L.table_stride + r.pg];
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

  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];
  int vis[2], len = 0, b = 0, head = 0, tile = 0, pg0 = 0, rows = 0, tok0 = 0;
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
      const Request r = L.request(b);
      len = r.len;
      tok0 = r.tok0;
      rows = min(kRows, r.n * p.gqa - tile * kRows);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = tile * kRows + g + 8 * e;
        const bool there = g + 8 * e < rows;
        const int j = row / p.gqa;
        vis[e] = !there ? 0 : L.causal ? max(r.len - r.n + j + 1, 0) : r.len;
        const uint16_t* src = p.q + (tok0 + j) * p.q_stride + (head * p.gqa + row % p.gqa) * D + 2 * t;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][e] = there ? *reinterpret_cast<const uint32_t*>(src + 16 * k) : 0u;
          qf[k][2 + e] = there ? *reinterpret_cast<const uint32_t*>(src + 16 * k + 8) : 0u;
        }
        m[e] = -INFINITY;
        l[e] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
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
        return;
      }
    }
    float sc[2][4] = {};
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      uint32_t kf[4];
      ldsm4(kf, page_at(kb, (lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)));
      mma16816<kHalf>(sc[0], qf[k], kf[0], kf[1]);
      mma16816<kHalf>(sc[1], qf[k], kf[2], kf[3]);
    }
    const int tk0 = pg * kPage;
    if (tk0 + kPage > vis[0] || tk0 + kPage > vis[1]) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tk0 + n * 8 + 2 * t + (e & 1) >= vis[e >> 1]) sc[n][e] = -INFINITY;
    }
    uint32_t pf[4];
    float alpha[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mx = fmaxf(fmaxf(sc[0][2 * e], sc[0][2 * e + 1]), fmaxf(sc[1][2 * e], sc[1][2 * e + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m[e], mx * p.scale_log2);
      const float off = m_new == -INFINITY ? 0.f : m_new;  // nothing seen yet
      alpha[e] = m[e] == m_new ? 1.f : ptx::ex2(m[e] - off);
      m[e] = m_new;
      float w4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w4[k] = ptx::ex2(fmaf(sc[k >> 1][2 * e + (k & 1)], p.scale_log2, -off));
      l[e] = fmaf(l[e], alpha[e], (w4[0] + w4[1]) + (w4[2] + w4[3]));
      pf[e] = pack2<kHalf>(w4[0], w4[1]);
      pf[2 + e] = pack2<kHalf>(w4[2], w4[3]);
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= alpha[0];
        o[n][1] *= alpha[0];
        o[n][2] *= alpha[1];
        o[n][3] *= alpha[1];
      }
    }
    // V rows past the request's end may hold anything: their weight is 0, but
    // 0 * NaN is not 0
    const int left = len - tk0;
    const uint32_t keep0 = (2 * t < left ? 0xffffu : 0u) | (2 * t + 1 < left ? 0xffff0000u : 0u);
    const uint32_t keep1 = (2 * t + 8 < left ? 0xffffu : 0u) | (2 * t + 9 < left ? 0xffff0000u : 0u);
#pragma unroll
    for (int n = 0; n < D / 8; n += 2) {
      uint32_t vf[4];
      ldsm4t(vf, page_at(vb, (lane & 7) + (((lane >> 3) & 1) << 3), n + (lane >> 4)));
      mma16816<kHalf>(o[n], pf, vf[0] & keep0, vf[1] & keep1);
      mma16816<kHalf>(o[n + 1], pf, vf[2] & keep0, vf[3] & keep1);
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
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      }
      const bool whole = pg0 == 0 && pg + 1 == np;
      const long long slot = (2ll * w + (pg0 == 0 ? 1 : 0)) * kRows;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = g + 8 * e;
        if (r < rows) {
          const int row = tile * kRows + r;
          const long long at_row =
              (long long)(tok0 + row / p.gqa) * p.hq + head * p.gqa + row % p.gqa;
          float* dst = whole ? L.row_o + at_row * D : L.piece_o + (slot + r) * D;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2*>(dst + 8 * n + 2 * t) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
          if (t == 0) (whole ? L.row_ml[at_row] : L.piece_ml[slot + r]) = make_float2(m[e], l[e]);
        }
      }
    }
  }
}

// ------------------------------------------------------------- merge
// A warp a row (token, q head): joins the pieces of both lines.
template <int D, bool kHalf>
__global__ void __launch_bounds__(256) prefix_merge_kernel(const Args a) {
  const PrefixParams& p = a.p;
  const int lane = threadIdx.x & 31;
  const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (row >= (long long)p.n_tokens * p.hq) return;
  constexpr int E = D / 32;
  const int tok = (int)(row / p.hq), h = (int)(row % p.hq);
  float M = -INFINITY, den = 0.f, acc[E] = {};
  auto fold = [&](const float* o, const float2 ml) {
    if (ml.x == -INFINITY) return;
    const float m_new = fmaxf(M, ml.x);
    const float a0 = ptx::ex2(M - m_new), a1 = ptx::ex2(ml.x - m_new);
    den = den * a0 + ml.y * a1;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * a0 + o[lane * E + e] * a1;
    M = m_new;
  };
  const int b = find_warp(p.n_req, tok, lane, [&](int i) { return (long long)a.line[0].req[i].tok0; });
  const Request own = a.line[0].req[b];
  const bool there = p.n_req > 0 && tok >= own.tok0 && tok < own.tok0 + own.n;
  if (there) {
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const Line& L = a.line[which];
      const Request r = which ? L.one : own;
      if (r.np == 0) continue;
      const int in = (tok - r.tok0) * p.gqa + h % p.gqa;
      const long long seg = (long long)(h / p.gqa) * tiles_of(r, p.gqa, L.tile_rows) + in / L.tile_rows;
      const long long first = r.p0 + seg * r.np, run = L.length();
      const long long w0 = first / run, w1 = (first + r.np - 1) / run;
      if (w0 == w1) {
        fold(L.row_o + row * D, L.row_ml[row]);
      } else {
        for (long long w = w0; w <= w1; ++w) {
          const long long at = (2 * w + (w == w0 ? 1 : 0)) * L.tile_rows + in % L.tile_rows;
          fold(L.piece_o + at * D, L.piece_ml[at]);
        }
      }
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<kHalf>(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && p.lse) p.lse[row] = den > 0.f ? (M + log2f(den)) * kLn2 : -INFINITY;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Query rows from which the prefix goes to the tensor-core tiles.
constexpr int kTileMinRows = 17;
bool by_tiles(const PrefixParams& p) { return (long long)p.n_tokens * p.gqa >= kTileMinRows; }

// Lays the workspace out; returns its size.
size_t lay_out(const PrefixParams& p, uint8_t* base, Args* a) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* q = base + at;
    at += up(bytes);
    return q;
  };
  const size_t rows = (size_t)p.n_tokens * p.hq;
  for (int i = 0; i < 2; ++i) {
    Line& L = a->line[i];
    L = Line{};
    L.n_req = i ? 1 : p.n_req;
    L.width = i ? 0 : p.width;
    L.causal = i ? 0 : 1;
    L.table = i ? p.prefix_pages : p.table;
    L.table_stride = i ? 0 : p.table_stride;
    L.tile_rows = kRows;
    if (i == 1) {
      if (p.prefix_len == 0) continue;
      const bool tiles = by_tiles(p);
      L.tile_rows = tiles ? kTileRows : kRows;
      const int step = tiles ? kTileTokens : kPage;
      L.one.len = p.prefix_len;
      L.one.n = p.n_tokens;
      L.one.np = (p.prefix_len + step - 1) / step;
      const long long blocks = ((long long)p.n_tokens * p.gqa + L.tile_rows - 1) / L.tile_rows;
      const long long runs = tiles ? p.num_sms : (long long)p.num_sms * kWarps;
      L.total = blocks * p.hkv * L.one.np;
      L.run = std::max((L.total + runs - 1) / runs, tiles ? 1ll : (long long)kMinPages);
    } else {
      L.req = reinterpret_cast<Request*>(take(sizeof(Request) * (size_t)(L.n_req + 1)));
      L.sizes = reinterpret_cast<long long*>(take(16));
    }
    const size_t pieces =
        2 * (size_t)p.num_sms * (L.tile_rows == kTileRows ? kTileRows : kWarps * kRows);
    L.piece_o = reinterpret_cast<float*>(take(pieces * p.d * 4));
    L.piece_ml = reinterpret_cast<float2*>(take(pieces * 8));
    L.row_o = reinterpret_cast<float*>(take(rows * p.d * 4));
    L.row_ml = reinterpret_cast<float2*>(take(rows * 8));
  }
  return at;
}

template <int D, bool kHalf>
cudaError_t run(const Args& a, cudaStream_t s) {
  const PrefixParams& p = a.p;
  cudaError_t e = cudaFuncSetAttribute(prefix_line_kernel<D, kHalf>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::kSmem);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  e = make_page_map(&mk, p.k_pages, D, p.hkv, p.num_pages, true);
  if (e != cudaSuccess) return e;
  e = make_page_map(&mv, p.v_pages, D, p.hkv, p.num_pages, true);
  if (e != cudaSuccess) return e;
  if (p.prefix_len > 0) {
    if (by_tiles(p)) {
      CUtensorMap half;  // one 64-column half of a page-head
      e = make_page_map(&half, p.k_pages, D, p.hkv, p.num_pages, false);
      if (e != cudaSuccess) return e;
      e = launch_prefix_tiles(a, half, mv, s);
      if (e != cudaSuccess) return e;
    } else {
      prefix_line_kernel<D, kHalf><<<p.num_sms, kWarps * 32, Ring<D>::kSmem, s>>>(mk, mv, a, 1);
    }
  }
  prefix_schedule_kernel<<<1, 1024, 0, s>>>(a);
  prefix_line_kernel<D, kHalf><<<p.num_sms, kWarps * 32, Ring<D>::kSmem, s>>>(mk, mv, a, 0);
  const long long rows = (long long)p.n_tokens * p.hq;
  prefix_merge_kernel<D, kHalf><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(a);
  return cudaGetLastError();
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
