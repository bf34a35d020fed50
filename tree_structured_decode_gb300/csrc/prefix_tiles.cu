// The shared prefix on the tensor cores (sm_103a): partial attention of all
// query rows of a kv head against the prefix's keys.
//
// A CTA (one per SM) holds two tiles of 128 query rows (rows are (token, head
// of the group): they share the kv head) and streams the prefix's K and V past
// both, 128 tokens a step, so each byte read from L2 serves 256 rows.  Per step
// and tile, on tcgen05 with the accumulators in TMEM:
//   S = Q K^T (128 x 128), online softmax on one row per thread, P as 16-bit
//   pairs over S (see kFp16Base), O += P V.
// The two tiles alternate: while one's softmax runs, the other's products do.
// A step's products are 4 * 256 * 128 * d operations, its exponentials 256 * 128:
// at d = 128 tensor cores and exponential units have about the same to do.  A step
// takes 1.66 us at d = 128 (1.54 PFLOP/s on 152 SMs); the products would take 1.05:
// what binds is the chain S, softmax, P V of a tile, which the other tile's only
// half covers.  (P handed over in two parts was slower, 434 against 371 us for 512
// queries of 64 heads behind 32768 tokens.)  A segment costs another 8 us for its
// queries, first S and output.
//
// Roles: warps 0-3 and 4-7 are the softmax of tile 0 and 1 (thread = row =
// TMEM lane), warp 8 streams K and V by TMA (and zeroes V's rows past the
// prefix), warp 9 issues the products.  Products run in the order of issue, so
// S of the next step may be issued right behind the P V that still reads P from
// the same columns.
//
// Steps of all (kv head, row block) segments stand in one line; a CTA takes a
// contiguous run of it.  What it has of a segment goes out as {m, l} and the
// unnormalised O in 32 bits.  This kernel starts while the line kernel runs on
// some of the SMs; CTAs that start behind it there have shorter runs.
//
// Every wait has a limit.  One that runs out sets the status word's timeout bit
// and the CTA's abort flag; every role then stops issuing, waits (with a limit)
// for its copies or products in flight, and the CTA frees its TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "prefix_attn.h"
#include "ptx.cuh"

namespace ta {
namespace {

constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 224, kIssueRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kIssueRegs <= kThreads * 168, "register split too large");
constexpr float kRescaleLog2 = 8.f;  // O is rescaled when a row's maximum grows by more than 2^8
constexpr long long kWaitLimitNs = 2000000000ll, kDrainLimitNs = 200000000ll;
constexpr uint32_t kTmemCols = 512;  // S of both tiles (128 columns each), O of both (128 each)
constexpr int kStepPages = kTileTokens / kPage;

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kQBytes = 128 * D * 2;               // one tile of queries
  static constexpr int kStageBytes = kTileTokens * D * 2;   // K or V of a step
  static constexpr int kStages = D == 128 ? 5 : 10;         // K and V take turns
  static constexpr int kHead = kPage * D * 2;               // a page-head
  static constexpr int kOffStage = 2 * kQBytes;
  static constexpr int kOffBar = kOffStage + kStages * kStageBytes;
  static constexpr int kBars = 3 * kStages + 11;
  static constexpr int kSmem = kOffBar + kBars * 8 + 8;  // TMEM address, abort flag
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

template <int D>
struct Cta {
  using C = Cfg<D>;
  uint32_t base;
  uint8_t* ptr;
  volatile int* abort_flag;
  int32_t* status;

  __device__ uint32_t bar(int i) const { return base + C::kOffBar + 8 * i; }
  __device__ uint32_t full(int s) const { return bar(s); }
  __device__ uint32_t empty(int s) const { return bar(C::kStages + s); }
  __device__ uint32_t land(int s) const { return bar(2 * C::kStages + s); }
  __device__ uint32_t q_full(int t) const { return bar(3 * C::kStages + t); }
  __device__ uint32_t s_full(int t) const { return bar(3 * C::kStages + 2 + t); }
  __device__ uint32_t p_full(int t) const { return bar(3 * C::kStages + 4 + t); }
  __device__ uint32_t o_full(int t) const { return bar(3 * C::kStages + 6 + t); }
  __device__ uint32_t o_empty(int t) const { return bar(3 * C::kStages + 8 + t); }
  __device__ uint32_t drain() const { return bar(3 * C::kStages + 10); }
  __device__ uint32_t stage(int s) const { return base + C::kOffStage + s * C::kStageBytes; }
};

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
// True once the phase is complete; false when the CTA has given up.  The same
// in all lanes of the warp.
template <int kRole, int D>
__device__ __forceinline__ bool wait(const Cta<D>& c, uint32_t bar, uint32_t parity) {
  bool ok = ptx::mbar_try_wait(bar, parity);
  if (!ok) ok = wait_slow<kRole>(bar, parity, c.abort_flag, c.status);
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity))
    if ((long long)(ptx::globaltimer() - t0) > kDrainLimitNs) return;
}

// The CTA's run, segment by segment: kv head, row block, steps [j0, j1) of n.
struct Segment {
  int head, block, j0, j1;
};
struct Walk {
  int head, block, j, left;  // the next step's place, steps left
  int n, blocks;             // steps of a segment, row blocks of a kv head
  __device__ __forceinline__ bool next(Segment& s) {
    if (left <= 0) return false;
    s.head = head;
    s.block = block;
    s.j0 = j;
    s.j1 = min(n, j + left);
    left -= s.j1 - s.j0;
    j = 0;
    if (++block == blocks) block = 0, ++head;
    return true;
  }
};
__device__ __forceinline__ Walk walk_of(const Cuts& cuts, const Runs& runs, int rows) {
  Walk w;
  w.n = cuts.one.np;
  w.blocks = (rows + kTileRows - 1) / kTileRows;
  const long long x = min(runs.start(blockIdx.x), cuts.total);
  w.left = (int)(min(runs.start(blockIdx.x + 1ll), cuts.total) - x);
  const long long u = quotient(x, max(w.n, 1));
  w.j = (int)(x - u * w.n);
  w.head = (int)quotient(u, max(w.blocks, 1));
  w.block = (int)(u - (long long)w.head * w.blocks);
  return w;
}

// ------------------------------------------------------------- copies
template <int D>
__device__ void stream_kv(const CUtensorMap* tmk, const CUtensorMap* tmv, const Args& a,
                          const Cta<D>& c, Walk walk) {
  using C = Cfg<D>;
  const PrefixParams& p = a.p;
  const int lane = threadIdx.x & 31;
  const int n_pages = (p.prefix_len + kPage - 1) / kPage;
  auto page_of = [&](int j) {  // lane i < 8: page i of step j
    const int i = j * kStepPages + lane;
    if (lane >= kStepPages || i >= n_pages) return 0;
    const int id = p.prefix_pages[i];
    if ((unsigned)id < (unsigned)p.num_pages) return id;
    if (p.status) atomicOr(p.status, kBatchBadSlot);
    return p.num_pages;  // outside the tensor map: read as zeros
  };
  Segment s;
  uint32_t g = 0;
  uint32_t zeroed = 0;  // phase of each stage's land barrier
  bool ok = true;
  while (ok && walk.next(s)) {
    int next = page_of(s.j0);
    for (int j = s.j0; ok && j < s.j1; ++j) {
      const int ids = next;
      if (j + 1 < s.j1) next = page_of(j + 1);
      const int nb = min(kStepPages, n_pages - j * kStepPages);
      const int last = p.prefix_len - (j * kStepPages + nb - 1) * kPage;  // tokens of the step's last page
#pragma unroll
      for (int v = 0; v < 2; ++v, ++g) {
        const int st = g % C::kStages;
        if (g >= (uint32_t)C::kStages && !wait<1>(c, c.empty(st), (g / C::kStages + 1) & 1)) {
          ok = false;
          break;
        }
        const bool zero = v == 1 && last < kPage;
        const uint32_t bar = zero ? c.land(st) : c.full(st);
        const uint32_t dst = c.stage(st);
        const bool leader = ptx::elect_one();
        if (leader) ptx::mbar_arrive_expect_tx(bar, nb * C::kHead);
        for (int b = 0; b < nb; ++b) {
          const int page = __shfl_sync(0xffffffffu, ids, b);
          if (leader) {
            if (v == 0) {  // K: [64-column half][128 tokens][128 B]
#pragma unroll
              for (int h = 0; h < C::kHalves; ++h)
                ptx::tma_load_4d(dst + h * (kTileTokens * 128) + b * 2048, tmk, 64 * h, 0, s.head, page, bar);
            } else if constexpr (D == 128) {  // V: [page][64-column half][16 tokens][128 B]
              ptx::tma_load_5d(dst + b * C::kHead, tmv, 0, 0, 0, s.head, page, bar);
            } else {
              ptx::tma_load_4d(dst + b * C::kHead, tmv, 0, 0, s.head, page, bar);
            }
          }
        }
        if (zero) {
          // slots past the prefix may hold anything: their weight is 0, but
          // 0 * NaN is not 0
          const uint32_t par = (zeroed >> st) & 1;
          zeroed ^= 1u << st;
          if (wait<1>(c, bar, par)) {
            uint8_t* head = c.ptr + C::kOffStage + st * C::kStageBytes + (nb - 1) * C::kHead;
            for (int i = lane; i < (kPage - last) * 8 * C::kHalves; i += 32) {
              const int r = last + i / (8 * C::kHalves), h = (i >> 3) % C::kHalves, ch = i & 7;
              *reinterpret_cast<uint4*>(head + h * 2048 + r * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
          } else {
            drain_wait(bar, par);
            ok = false;
          }
          __syncwarp();
          if (ptx::elect_one()) ptx::mbar_arrive(c.full(st));
        }
      }
    }
  }
  if (!ok)  // the copies in flight land before the CTA may end
    for (uint32_t k = g > (uint32_t)C::kStages ? g - C::kStages : 0; k < g; ++k)
      drain_wait(c.full(k % C::kStages), (k / C::kStages) & 1);
}

// ------------------------------------------------------------- products
template <int D, bool kHalf>
__device__ void issue_products(const Args& a, const Cta<D>& c, Walk walk, int rows,
                               uint32_t tmem) {
  using C = Cfg<D>;
  constexpr uint32_t kType = kHalf ? 0u : (1u << 7) | (1u << 10);
  constexpr uint32_t kDescQK =
      (ptx::idesc_bf16(128, kTileTokens, 0) & ~((1u << 7) | (1u << 10))) | kType;
  constexpr uint32_t kDescPV = (ptx::idesc_bf16(128, D, 1) & ~((1u << 7) | (1u << 10))) | kType;
  const int n_pages = (a.p.prefix_len + kPage - 1) / kPage;
  Segment s;
  uint32_t g = 0;             // steps before this segment: K is ring entry 2 g, V 2 g + 1
  uint32_t done[2] = {0, 0};  // steps of each tile before this segment
  uint32_t segs[2] = {0, 0};  // segments of each tile
  bool ok = true, issued = false;
  while (ok && walk.next(s)) {
    const int n = s.j1 - s.j0;
    const int tiles = s.block * kTileRows + 128 < rows ? 2 : 1;
    auto qk = [&](int t, int j) {  // S of tile t, step j
      const uint32_t k = 2 * (g + j);
      const uint64_t dk = ptx::sdesc_sw128(c.stage(k % C::kStages), 16, 1024);
      const uint64_t dq = ptx::sdesc_sw128(c.base + t * C::kQBytes, 16, 1024);
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
          ptx::mma_bf16(tmem + t * 128, dq + (off >> 4), dk + (off >> 4), kDescQK, kk > 0);
        }
        ptx::mma_commit(c.s_full(t));
        if (t == tiles - 1) ptx::mma_commit(c.empty(k % C::kStages));
      }
      issued = true;
    };
    auto wait_k = [&](int j) {
      const uint32_t k = 2 * (g + j);
      return wait<1>(c, c.full(k % C::kStages), (k / C::kStages) & 1);
    };
    ok = wait_k(0);
    for (int t = 0; ok && t < tiles; ++t) {
      ok = wait<1>(c, c.q_full(t), segs[t] & 1);
      if (!ok) break;
      ptx::fence_proxy_async_smem();  // the queries came by cp.async
      ptx::tc_fence_after();
      qk(t, 0);
    }
    for (int j = 0; ok && j < n; ++j) {
      const uint32_t v = 2 * (g + j) + 1;
      const int pages = min(kStepPages, n_pages - (s.j0 + j) * kStepPages);
      for (int t = 0; ok && t < tiles; ++t) {
        ok = wait<1>(c, c.p_full(t), (done[t] + j) & 1);
        if (ok && t == 0) ok = wait<1>(c, c.full(v % C::kStages), (v / C::kStages) & 1);
        // the first P V of a segment overwrites O: the last segment's must have been read
        if (ok && j == 0 && segs[t] > 0) ok = wait<1>(c, c.o_empty(t), (segs[t] - 1) & 1);
        if (!ok) break;
        ptx::tc_fence_after();
        if (ptx::elect_one()) {
          const uint64_t dv = ptx::sdesc_sw128(c.stage(v % C::kStages), 2048, 1024);
          for (int b = 0; b < pages; ++b)  // 16 tokens: 8 columns of P
            ptx::mma_bf16_ts(tmem + 256 + t * 128, tmem + t * 128 + b * 8, dv + b * (C::kHead >> 4),
                             kDescPV, j > 0 || b > 0);
          if (t == tiles - 1) ptx::mma_commit(c.empty(v % C::kStages));
          if (j == n - 1) ptx::mma_commit(c.o_full(t));
        }
        issued = true;
        if (j + 1 < n) {
          if (t == 0) ok = wait_k(j + 1);
          if (!ok) break;
          ptx::tc_fence_after();
          qk(t, j + 1);
        }
      }
    }
    g += n;
    for (int t = 0; t < tiles; ++t) done[t] += n, ++segs[t];
  }
  if (!ok && issued) {
    if (ptx::elect_one()) ptx::mma_commit(c.drain());
    __syncwarp();
    drain_wait(c.drain(), 0);
  }
}

// ------------------------------------------------------------- softmax
__device__ __forceinline__ uint32_t sw128(int row, int chunk) {
  return row * 128 + ((chunk ^ (row & 7)) << 4);
}

// Copies a tile's query rows (zeros past the last) into the swizzled buffer: a
// warp its own 32 rows, whole rows per instruction.
template <int D>
__device__ __forceinline__ void load_q(const uint16_t* src, bool there, uint32_t q, int tid) {
  constexpr int kChunks = D / 8, kPer = 32 / kChunks;
  const int lane = tid & 31, ch = lane % kChunks;
  const unsigned long long at = reinterpret_cast<unsigned long long>(src);
#pragma unroll
  for (int k = 0; k < 32 / kPer; ++k) {
    const int r = k * kPer + lane / kChunks;
    const unsigned long long s = __shfl_sync(0xffffffffu, at, r);
    const int h = __shfl_sync(0xffffffffu, (int)there, r);
    ptx::cp_async16(q + (ch >> 3) * (128 * 128) + sw128((tid & ~31) + r, ch & 7),
                    reinterpret_cast<const uint16_t*>(s) + ch * 8, h ? 16u : 0u);
  }
  ptx::cp_async_commit();
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

template <int D, bool kHalf>
__device__ void softmax_rows(const Args& a, const Cta<D>& c, Walk walk, int rows,
                             uint32_t tmem, int t) {
  using C = Cfg<D>;
  constexpr float kBase = kHalf ? kFp16Base : 0.f;  // m is that much below the largest score
  const PrefixParams& p = a.p;
  const Line& L = a.line[1];
  const int tid = threadIdx.x & 127, warp = tid >> 5;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t s_tmem = tmem + lanes + t * 128, o_tmem = tmem + lanes + 256 + t * 128;
  const uint32_t q_smem = c.base + t * C::kQBytes;
  // the walk's next segment that has rows in this tile
  auto next = [&](Segment& s) {
    while (walk.next(s))
      if (s.block * kTileRows + t * 128 < rows) return true;
    return false;
  };
  auto start = [&](const Segment& s) {
    const int row = s.block * kTileRows + t * 128 + tid;
    const bool there = row < rows;
    const int tok = there ? row / p.gqa : 0, h = there ? row % p.gqa : 0;
    load_q<D>(p.q + tok * p.q_stride + (s.head * p.gqa + h) * D, there, q_smem, tid);
    ptx::cp_async_mbar_arrive_noinc(c.q_full(t));
  };
  Segment s, s_next;
  bool more = next(s), ok = true;
  if (more) start(s);
  uint32_t done = 0, segs = 0;
  while (ok && more) {
    const int row = s.block * kTileRows + t * 128 + tid;
    const bool act = row - (tid & 31) < rows;  // this warp has rows
    const int n = s.j1 - s.j0;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      ok = wait<0>(c, c.s_full(t), (done + j) & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      if (act) {
        float v[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) ptx::tmem_ld32(s_tmem + k * 32, *reinterpret_cast<float(*)[32]>(v + k * 32));
        ptx::tmem_wait_ld();
        const int valid = p.prefix_len - (s.j0 + j) * kTileTokens;
        if (valid < kTileTokens) {
#pragma unroll
          for (int k = 0; k < 128; ++k) v[k] = k < valid ? v[k] : -INFINITY;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 2) m4[(k >> 1) & 3] = ptx::max3(m4[(k >> 1) & 3], v[k], v[k + 1]);
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2;
        float alpha = 1.f;
        if (mx > m + (kBase + kRescaleLog2) || j == 0) {
          alpha = j == 0 ? 1.f : ptx::ex2(m - (mx - kBase));
          m = mx - kBase;
        }
        l *= alpha;
        // the S that was waited for was issued behind the last P V: O holds it
        if (__any_sync(0xffffffffu, alpha != 1.f)) rescale_o<D>(o_tmem, alpha);
        const float nm = m == -INFINITY ? 0.f : -m;
        const uint64_t sc2 = ptx::f2(p.scale_log2, p.scale_log2), nm2 = ptx::f2(nm, nm);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            float x, y;
            ptx::f2_split(ptx::fma_f32x2(ptx::f2(v[half * 64 + k], v[half * 64 + k + 1]), sc2, nm2), x, y);
            x = ptx::ex2(x), y = ptx::ex2(y);
            pk[k >> 1] = pack2<kHalf>(x, y);
            acc[(k >> 1) & 3] = ptx::add_f32x2(acc[(k >> 1) & 3], ptx::f2(x, y));
          }
          ptx::tmem_st32u(s_tmem + half * 32, pk);
        }
        ptx::tmem_wait_st();
        float e[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) ptx::f2_split(acc[k], e[2 * k], e[2 * k + 1]);
        l += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(c.p_full(t));
    }
    if (!ok) break;
    // every S of this segment is done: the query buffer is free
    more = next(s_next);
    if (more) start(s_next);
    ok = wait<0>(c, c.o_full(t), segs & 1);
    if (!ok) break;
    ptx::tc_fence_after();
    if (act) {
      const bool whole = s.j0 == 0 && s.j1 == walk.n;
      const long long slot = (2ll * blockIdx.x + (s.j0 == 0 ? 1 : 0)) * kTileRows + t * 128 + tid;
      const long long at = (long long)(row / p.gqa) * p.hq + s.head * p.gqa + row % p.gqa;
      float* dst = whole ? L.row_o + at * D : L.piece_o + slot * D;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        float o[32];
        ptx::tmem_ld32(o_tmem + k * 32, o);
        ptx::tmem_wait_ld();
        if (row < rows) {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            ptx::st_global_v8(dst + k * 32 + e, __float_as_uint(o[e]), __float_as_uint(o[e + 1]),
                              __float_as_uint(o[e + 2]), __float_as_uint(o[e + 3]), __float_as_uint(o[e + 4]),
                              __float_as_uint(o[e + 5]), __float_as_uint(o[e + 6]), __float_as_uint(o[e + 7]));
        }
      }
      if (row < rows) (whole ? L.row_ml[at] : L.piece_ml[slot]) = make_float2(m, l);
    }
    ptx::tc_fence_before();
    ptx::mbar_arrive(c.o_empty(t));
    done += n;
    ++segs;
    s = s_next;
  }
  ptx::cp_async_wait_all();
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tile_kernel(const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const Args a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Cta<D> c;
  c.base = ptx::smem_u32(smem);
  c.ptr = smem;
  c.status = a.p.status;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kOffBar + C::kBars * 8);
  c.abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + C::kBars * 8 + 4);
  const int warp = threadIdx.x >> 5;
  __shared__ Walk s_walk;
  __shared__ int s_rows;
  if (c.base & 1023) {  // the swizzled layouts need it
    if (threadIdx.x == 0 && c.status) atomicOr(c.status, kBatchTimeout);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  // the merge may set itself up where there is room
  asm volatile("griddepcontrol.launch_dependents;");
  // pages in the own tokens' line, of which this kernel waits for no sum
  __shared__ long long s_sums[kThreads / 32];
  long long pages = 0, all_pages;
  int bad = 0;
  for (int b = threadIdx.x; b < a.p.n_req; b += kThreads) pages += steps_of(a, checked(a.p, b, bad));
  if (__syncthreads_or(bad & kBadOffsets)) pages = 0;
  scan_block(pages, s_sums, all_pages);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(c.full(s), 1);
      ptx::mbar_init(c.empty(s), 1);
      ptx::mbar_init(c.land(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(c.q_full(t), 128);
      ptx::mbar_init(c.s_full(t), 1);
      ptx::mbar_init(c.p_full(t), 128);
      ptx::mbar_init(c.o_full(t), 1);
      ptx::mbar_init(c.o_empty(t), 128);
    }
    ptx::mbar_init(c.drain(), 1);
    const Cuts cuts = prefix_cuts(a);
    s_rows = cuts.one.n * a.p.gqa;
    s_walk = walk_of(cuts, split_of(a, cuts, all_pages).runs, s_rows);
    *c.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(c.base + C::kOffBar + C::kBars * 8, kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Walk walk = s_walk;
  const int rows = s_rows;
  if (warp < 8) {
    ptx::setmaxnreg_inc<kSoftmaxRegs>();
    softmax_rows<D, kHalf>(a, c, walk, rows, tmem, warp >> 2);
  } else {
    ptx::setmaxnreg_dec<kIssueRegs>();
    if (warp == 8)
      stream_kv<D>(&tmk, &tmv, a, c, walk);
    else if (warp == 9)
      issue_products<D, kHalf>(a, c, walk, rows, tmem);
    else if (warp == 10) {
      // This kernel has ended only when the line kernel has: the merge waits for this one.
      asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, bool kHalf>
cudaError_t launch(const Args& a, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(prefix_tile_kernel<D, kHalf>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  // as many CTAs as there can be steps
  const PrefixParams& p = a.p;
  const long long blocks = ((long long)p.n_tokens * p.gqa + kTileRows - 1) / kTileRows;
  const long long steps = blocks * p.hkv * ((p.prefix_len + kTileTokens - 1) / kTileTokens);
  const unsigned grid = (unsigned)(steps < p.num_sms ? steps : p.num_sms);
  // a programmatic dependent of the line kernel, of which it reads nothing
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_tile_kernel<D, kHalf>, mk, mv, a);
}

}  // namespace

cudaError_t launch_prefix_tiles(const Args& a, const CUtensorMap& mk, const CUtensorMap& mv,
                                cudaStream_t s) {
  if (a.p.d == 128)
    return a.p.dtype == kFp16 ? launch<128, true>(a, mk, mv, s) : launch<128, false>(a, mk, mv, s);
  return a.p.dtype == kFp16 ? launch<64, true>(a, mk, mv, s) : launch<64, false>(a, mk, mv, s);
}

}  // namespace ta
