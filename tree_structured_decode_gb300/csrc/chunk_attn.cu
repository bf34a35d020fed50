// Attention of several new tokens of each request over its pages, prompts and
// trees of drafts alike, on tcgen05 (sm_103a).
//
// Query rows are (token, q head of a kv head's group); a block of a request's
// new tokens gives up to 256 rows that share a kv head's keys.  A CTA (one per SM)
// streams K and V past them, 128 keys a step, with the products' accumulators in
// TMEM:
//   S = Q K^T (128 x 128), online softmax on one row per thread, P as 16-bit
//   pairs over S, O += P V.
// Two tiles alternate: while one's softmax runs, the other's products do.  With
// more than 128 rows the tiles are the block's two halves and share each step's
// keys (a prompt: bound by the products and the softmax between them).  With fewer
// they are the same rows and take the steps in turn (drafts: bound by reading K
// and V once); their sums are joined where the segment ends.
//
// Steps of all (request, kv head, block) segments stand in one line, and a CTA
// takes an equal, contiguous run of it, whatever the lengths are.  A segment
// within one run is final; pieces of one that lies in several go out as {m, l} and
// the unnormalised O in 32 bits and are joined by the merge,
//   m = max m_i, out = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i.
// A CTA has at most one piece that began before its run and one that goes on
// behind it.
//
// Which keys a row sees is a mask of 128 bits a step, made only in steps that hold
// a key that some row does not see: from the row's end for a prompt, and for a
// tree from the nodes above the row's, which its thread collects along parents.
//
// Roles: warps 0-3 and 4-7 are the softmax of tile 0 and 1 (thread = row = TMEM
// lane), warp 8 streams K and V by TMA (and zeroes V's rows past a request's end),
// warp 9 issues the products, warps 10 and 11 fill rows that see nothing.
// Products run in the order of issue, so S of a tile's next step may be issued
// right behind the P V that still reads P from the same columns.
//
// Every wait has a limit.  One that runs out sets the status word's timeout bit
// and the CTA's abort flag; every role then stops issuing, waits (with a limit)
// for its copies or products in flight, and the CTA frees its TMEM and returns.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "drafts.h"
#include "kernels.h"
#include "prefix_attn.h"
#include "ptx.cuh"
#include "tiles.cuh"

namespace ta {
namespace {

using tiles::drain_wait;
using tiles::load_q;
using tiles::pack2;
using tiles::rescale_o;
using tiles::wait;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 224, kIssueRegs = 56;
static_assert(256 * kSoftmaxRegs + 128 * kIssueRegs <= kThreads * 168, "register split too large");
constexpr float kRescaleLog2 = 8.f;  // O is rescaled when a row's maximum grows by more than 2^8
constexpr uint32_t kTmemCols = 512;  // S of both tiles (128 columns each), O of both (128 each)
constexpr int kBlockRows = 256;      // query rows of a segment, at most
constexpr int kStepPages = kTileTokens / kPage;

struct Cut {  // a segment that lies in several runs, told by the run where it ends
  int pieces, first, tok, rows, head, pad[3];
};

struct ChunkArgs {
  ChunkParams p;
  Cut* cuts;         // [grid]
  float2* piece_ml;  // [2 * grid][piece_rows]: {m, l}
  float* piece_o;    // [2 * grid][piece_rows][d]
  int piece_rows, block_tokens, grid;
};

// A request's lengths, checked: its tokens lie in the batch, its pages in the
// table.  (kBadOffsets: see prefix_attn.h.)
struct Chunk {
  int len, n, tok0;
};
struct Raw {
  int len, first, last;
};
__device__ __forceinline__ Raw raw_of(const ChunkParams& p, int b) {
  Raw r{p.lens[b], b, b + 1};
  if (p.cu) r.first = p.cu[b], r.last = p.cu[b + 1];
  return r;
}
__device__ __forceinline__ Chunk checked(const ChunkParams& p, const Raw& raw, int& bad) {
  Chunk r;
  if (raw.len < 0 || raw.len > p.width * kPage) bad |= kBatchBadInput;
  if (raw.first < 0 || raw.last < raw.first || raw.last > p.n_tokens) bad |= kBatchBadInput | kBadOffsets;
  r.len = min(max(raw.len, 0), p.width * kPage);
  r.tok0 = min(max(raw.first, 0), p.n_tokens);
  r.n = min(max(raw.last, r.tok0), p.n_tokens) - r.tok0;
  if (p.parents && r.n > kMaxNodes) bad |= kBatchBadInput, r.n = 0;
  return r;
}

// sum over i < n of floor((a i + b) / m): whole multiples of m out of a and b,
// then the same lattice points counted along the other axis, as in Euclid's
// algorithm.
__device__ __forceinline__ long long floor_sum(long long n, long long m, long long a, long long b) {
  long long sum = 0;
  while (n > 0) {
    const long long qa = quotient(a, m), qb = quotient(b, m);
    sum += n * (n - 1) / 2 * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const long long y = a * n + b;
    if (y < m) break;
    n = quotient(y, m);
    b = y - n * m;
    const long long t = m;
    m = a;
    a = t;
  }
  return sum;
}

// Blocks of a request's new tokens; block k's keys end with its last token's own.
__device__ __forceinline__ int blocks_of(const ChunkArgs& a, const Chunk& r) {
  return (r.n + a.block_tokens - 1) / a.block_tokens;
}
__device__ __forceinline__ int end_of(const ChunkArgs& a, const Chunk& r, int k) {
  return max(r.len - r.n + min((k + 1) * a.block_tokens, r.n), 0);
}
__device__ __forceinline__ int steps_of_block(const ChunkArgs& a, const Chunk& r, int k) {
  return (end_of(a, r, k) + kTileTokens - 1) / kTileTokens;
}
// Steps of the first k blocks, one kv head.
__device__ __forceinline__ long long steps_before(const ChunkArgs& a, const Chunk& r, int k) {
  const int blocks = blocks_of(a, r), base = r.len - r.n, t = a.block_tokens;
  long long sum = 0;
  if (k == blocks && k > 0) sum = (r.len + kTileTokens - 1) / kTileTokens, --k;
  const int k0 = base < 0 ? min(-base / t, k) : 0;  // blocks that see nothing
  return sum + floor_sum(k - k0, kTileTokens, t, base + (long long)(k0 + 1) * t + kTileTokens - 1);
}
__device__ __forceinline__ long long steps_of_request(const ChunkArgs& a, const Chunk& r) {
  if (r.n <= a.block_tokens) return r.n ? (long long)a.p.hkv * ((r.len + kTileTokens - 1) / kTileTokens) : 0;
  return a.p.hkv * steps_before(a, r, blocks_of(a, r));
}

struct Segment {
  int b, head;
  int tok, first, rows;  // the block's first token, its number among the request's new ones, query rows
  int len, base, end;    // tokens of the request, those before its new ones, keys of the block
  int np, j0, j1;        // steps in all, this run's
  int buf;               // (one tile's rows) which query buffer
  __device__ __forceinline__ bool pair() const { return rows > 128; }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == np; }
};

// The CTA's run, segment by segment.
struct Walk {
  int b, head, block, j, left;  // the next step's place, steps left
  Chunk r;
  Raw ahead;                    // the next request's
  int buf;                      // of the last segment: -1 after two tiles' rows

  __device__ __forceinline__ void look_ahead(const ChunkParams& p) {
    if (b + 1 < p.n_req) ahead = raw_of(p, b + 1);
  }
  __device__ __forceinline__ bool next(const ChunkArgs& a, Segment& s) {
    if (left <= 0) return false;
    const int t = a.block_tokens, count = min(r.n - block * t, t);
    s.b = b;
    s.head = head;
    s.first = block * t;
    s.tok = r.tok0 + s.first;
    s.rows = count * a.p.gqa;
    s.len = r.len;
    s.base = r.len - r.n;
    s.end = end_of(a, r, block);
    s.np = (s.end + kTileTokens - 1) / kTileTokens;
    s.j0 = j;
    s.j1 = min(s.np, j + left);
    left -= s.j1 - s.j0;
    buf = s.pair() ? -1 : buf < 0 ? 0 : buf ^ 1;
    s.buf = buf;
    j = 0;
    if (left > 0 && (++block) * t >= r.n) {
      if (++head == a.p.hkv) {
        head = 0;
        int bad = 0;
        do {  // the steps left are some request's
          ++b;
          r = checked(a.p, ahead, bad);
          look_ahead(a.p);
        } while ((r.n == 0 || r.len == 0) && b + 1 < a.p.n_req);
      }
      block = r.len < r.n ? (r.n - r.len) / t : 0;  // blocks before it see nothing
    }
    return true;
  }
};

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kQBytes = 128 * D * 2;               // one tile of queries
  static constexpr int kStageBytes = kTileTokens * D * 2;   // K or V of a step
  static constexpr int kStages = D == 128 ? 5 : 10;         // K and V take turns
  static constexpr int kHead = kPage * D * 2;               // a page-head
  static constexpr int kOffStage = 2 * kQBytes;
  static constexpr int kOffMl = kOffStage + kStages * kStageBytes;  // {m, l} of both tiles' rows
  static constexpr int kOffBar = kOffMl + 2 * 128 * 8;
  static constexpr int kBars = 3 * kStages + 12;
  static constexpr int kOffWalk = kOffBar + kBars * 8 + 8;  // behind the TMEM address and the abort flag
  static constexpr int kSmem = kOffWalk + sizeof(Walk);
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
  __device__ uint32_t joined() const { return bar(3 * C::kStages + 10); }
  __device__ uint32_t drain() const { return bar(3 * C::kStages + 11); }
  __device__ uint32_t stage(int s) const { return base + C::kOffStage + s * C::kStageBytes; }
  __device__ float2* ml() const { return reinterpret_cast<float2*>(ptr + C::kOffMl); }
};

// ------------------------------------------------------------- copies
template <int D>
__device__ void stream_kv(const CUtensorMap* tmk, const CUtensorMap* tmv, const ChunkArgs& a,
                          const Cta<D>& c, Walk walk) {
  using C = Cfg<D>;
  const ChunkParams& p = a.p;
  const int lane = threadIdx.x & 31;
  auto page_of = [&](const Segment& s, int j) {  // lane i < 8: page i of step j
    const int i = j * kStepPages + lane;
    if (lane >= kStepPages || i * kPage >= s.end) return 0;
    const int id = p.table[s.b * p.table_stride + i];
    if ((unsigned)id < (unsigned)p.num_pages) return id;
    if (p.status) atomicOr(p.status, kBatchBadSlot);
    return p.num_pages;  // outside the tensor map: read as zeros
  };
  Segment s, s_next;
  uint32_t g = 0;
  uint32_t zeroed = 0;  // phase of each stage's land barrier
  bool ok = true, more = walk.next(a, s);
  int next = more ? page_of(s, s.j0) : 0;
  while (ok && more) {
    more = walk.next(a, s_next);
    const int n_pages = (s.end + kPage - 1) / kPage;
    for (int j = s.j0; ok && j < s.j1; ++j) {
      const int ids = next;
      if (j + 1 < s.j1)
        next = page_of(s, j + 1);
      else if (more)
        next = page_of(s_next, s_next.j0);
      const int nb = min(kStepPages, n_pages - j * kStepPages);
      const int last = s.len - (j * kStepPages + nb - 1) * kPage;  // the request's tokens in the step's last page
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
          // slots past the request's end may hold anything: their weight is 0, but
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
    s = s_next;
  }
  if (!ok)  // the copies in flight land before the CTA may end
    for (uint32_t k = g > (uint32_t)C::kStages ? g - C::kStages : 0; k < g; ++k)
      drain_wait(c.full(k % C::kStages), (k / C::kStages) & 1);
}

// ------------------------------------------------------------- products
template <int D, bool kHalf>
__device__ void issue_products(const ChunkArgs& a, const Cta<D>& c, Walk walk, uint32_t tmem) {
  using C = Cfg<D>;
  constexpr uint32_t kType = kHalf ? 0u : (1u << 7) | (1u << 10);
  constexpr uint32_t kDescQK =
      (ptx::idesc_bf16(128, kTileTokens, 0) & ~((1u << 7) | (1u << 10))) | kType;
  constexpr uint32_t kDescPV = (ptx::idesc_bf16(128, D, 1) & ~((1u << 7) | (1u << 10))) | kType;
  Segment s;
  uint32_t g = 0;              // steps before this segment: K is ring entry 2 g, V 2 g + 1
  uint32_t done[2] = {0, 0};   // steps of each tile before this segment
  uint32_t loads[2] = {0, 0};  // of each query buffer
  uint32_t segs = 0;
  bool ok = true, issued = false;
  while (ok && walk.next(a, s)) {
    const int n = s.j1 - s.j0;
    const bool pair = s.pair();
    const int n_pages = (s.end + kPage - 1) / kPage;
    auto qk = [&](int t, int j, bool last_use) {  // S of tile t, step j
      const uint32_t k = 2 * (g + j);
      const uint64_t dk = ptx::sdesc_sw128(c.stage(k % C::kStages), 16, 1024);
      const uint64_t dq = ptx::sdesc_sw128(c.base + (pair ? t : s.buf) * C::kQBytes, 16, 1024);
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
          ptx::mma_bf16(tmem + t * 128, dq + (off >> 4), dk + (off >> 4), kDescQK, kk > 0);
        }
        ptx::mma_commit(c.s_full(t));
        if (last_use) ptx::mma_commit(c.empty(k % C::kStages));
      }
      issued = true;
    };
    auto pv = [&](int t, int j, bool first, bool last_use) {  // O of tile t, step j
      const uint32_t v = 2 * (g + j) + 1;
      const int pages = min(kStepPages, n_pages - (s.j0 + j) * kStepPages);
      if (ptx::elect_one()) {
        const uint64_t dv = ptx::sdesc_sw128(c.stage(v % C::kStages), 2048, 1024);
        for (int b = 0; b < pages; ++b)  // 16 tokens: 8 columns of P
          ptx::mma_bf16_ts(tmem + 256 + t * 128, tmem + t * 128 + b * 8, dv + b * (C::kHead >> 4),
                           kDescPV, !first || b > 0);
        if (last_use) ptx::mma_commit(c.empty(v % C::kStages));
        if (j == n - 1) {
          if (pair) {
            ptx::mma_commit(c.o_full(t));
          } else {
            ptx::mma_commit(c.o_full(0));
            ptx::mma_commit(c.o_full(1));
          }
        }
      }
      issued = true;
    };
    auto wait_k = [&](int j) {
      const uint32_t k = 2 * (g + j);
      return wait<1>(c, c.full(k % C::kStages), (k / C::kStages) & 1);
    };
    auto wait_v = [&](int j) {
      const uint32_t v = 2 * (g + j) + 1;
      return wait<1>(c, c.full(v % C::kStages), (v / C::kStages) & 1);
    };
    auto wait_q = [&](int buf) {
      const bool there = wait<1>(c, c.q_full(buf), loads[buf]++ & 1);
      ptx::fence_proxy_async_smem();  // the queries came by cp.async
      return there;
    };
    // the first P V of a segment overwrites O: the last segment's must have been read
    auto wait_o = [&](int t) { return segs == 0 || wait<1>(c, c.o_empty(t), (segs - 1) & 1); };
    if (pair) {
      ok = wait_k(0);
      for (int t = 0; ok && t < 2; ++t) {
        ok = wait_q(t);
        if (!ok) break;
        ptx::tc_fence_after();
        qk(t, 0, t == 1);
      }
      for (int j = 0; ok && j < n; ++j) {
        for (int t = 0; ok && t < 2; ++t) {
          ok = wait<1>(c, c.p_full(t), (done[t] + j) & 1);
          if (ok && t == 0) ok = wait_v(j);
          if (ok && j == 0) ok = wait_o(t);
          if (!ok) break;
          ptx::tc_fence_after();
          pv(t, j, j == 0, t == 1);
          if (j + 1 < n) {
            if (t == 0) ok = wait_k(j + 1);
            if (!ok) break;
            ptx::tc_fence_after();
            qk(t, j + 1, t == 1);
          }
        }
      }
      done[0] += n;
      done[1] += n;
    } else {
      ok = wait_q(s.buf);
      for (int j = 0; ok && j < min(n, 2); ++j) {
        ok = wait_k(j);
        if (!ok) break;
        ptx::tc_fence_after();
        qk(j, j, true);
      }
      for (int j = 0; ok && j < n; ++j) {
        const int t = j & 1;
        ok = wait<1>(c, c.p_full(t), (done[t] + (j >> 1)) & 1);
        if (ok) ok = wait_v(j);
        if (ok && j < 2) ok = wait_o(t);
        if (!ok) break;
        ptx::tc_fence_after();
        pv(t, j, j < 2, true);
        if (j + 2 < n) {
          ok = wait_k(j + 2);
          if (!ok) break;
          ptx::tc_fence_after();
          qk(t, j + 2, true);
        }
      }
      done[0] += (n + 1) / 2;
      done[1] += n / 2;
    }
    g += n;
    ++segs;
  }
  if (!ok && issued) {
    if (ptx::elect_one()) ptx::mma_commit(c.drain());
    __syncwarp();
    drain_wait(c.drain(), 0);
  }
}

// ------------------------------------------------------------- softmax
struct Mask {
  uint32_t w[4];
};
// The nodes above new token i, and i itself.
__device__ __forceinline__ Mask nodes_above(const ChunkParams& p, int tok0, int i) {
  Mask m{};
  for (int at = i; at >= 0;) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at >> 5 == k) m.w[k] |= 1u << (at & 31);
    const int up = p.parents[tok0 + at];
    if ((up < -1 || up >= at) && p.status) atomicOr(p.status, kBatchBadInput);
    at = up >= at ? -1 : up;
  }
  return m;
}
// The first n bits of 128.
__device__ __forceinline__ Mask first_bits(int n) {
  Mask m;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int x = n - 32 * k;
    m.w[k] = x >= 32 ? 0xffffffffu : x <= 0 ? 0u : (1u << x) - 1;
  }
  return m;
}
// The mask moved up by n places (down, where n is negative), |n| < 128.
__device__ __forceinline__ Mask moved(const Mask& m, int n) {
  unsigned __int128 x = 0;
#pragma unroll
  for (int k = 3; k >= 0; --k) x = x << 32 | m.w[k];
  x = n >= 0 ? x << n : x >> -n;
  Mask r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.w[k] = (uint32_t)(x >> 32 * k);
  return r;
}

template <int D, bool kHalf>
__device__ void softmax_rows(const ChunkArgs& a, const Cta<D>& c, Walk walk, uint32_t tmem, int t) {
  using C = Cfg<D>;
  constexpr float kBase = kHalf ? kFp16Base : 0.f;  // m is that much below the largest score
  const ChunkParams& p = a.p;
  const int tid = threadIdx.x & 127, warp = tid >> 5;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t s_tmem = tmem + lanes + t * 128;
  const uint32_t o_tmem0 = tmem + lanes + 256, o_tmem = o_tmem0 + t * 128;
  // the segment's query rows of this tile, into buffer `buf`
  auto start = [&](const Segment& s, int buf) {
    const int row = (s.pair() ? t * 128 : 0) + tid;
    const bool there = row < s.rows;
    const int i = there ? row / p.gqa : 0, h = there ? row % p.gqa : 0;
    load_q<D>(p.q + (s.tok + i) * p.q_stride + (s.head * p.gqa + h) * D, there, c.base + buf * C::kQBytes, tid);
    ptx::cp_async_mbar_arrive_noinc(c.q_full(buf));
  };
  auto start_next = [&](const Segment& s) {
    if (s.pair())
      start(s, t);
    else if (t == 0)
      start(s, s.buf);
  };
  Segment s, s_next;
  bool more = walk.next(a, s), ok = true;
  if (more) start_next(s);
  uint32_t done = 0, segs = 0, joins = 0;
  while (ok && more) {
    const bool pair = s.pair();
    more = walk.next(a, s_next);
    // one tile's rows behind one tile's: the other buffer is free
    const bool early = more && !pair && !s_next.pair();
    if (early) start_next(s_next);
    const int row = (pair ? t * 128 : 0) + tid;
    const bool act = row - (tid & 31) < s.rows;  // this warp has rows
    const int i = s.first + row / p.gqa;         // the row's new token
    Mask above{};
    const bool tree = p.parents != nullptr;
    if (tree && row < s.rows && s.j1 * kTileTokens > s.base) above = nodes_above(p, s.tok - s.first, i);
    // keys before `clear` are seen by this row
    const int clear = row < s.rows ? (tree ? s.base : s.base + i + 1) : INT32_MAX;
    const int n = s.j1 - s.j0;
    float m = -INFINITY, l = 0.f;
    bool first = true;
    for (int j = pair ? 0 : t; j < n; j += pair ? 1 : 2) {
      ok = wait<0>(c, c.s_full(t), done++ & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      if (act) {
        float v[128];
#pragma unroll
        for (int k = 0; k < 4; ++k) ptx::tmem_ld32(s_tmem + k * 32, *reinterpret_cast<float(*)[32]>(v + k * 32));
        ptx::tmem_wait_ld();
        const int key0 = (s.j0 + j) * kTileTokens;
        if (__any_sync(0xffffffffu, clear < key0 + kTileTokens)) {
          const int in = clear - key0;  // seen keys of the step, a tree's aside
          Mask see = first_bits(in);
          if (tree && in < kTileTokens && in > -kTileTokens) {
            const Mask nodes = moved(above, in);
#pragma unroll
            for (int k = 0; k < 4; ++k) see.w[k] |= nodes.w[k];
          }
#pragma unroll
          for (int k = 0; k < 128; ++k) v[k] = see.w[k >> 5] >> (k & 31) & 1 ? v[k] : -INFINITY;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < 128; k += 2) m4[(k >> 1) & 3] = ptx::max3(m4[(k >> 1) & 3], v[k], v[k + 1]);
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.scale_log2;
        float alpha = 1.f;
        if (mx > m + (kBase + kRescaleLog2) || first) {
          alpha = first || m == -INFINITY ? 1.f : ptx::ex2(m - (mx - kBase));
          m = mx - kBase;
        }
        first = false;
        l *= alpha;
        // the S that was waited for was issued behind the tile's last P V: O holds it
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
    // every S of this tile is done: where it had its own query buffer, that is free
    if (more && pair) start_next(s_next);
    float a0 = 1.f, a1 = 0.f;  // factors of this tile's and the other's O
    if (!pair) {
      c.ml()[t * 128 + tid] = make_float2(m, l);
      ptx::mbar_arrive(c.joined());
      ok = wait<0>(c, c.joined(), joins++ & 1);
      if (!ok) break;
      const float2 o = c.ml()[(t ^ 1) * 128 + tid];
      const float top = fmaxf(m, o.x);
      a0 = m == -INFINITY ? 0.f : ptx::ex2(m - top);
      a1 = o.x == -INFINITY ? 0.f : ptx::ex2(o.x - top);
      l = a0 * l + a1 * o.y;
      m = top;
      if (n == 1) (t ? a0 : a1) = 0.f;
    }
    ok = wait<0>(c, c.o_full(t), segs & 1);
    if (!ok) break;
    ptx::tc_fence_after();
    if (more && !pair && !early) start_next(s_next);
    if (act) {
      const bool there = row < s.rows;
      const long long at = (long long)(s.tok + row / p.gqa) * p.hq + s.head * p.gqa + row % p.gqa;
      const long long slot = (2ll * blockIdx.x + (s.j0 == 0 ? 1 : 0)) * a.piece_rows + row;
      const bool whole = s.whole();
      const float inv = !whole ? 1.f : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
      a0 *= inv;
      a1 *= inv;
      // both tiles' warps have the same rows' lanes: with one tile's rows each takes half the columns
      constexpr int kColumns = D / 32;
      const int k0 = pair ? 0 : t * (kColumns / 2), k1 = pair ? kColumns : k0 + kColumns / 2;
      const uint32_t other = o_tmem0 + (t ^ 1) * 128;
      for (int k = k0; k < k1; ++k) {
        float o[32];
        if (pair || n > 1 || t == 0) {
          ptx::tmem_ld32(o_tmem + k * 32, o);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= a0;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
        }
        if (!pair && (n > 1 || t == 1)) {
          float o2[32];
          ptx::tmem_ld32(other + k * 32, o2);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = fmaf(o2[e], a1, o[e]);
        }
        if (there && whole) {
          uint16_t* dst = p.out + at * D + k * 32;
#pragma unroll
          for (int e = 0; e < 32; e += 16)
            ptx::st_global_v8(dst + e, pack2<kHalf>(o[e], o[e + 1]), pack2<kHalf>(o[e + 2], o[e + 3]),
                              pack2<kHalf>(o[e + 4], o[e + 5]), pack2<kHalf>(o[e + 6], o[e + 7]),
                              pack2<kHalf>(o[e + 8], o[e + 9]), pack2<kHalf>(o[e + 10], o[e + 11]),
                              pack2<kHalf>(o[e + 12], o[e + 13]), pack2<kHalf>(o[e + 14], o[e + 15]));
        } else if (there) {
          float* dst = a.piece_o + slot * D + k * 32;
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            ptx::st_global_v8(dst + e, __float_as_uint(o[e]), __float_as_uint(o[e + 1]),
                              __float_as_uint(o[e + 2]), __float_as_uint(o[e + 3]), __float_as_uint(o[e + 4]),
                              __float_as_uint(o[e + 5]), __float_as_uint(o[e + 6]), __float_as_uint(o[e + 7]));
        }
      }
      if (there && (pair || t == 0)) {
        if (!whole)
          a.piece_ml[slot] = make_float2(m, l);
        else if (p.lse)
          p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    }
    ptx::tc_fence_before();
    if (pair) {
      ptx::mbar_arrive_n(c.o_empty(t), 2);
    } else {
      ptx::mbar_arrive(c.o_empty(0));
      ptx::mbar_arrive(c.o_empty(1));
    }
    ++segs;
    s = s_next;
  }
  ptx::cp_async_wait_all();
}

// ------------------------------------------------------------- rows that see nothing
__device__ __forceinline__ void fill_tokens(const ChunkParams& p, int from, int to, int thread, int threads) {
  if (from >= to) return;
  const long long pieces = (long long)p.hq * p.d / 8;
  uint4* out = reinterpret_cast<uint4*>(p.out);
  for (long long i = from * pieces + thread; i < to * pieces; i += threads) out[i] = make_uint4(0, 0, 0, 0);
  if (p.lse)
    for (long long i = (long long)from * p.hq + thread; i < (long long)to * p.hq; i += threads) p.lse[i] = -INFINITY;
}
__device__ void fill_empty(const ChunkParams& p, bool broken, int thread) {
  constexpr int kFill = 64;
  const int all = gridDim.x * kFill, mine = blockIdx.x * kFill + thread;
  if (broken || p.n_req == 0) return fill_tokens(p, 0, p.n_tokens, mine, all);
  if (p.cu) {
    fill_tokens(p, 0, p.cu[0], mine, all);
    fill_tokens(p, p.cu[p.n_req], p.n_tokens, mine, all);
  }
  for (int b = blockIdx.x; b < p.n_req; b += gridDim.x) {
    const Raw raw = raw_of(p, b);
    int bad = 0;
    const Chunk r = checked(p, raw, bad);
    const int n = raw.last - raw.first;
    fill_tokens(p, raw.first, raw.first + (r.n < n ? n : min(max(r.n - r.len, 0), n)), thread, kFill);
  }
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tile_kernel(const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const ChunkArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const ChunkParams& p = a.p;
  Cta<D> c;
  c.base = ptx::smem_u32(smem);
  c.ptr = smem;
  c.status = p.status;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kOffBar + C::kBars * 8);
  c.abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + C::kBars * 8 + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Walk& s_walk = *reinterpret_cast<Walk*>(smem + C::kOffWalk);
  long long* s_sums = reinterpret_cast<long long*>(smem + C::kOffMl);  // (before it holds anything else)
  long long& s_in = s_sums[kThreads / 32];
  if (c.base & 1023) {  // the swizzled layouts need it
    if (threadIdx.x == 0) {
      if (p.status) atomicOr(p.status, kBatchTimeout);
      a.cuts[blockIdx.x].pieces = 0;
    }
    return;
  }
  // the merge may set itself up where there is room
  asm volatile("griddepcontrol.launch_dependents;");
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
      ptx::mbar_init(c.o_empty(t), 256);
    }
    ptx::mbar_init(c.joined(), 256);
    ptx::mbar_init(c.drain(), 1);
    *c.abort_flag = 0;
    s_walk.left = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(c.base + C::kOffBar + C::kBars * 8, kTmemCols);
    ptx::tmem_relinquish();
  }
  // Where the run starts: each thread sums up some requests, and the one whose
  // requests hold the run's first step looks for it.
  const int per = (p.n_req + kThreads - 1) / kThreads;
  const int b0 = min((int)threadIdx.x * per, p.n_req), b1 = min(b0 + per, p.n_req);
  int bad = 0;
  long long mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += steps_of_request(a, checked(p, raw_of(p, b), bad));
  const bool broken = __syncthreads_or(bad & kBadOffsets);
  if (broken) mine = 0;
  if (blockIdx.x == 0 && bad && p.status) atomicOr(p.status, bad & ~kBadOffsets);
  const long long before = scan_block(mine, s_sums, total) - mine;
  const long long run = max(quotient(total + a.grid - 1, a.grid), 1ll);
  const long long x0 = run * blockIdx.x, x1 = min(x0 + run, total);
  if (x0 < x1 && x0 >= before && x0 < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const Chunk r = checked(p, raw_of(p, b), bad);
      const long long steps = steps_of_request(a, r);
      if (x0 < at + steps) {
        s_walk.b = b;
        s_walk.r = r;
        s_walk.left = (int)(x1 - x0);
        s_in = x0 - at;
        break;
      }
      at += steps;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp == 0) {
    Walk w = s_walk;
    __syncwarp();
    int pieces = 0;
    if (w.left > 0) {
      const long long head_steps = steps_before(a, w.r, blocks_of(a, w.r));
      w.head = (int)quotient(s_in, head_steps);
      const long long in = s_in - w.head * head_steps;
      // the last block that starts at or before step `in`: 32 places at a time
      int lo = 0, hi = blocks_of(a, w.r);  // it lies in [lo, hi)
      while (hi - lo > 1) {
        const int each = (hi - lo + 31) / 32, k = lo + lane * each;
        const bool at_or_before = k < hi && steps_before(a, w.r, k) <= in;
        const int n = __popc(__ballot_sync(0xffffffffu, at_or_before));  // lane 0's is
        lo += (n - 1) * each;
        hi = min(hi, lo + each);
      }
      w.block = lo;
      w.j = (int)(in - steps_before(a, w.r, lo));
      w.buf = -1;
      w.look_ahead(p);
      const int np = steps_of_block(a, w.r, lo);
      if (w.j > 0 && w.j + w.left >= np) {
        const int first = (int)quotient(x0 - w.j, run), t = a.block_tokens;
        if (lane == 0) {
          Cut cut{};
          cut.pieces = (int)blockIdx.x - first + 1;
          cut.first = first;
          cut.tok = w.r.tok0 + lo * t;
          cut.rows = min(w.r.n - lo * t, t) * p.gqa;
          cut.head = w.head;
          a.cuts[blockIdx.x] = cut;
        }
        pieces = 1;
      }
    }
    if (lane == 0) {
      if (!pieces) a.cuts[blockIdx.x].pieces = 0;
      s_walk = w;
    }
  }
  __syncthreads();
  const Walk walk = s_walk;
  if (warp < 8) {
    ptx::setmaxnreg_inc<kSoftmaxRegs>();
    softmax_rows<D, kHalf>(a, c, walk, tmem, warp >> 2);
  } else {
    ptx::setmaxnreg_dec<kIssueRegs>();
    if (warp == 8)
      stream_kv<D>(&tmk, &tmv, a, c, walk);
    else if (warp == 9)
      issue_products<D, kHalf>(a, c, walk, tmem);
    else
      fill_empty(p, broken, threadIdx.x - 320);
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------- merge
// A warp a row of a segment that was cut; blockIdx.x is the run where it ends.
constexpr int kMergeWarps = 8;

template <int D, bool kHalf>
__global__ void __launch_bounds__(kMergeWarps * 32) chunk_merge_kernel(const ChunkArgs a) {
  constexpr int E = D / 32;  // columns of a lane
  const ChunkParams& p = a.p;
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = a.cuts[blockIdx.x];
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  if (cut.pieces == 0 || row >= cut.rows) return;
  auto slot = [&](int k) { return (2ll * (cut.first + k) + (k == 0 ? 1 : 0)) * a.piece_rows + row; };
  float m = -INFINITY;
  for (int k = lane; k < cut.pieces; k += 32) m = fmaxf(m, a.piece_ml[slot(k)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, acc[E] = {};
  for (int k0 = 0; k0 < cut.pieces; k0 += 32) {
    const int count = min(cut.pieces - k0, 32);
    float w = 0.f;
    if (lane < count) {
      const float2 ml = a.piece_ml[slot(k0 + lane)];
      w = ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - m);
      l = fmaf(w, ml.y, l);
    }
#pragma unroll 4
    for (int k = 0; k < count; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float* src = a.piece_o + slot(k0 + k) * D + lane * E;
      float v[E];
      if constexpr (E == 4) {
        const float4 x = *reinterpret_cast<const float4*>(src);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(src);
        v[0] = x.x, v[1] = x.y;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(wk, v[e], acc[e]);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  const long long at = (long long)(cut.tok + row / p.gqa) * p.hq + cut.head * p.gqa + row % p.gqa;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<kHalf>(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Sizes of a run, and where its workspace lies.
size_t lay_out(const ChunkParams& p, uint8_t* work, ChunkArgs* a) {
  a->p = p;
  a->block_tokens = kBlockRows / p.gqa;
  const long long blocks = ((long long)p.n_tokens / a->block_tokens + std::min(p.n_req, p.n_tokens)) * p.hkv;
  a->grid = (int)std::max(1ll, std::min<long long>(p.num_sms, blocks * (p.width ? p.width / kStepPages + 1 : p.num_sms)));
  a->piece_rows = (int)std::min<long long>(kBlockRows, (long long)p.n_tokens * p.gqa);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* from = work ? work + at : nullptr;
    at += (bytes + 255) / 256 * 256;
    return from;
  };
  // (for a whole grid: the tables' width is not among the sizes that ask for the workspace)
  const size_t rows = 2 * (size_t)p.num_sms * a->piece_rows;
  a->cuts = reinterpret_cast<Cut*>(take(p.num_sms * sizeof(Cut)));
  a->piece_ml = reinterpret_cast<float2*>(take(rows * sizeof(float2)));
  a->piece_o = reinterpret_cast<float*>(take(rows * p.d * sizeof(float)));
  return at;
}

template <int D, bool kHalf>
cudaError_t run(const ChunkArgs& a, cudaStream_t s) {
  const ChunkParams& p = a.p;
  CUtensorMap mk, mv;
  cudaError_t e = make_page_map(&mk, p.k_pages, D, p.hkv, p.num_pages, false);
  if (e != cudaSuccess) return e;
  e = make_page_map(&mv, p.v_pages, D, p.hkv, p.num_pages, true);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(chunk_tile_kernel<D, kHalf>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem;
  cfg.stream = s;
  e = cudaLaunchKernelEx(&cfg, chunk_tile_kernel<D, kHalf>, mk, mv, a);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.grid, (a.piece_rows + kMergeWarps - 1) / kMergeWarps);
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<D, kHalf>, a);
}

}  // namespace

size_t chunk_workspace(const ChunkParams& p) {
  ChunkArgs a{};
  return p.n_tokens ? lay_out(p, nullptr, &a) : 0;
}

cudaError_t launch_chunk_attention(const ChunkParams& p, void* workspace, cudaStream_t s) {
  if (p.n_tokens == 0) return cudaSuccess;
  ChunkArgs a{};
  lay_out(p, static_cast<uint8_t*>(workspace), &a);
  if (p.d == 128) return p.dtype == kFp16 ? run<128, true>(a, s) : run<128, false>(a, s);
  return p.dtype == kFp16 ? run<64, true>(a, s) : run<64, false>(a, s);
}

}  // namespace ta
