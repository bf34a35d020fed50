// Attention of several new tokens of each request over its pages, prompts and
// trees of drafts alike, on tcgen05 (sm_103a).
//
// Query rows are (token, q head of a kv head's group); a block of a request's new
// tokens gives two tiles of up to 128 rows that share a kv head's keys.  A CTA (one
// per SM) streams K and V past them, 128 keys a step, with the products'
// accumulators in TMEM:
//   S = Q K^T (128 x 128), online softmax on one row per thread, P as 16-bit
//   pairs over S, O += P V.
// A tile's step is a task.  Tasks stand in one row, segment behind segment, and go
// to the two halves of TMEM and of the softmax warps in turn: while one task's
// softmax runs, the products of its neighbours do, also across segments.  With two
// tiles in the block (a prompt: bound by the products and the softmax between
// them) each step is two tasks.  With one (drafts: bound by reading K and V once)
// a step is one task, the halves take the steps in turn, and their sums are joined
// where the segment ends.
//
// Steps of all (request, kv head, block) segments stand in one line, and a CTA
// takes a contiguous run of it, whatever the lengths are.  Runs are equal in cost:
// a segment's steps and kSegmentCost more.  A segment within one run is final;
// pieces of one that lies in several go out as {m, l} and the unnormalised O in 32
// bits and are joined by the merge,
//   m = max m_i, out = sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i.
// A CTA has at most one piece that began before its run and one that goes on
// behind it.
//
// Which keys a row sees is a mask of 128 bits a step, made only in steps that hold
// a key that some row does not see: from the row's end for a prompt, and for a
// tree from the nodes above the row's, collected along parents once a block.
//
// Roles: warps 0-3 and 4-7 are the softmax of the two halves (thread = row = TMEM
// lane), warp 8 streams K and V by TMA (and zeroes V's rows past a request's end),
// warps 9 and 11 issue the products of a half each, warp 10 (one thread) lists the
// run's segments for the others and brings their queries.  A half's products run
// in the order of issue, so S of its next task may be issued right behind the P V
// that still reads P from the same columns.
//
// P is rounded to the queries' type, as the products take it (see prefix_attn.h for
// what that costs and for fp16's base); l sums the weights in 32 bits before that.
// The output is off by 0.0020 of itself in bf16 (rounding the exact result: 0.0016),
// 0.00029 in fp16 (0.00021).
//
// Measured (d = 128, 64 q heads on 8): a prompt of 16384 tokens in 3.05 ms, 1440
// TFLOP/s, 0.74 of the measured bf16 peak and 0.84 of what it sustains.  A pair of
// tasks takes about 2900 cycles where its products take 2048: S, softmax and P V of
// one half follow one another, and two halves cover each other only in part (P
// handed over in two parts: 3200 us; two threads a row: 3560).  What takes the
// softmax a few registers more spills its scores (finished rows by TMA through shared
// memory: 4500).  26 drafts behind 500 to 4000 tokens (64 requests, 32 heads on 8,
// 458 MB) in 107 us: 4.3 TB/s in all, about 6 while K and V stream; the rest is the
// start, runs that do not end together, and the merge.
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
using tiles::pack2;
using tiles::rescale_o;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kThreads = 384;
constexpr int kSoftmaxRegs = 216, kIssueRegs = 72;
static_assert(256 * kSoftmaxRegs + 128 * kIssueRegs <= kThreads * 168, "register split too large");
constexpr float kRescaleLog2 = 8.f;  // O is rescaled when a row's maximum grows by more than 2^8
constexpr uint32_t kTmemCols = 512;  // S of both tiles (128 columns each), O of both (128 each)
constexpr int kTile = 128;           // query rows of a tile, at most
constexpr int kTurnTries = 1 << 24;  // a second or so
constexpr long long kIdleLimitNs = 20000000000ll;  // without a segment to list or queries to bring
// What a segment costs beside its steps, in steps (24 packed prompts took 166 us
// with 2, 176 with 1, 172 with 3).
constexpr int kSegmentCost = 2;
constexpr int kStepPages = kTileTokens / kPage;

struct Cut {  // a segment that lies in several runs, told by the run where it ends
  int pieces, first, tok, tokens, head;
  int broken;  // (the first one's) no token has a request
  int pad[2];
};

struct ChunkArgs {
  ChunkParams p;
  Cut* cuts;         // [grid]
  float2* piece_ml;  // [2 * grid][piece_rows]: {m, l}
  float* piece_o;    // [2 * grid][piece_rows][d]
  int piece_rows, grid;
  int tile_tokens, block_tokens;  // of a tile (its rows are whole tokens), of two
  int block_shift;                // log2(block_tokens), or -1
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
// sum over i < n of floor((i + c) / 2^s)
__device__ __forceinline__ long long shifted_sum(long long n, long long c, int s) {
  const auto below = [&](long long x) {  // over i < x of floor(i / 2^s)
    const long long q = x >> s, r = x & ((1ll << s) - 1);
    return (q * (q - 1) / 2 << s) + q * r;
  };
  return below(c + n) - below(c);
}
// Blocks of a request that see nothing (all before the first token of the cache).
__device__ __forceinline__ int blind_blocks(const ChunkArgs& a, const Chunk& r) {
  return r.len < r.n ? (r.n - r.len) / a.block_tokens : 0;
}
// (Out of line, and so is what calls it: code that runs once is fetched once.)
// What the first k blocks cost, one kv head: their steps, and kSegmentCost for each
// that has some.
__device__ __noinline__ long long cost_before(const ChunkArgs& a, const Chunk& r, int k) {
  const int blocks = blocks_of(a, r), base = r.len - r.n, t = a.block_tokens;
  const int k0 = min(blind_blocks(a, r), k);
  long long sum = (long long)kSegmentCost * (k - k0);
  if (k == blocks && k > 0) sum += (r.len + kTileTokens - 1) / kTileTokens, --k;
  const long long n = k - k0, first = base + (long long)(k0 + 1) * t + kTileTokens - 1;
  if (n <= 0) return sum;
  // of floor((first + i t) / 128)
  if (a.block_shift >= 7) return sum + (n * (n - 1) / 2 << (a.block_shift - 7)) + n * (first >> 7);
  if (a.block_shift >= 0) return sum + shifted_sum(n, first >> a.block_shift, 7 - a.block_shift);
  return sum + floor_sum(n, kTileTokens, t, first);
}
__device__ __forceinline__ long long cost_of_request(const ChunkArgs& a, const Chunk& r) {
  if (r.n == 0 || r.len == 0) return 0;
  if (r.n <= a.block_tokens) return (long long)a.p.hkv * ((r.len + kTileTokens - 1) / kTileTokens + kSegmentCost);
  return a.p.hkv * cost_before(a, r, blocks_of(a, r));
}

struct alignas(16) Segment {
  int b, head;
  int tok, first, tokens;  // the block's first token, its number among the request's new ones, how many
  int len, base, end;      // tokens of the request, those before its new ones, keys of the block
  int np, j0, j1;          // steps in all, this run's (none: there are no more segments)
  int buf;                 // which query buffer; 2: two tiles, a buffer each
  __device__ __forceinline__ bool pair() const { return buf == 2; }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == np; }
  __device__ __forceinline__ int tasks() const { return (j1 - j0) << (int)pair(); }
};

// The CTA's run, segment by segment.
struct Walk {
  int b, head, block, j, lead, left;  // the next step's place, cost units before it, cost units left
  Chunk r;
  Raw ahead;                          // the next request's
  int buf;                            // of the last segment

  __device__ __forceinline__ void look_ahead(const ChunkParams& p) {
    if (b + 1 < p.n_req) ahead = raw_of(p, b + 1);
  }
  __device__ __forceinline__ bool next(const ChunkArgs& a, Segment& s) {
    if (left <= lead) return false;
    left -= lead;
    const int t = a.block_tokens;
    s.b = b;
    s.head = head;
    s.first = block * t;
    s.tok = r.tok0 + s.first;
    s.tokens = min(r.n - s.first, t);
    s.len = r.len;
    s.base = r.len - r.n;
    s.end = end_of(a, r, block);
    s.np = (s.end + kTileTokens - 1) / kTileTokens;
    s.j0 = j;
    s.j1 = min(s.np, j + left);
    left -= s.j1 - s.j0;
    // one tile's queries: not into the buffer of the ones before
    buf = s.tokens > a.tile_tokens ? 2 : buf == 0;
    s.buf = buf;
    lead = kSegmentCost;
    if (left > lead) advance(a);
    return true;
  }
  // To the next segment, which there has to be.
  __device__ __forceinline__ void advance(const ChunkArgs& a) {
    j = 0;
    lead = kSegmentCost;
    if ((++block) * a.block_tokens < r.n) return;
    if (++head == a.p.hkv) {
      head = 0;
      int bad = 0;
      do {
        ++b;
        r = checked(a.p, ahead, bad);
        look_ahead(a.p);
      } while ((r.n == 0 || r.len == 0) && b + 1 < a.p.n_req);
    }
    block = blind_blocks(a, r);
  }
};

// A place in the line of costs: the request, and how far behind its start.
struct Place {
  long long in;
  int b;
  Chunk r;
};
// Its segment (a warp looks for it): how far behind that one's start, and its cost.
struct Spot {
  int head, block, behind, cost;
};
__device__ __noinline__ Spot spot_of(const ChunkArgs& a, const Place& at) {
  const int lane = threadIdx.x & 31, blocks = blocks_of(a, at.r);
  const auto cost_of = [&](int k) {
    const int end = k < blocks ? end_of(a, at.r, k) : 0;
    return end > 0 ? (end + kTileTokens - 1) / kTileTokens + kSegmentCost : 0;
  };
  Spot s;
  if (blocks <= 32) {  // a block a lane
    const int cost = cost_of(lane);
    int behind = cost;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, behind, o);
      if (lane >= o) behind += x;
    }
    const int head_cost = __shfl_sync(0xffffffffu, behind, 31);
    s.head = (int)quotient(at.in, head_cost);
    const int in = (int)(at.in - (long long)s.head * head_cost);
    s.block = __popc(__ballot_sync(0xffffffffu, behind <= in));  // those that end before it
    s.cost = __shfl_sync(0xffffffffu, cost, s.block);
    s.behind = in - __shfl_sync(0xffffffffu, behind - cost, s.block);
    return s;
  }
  const long long head_cost = cost_before(a, at.r, blocks);
  s.head = (int)quotient(at.in, head_cost);
  const long long in = at.in - s.head * head_cost;
  // the last block that starts at or before `in`: 32 places at a time
  int lo = 0, hi = blocks;  // it lies in [lo, hi)
  while (hi - lo > 1) {
    const int each = (hi - lo + 31) / 32, k = lo + lane * each;
    const bool at_or_before = k < hi && cost_before(a, at.r, k) <= in;
    const int n = __popc(__ballot_sync(0xffffffffu, at_or_before));  // lane 0's is
    lo += (n - 1) * each;
    hi = min(hi, lo + each);
  }
  s.block = lo;
  s.behind = (int)(in - cost_before(a, at.r, lo));
  s.cost = cost_of(lo);
  return s;
}

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kQBytes = 128 * D * 2;               // one tile of queries
  static constexpr int kStageBytes = kTileTokens * D * 2;   // K or V of a step
  // K and V take turns.  (A fifth stage, 10 at d = 64: 110 us against 106 for 64 trees of
  // drafts, 157 against 159 for 24 packed prompts, else the same.)
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kHead = kPage * D * 2;               // a page-head
  static constexpr int kOffStage = 2 * kQBytes;
  static constexpr int kOffMl = kOffStage + kStages * kStageBytes;  // {m, l} of both halves' rows
  static constexpr int kOffBar = kOffMl + 2 * 128 * 8;
  static constexpr int kListed = 8;  // segments that the roles may be apart
  static constexpr int kBars = 3 * kStages + 15 + 2 * kListed;
  // the TMEM address, the abort flag, copies issued: ring entries, of each query buffer
  static constexpr int kOffWords = kOffBar + kBars * 8;
  static constexpr int kOffList = (kOffWords + 20 + 15) / 16 * 16;
  static constexpr int kOffPlace = kOffList + kListed * sizeof(Segment);
  static constexpr int kSmem = kOffPlace + sizeof(Place);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

extern __shared__ __align__(1024) uint8_t chunk_smem[];

// Places in shared memory.  (No member: what the roles hold in registers decides how
// fast they are.)
template <int D>
struct Cta {
  using C = Cfg<D>;
  static __device__ uint32_t base() { return ptx::smem_u32(chunk_smem); }
  static __device__ volatile int* abort_flag() { return reinterpret_cast<volatile int*>(chunk_smem + C::kOffWords + 4); }

  __device__ uint32_t bar(int i) const { return base() + C::kOffBar + 8 * i; }
  __device__ uint32_t full(int s) const { return bar(s); }
  __device__ uint32_t empty(int s) const { return bar(C::kStages + s); }
  __device__ uint32_t land(int s) const { return bar(2 * C::kStages + s); }
  __device__ uint32_t q_full(int t) const { return bar(3 * C::kStages + t); }
  __device__ uint32_t s_full(int t) const { return bar(3 * C::kStages + 2 + t); }
  __device__ uint32_t p_full(int t) const { return bar(3 * C::kStages + 4 + t); }
  __device__ uint32_t o_full(int t) const { return bar(3 * C::kStages + 6 + t); }
  __device__ uint32_t o_empty(int t) const { return bar(3 * C::kStages + 8 + t); }
  __device__ uint32_t q_empty(int t) const { return bar(3 * C::kStages + 10 + t); }
  __device__ uint32_t joined() const { return bar(3 * C::kStages + 12); }
  __device__ uint32_t drain(int t) const { return bar(3 * C::kStages + 13 + t); }
  __device__ uint32_t listed(uint32_t i) const { return bar(3 * C::kStages + 15 + i % C::kListed); }
  __device__ uint32_t unlisted(uint32_t i) const { return bar(3 * C::kStages + 15 + C::kListed + i % C::kListed); }
  __device__ Segment* segment(uint32_t i) const {
    return reinterpret_cast<Segment*>(chunk_smem + C::kOffList) + i % C::kListed;
  }
  static __device__ uint32_t round(uint32_t i) { return i / C::kListed & 1; }
  __device__ uint32_t kv_issued() const { return base() + C::kOffWords + 8; }
  __device__ uint32_t q_issued(int buf) const { return base() + C::kOffWords + 12 + 4 * buf; }
  __device__ uint32_t stage(int s) const { return base() + C::kOffStage + s * C::kStageBytes; }
  __device__ float2* ml() const { return reinterpret_cast<float2*>(chunk_smem + C::kOffMl); }
};

// tiles::wait with this kernel's abort flag and status word.
template <int kRole, int D>
__device__ __forceinline__ bool wait(const Cta<D>& c, int32_t* status, uint32_t bar, uint32_t parity) {
  return tiles::wait<kRole>(bar, parity, c.abort_flag(), status);
}

// Copies issued, counted.  A reader that does not use every entry of a ring cannot
// tell by parity alone whether a stage's barrier is in the entry's phase or still in
// the one before: the entry must have been issued, and then it is.
__device__ __forceinline__ void publish_issued(uint32_t word, uint32_t n) {
  asm volatile("st.release.cta.shared::cta.u32 [%0], %1;" ::"r"(word), "r"(n) : "memory");
}
__device__ __forceinline__ uint32_t issued_of(uint32_t word) {
  uint32_t n;
  asm volatile("ld.acquire.cta.shared::cta.u32 %0, [%1];" : "=r"(n) : "r"(word) : "memory");
  return n;
}
__device__ __noinline__ bool wait_issued_slow(uint32_t word, uint32_t least, volatile int* abort_flag, int32_t* status) {
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t n = 1;; ++n) {
    if ((int32_t)(issued_of(word) - least) >= 0) return true;
    if ((n & 15) == 0) {
      if (*abort_flag) return false;
      if ((long long)(ptx::globaltimer() - t0) > tiles::kWaitLimitNs) {
        *abort_flag = 1;
        if (status) atomicOr(status, kBatchTimeout);
        return false;
      }
    }
  }
}
// True once at least so many have been issued; the same in all lanes of the warp.
template <int D>
__device__ __forceinline__ bool wait_issued(const Cta<D>& c, int32_t* status, uint32_t word, uint32_t least) {
  bool ok = (int32_t)(issued_of(word) - least) >= 0;
  if (!ok) ok = wait_issued_slow(word, least, c.abort_flag(), status);
  return __all_sync(0xffffffffu, ok);
}

// Those that let go of a listed segment: the copies' warp, the products' two, the
// queries' thread and eight warps of softmax.
constexpr uint32_t kReaders = 12;

// ------------------------------------------------------------- copies
template <int D>
__device__ void stream_kv(const CUtensorMap* tmk, const CUtensorMap* tmv, const ChunkArgs& a,
                          const Cta<D>& c) {
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
  Segment s, s_next{};
  uint32_t g = 0, seg = 0;
  uint32_t zeroed = 0;  // phase of each stage's land barrier
  const auto read = [&](Segment& to) {  // the next listed segment; false: given up
    if (!wait<1>(c, p.status, c.listed(seg), c.round(seg))) return false;
    to = *c.segment(seg);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(c.unlisted(seg));
    ++seg;
    return true;
  };
  bool ok = read(s);
  int next = ok && s.j0 < s.j1 ? page_of(s, s.j0) : 0;
  while (ok && s.j0 < s.j1) {
    ok = read(s_next);
    if (!ok) break;
    const bool more = s_next.j0 < s_next.j1;
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
        if (g >= (uint32_t)C::kStages && !wait<1>(c, p.status, c.empty(st), (g / C::kStages + 1) & 1)) {
          ok = false;
          break;
        }
        const bool zero = v == 1 && last < kPage;
        const uint32_t bar = zero ? c.land(st) : c.full(st);
        const uint32_t dst = c.stage(st);
        const bool leader = ptx::elect_one();
        if (leader) publish_issued(c.kv_issued(), g + 1);
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
          if (wait<1>(c, p.status, bar, par)) {
            uint8_t* head = chunk_smem + C::kOffStage + st * C::kStageBytes + (nb - 1) * C::kHead;
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

// A warp finds where the run [x0, x1) starts, and says what the merge has to know.
__device__ __forceinline__ Walk start_of_run(const ChunkArgs& a, const Place& place, long long x0, long long x1,
                                             long long run, bool broken) {
  Walk w{};  // (no steps: left and lead are 0)
  Cut cut{};
  cut.broken = broken;
  if (x0 < x1) {
    const Spot spot = spot_of(a, place);
    w.b = place.b;
    w.r = place.r;
    w.head = spot.head;
    w.block = spot.block;
    w.left = (int)(x1 - x0);
    w.j = max(spot.behind - kSegmentCost, 0);
    w.lead = max(kSegmentCost - spot.behind, 0);
    w.buf = 2;
    w.look_ahead(a.p);
    if (w.j > 0 && w.j + w.left >= spot.cost - kSegmentCost) {  // a piece that began before, and ends here
      cut.first = (int)quotient(x0 - w.j, run);                  // (x0 - j: its first step)
      cut.pieces = (int)blockIdx.x - cut.first + 1;
      cut.tok = w.r.tok0 + w.block * a.block_tokens;
      cut.tokens = min(w.r.n - w.block * a.block_tokens, a.block_tokens);
      cut.head = w.head;
    }
  }
  if ((threadIdx.x & 31) == 0) a.cuts[blockIdx.x] = cut;
  return w;
}

// One thread of a warp: lists the run's segments as there is room, and brings each
// one's queries as soon as its buffer is free.
template <int D>
__device__ void list_segments(const CUtensorMap* tmq, const ChunkArgs& a, const Cta<D>& c, Walk walk) {
  using C = Cfg<D>;
  if (threadIdx.x & 31) return;
  uint32_t listed = 0, brought = 0;  // segments
  uint32_t loads[2] = {0, 0};        // of each query buffer
  int tile = 0;                      // of two, brought already
  bool all = false;
  uint64_t since = ptx::globaltimer();
  for (uint32_t polls = 0; !all || brought < listed; ++polls) {
    bool idle = true;
    if (!all && (listed < C::kListed || ptx::mbar_test_wait(c.unlisted(listed), c.round(listed) ^ 1))) {
      Segment s{};
      if (!walk.next(a, s)) {
        all = true;
        s.j0 = s.j1 = 0;
      }
      *c.segment(listed) = s;
      ptx::mbar_arrive(c.listed(listed));
      if (!all) ++listed;
      idle = false;
    }
    if (brought < listed) {
      const Segment& s = *c.segment(brought);
      const int buf = s.pair() ? tile : s.buf;
      const uint32_t n = buf ? loads[1] : loads[0];
      if (n == 0 || ptx::mbar_test_wait(c.q_empty(buf), (n - 1) & 1)) {
        const uint32_t bar = c.q_full(buf);
        publish_issued(c.q_issued(buf), n + 1);
        ptx::mbar_arrive_expect_tx(bar, a.tile_tokens * a.p.gqa * D * 2);
        const int tok = s.tok + (s.pair() ? tile * a.tile_tokens : 0);
#pragma unroll
        for (int h = 0; h < C::kHalves; ++h)
          ptx::tma_load_3d(c.base() + buf * C::kQBytes + h * (kTile * 128), tmq, 64 * h, s.head * a.p.gqa, tok, bar);
        buf ? ++loads[1] : ++loads[0];
        if (s.pair() && tile == 0) {
          tile = 1;
        } else {
          tile = 0;
          ptx::mbar_arrive(c.unlisted(brought));
          ++brought;
        }
        idle = false;
      }
    }
    if (!idle) {
      since = ptx::globaltimer();
      continue;
    }
    __nanosleep(32);
    if ((polls & 15) == 0) {
      if (*c.abort_flag()) break;
      // (a segment may take as long as its steps, each of whose waits is limited)
      if ((long long)(ptx::globaltimer() - since) > kIdleLimitNs) {
        *c.abort_flag() = 1;
        if (a.p.status) atomicOr(a.p.status, kBatchTimeout);
        break;
      }
    }
  }
  if (*c.abort_flag())  // the copies in flight land before the CTA may end
#pragma unroll
    for (int buf = 0; buf < 2; ++buf)
      if (loads[buf] > 0) drain_wait(c.q_full(buf), (loads[buf] - 1) & 1);
}

// ------------------------------------------------------------- products
// A warp for each half, so that one's waits and the other's products overlap.  S of
// a half's next task is issued right behind P V of the one before, in one go where
// its keys are there already.
template <int D, bool kHalf>
__device__ void issue_products(const ChunkParams& p, const Cta<D>& c, uint32_t tmem, int t) {
  using C = Cfg<D>;
  constexpr uint32_t kType = kHalf ? 0u : (1u << 7) | (1u << 10);
  constexpr uint32_t kDescQK =
      (ptx::idesc_bf16(128, kTileTokens, 0) & ~((1u << 7) | (1u << 10))) | kType;
  constexpr uint32_t kDescPV = (ptx::idesc_bf16(128, D, 1) & ~((1u << 7) | (1u << 10))) | kType;
  const uint64_t desc_q = ptx::sdesc_sw128(c.base(), 16, 1024);
  const uint64_t desc_k = ptx::sdesc_sw128(c.stage(0), 16, 1024);
  const uint64_t desc_v = ptx::sdesc_sw128(c.stage(0), 2048, 1024);
  const uint32_t s_tmem = tmem + t * 128, o_tmem = tmem + 256 + t * 128;
  struct Task {
    uint32_t step;      // of the run: K is ring entry 2 step, V the next one
    int pages, buf;     // of 16 keys; the query buffer
    bool first, last;   // of the half's tasks of the segment
    bool pair, single;  // the block has two tiles; the segment is this task alone
  };
  int idx = 0, n = 0, j0 = 0, n_pages = 0, buf = 0;  // of the segment: this half's next step, steps, ...
  bool pair = false;
  uint32_t seg = 0, tasks = 0, before = 0;           // listed segments, all tasks and steps before the next one
  uint32_t base = 0;                                 // steps before this segment
  uint32_t q_loads[2] = {0, 0};                      // of each query buffer, with this segment's
  // This half's next task: 1, 0 where there is none, -1: given up.
  const auto next_task = [&](Task& k) {
    while (idx >= n) {
      if (!wait<1>(c, p.status, c.listed(seg), c.round(seg))) return -1;
      const Segment& s = *c.segment(seg);
      n = s.j1 - s.j0;
      if (n == 0) return 0;
      j0 = s.j0;
      n_pages = (s.end + kPage - 1) / kPage;
      pair = s.pair();
      buf = s.buf;
      __syncwarp();
      if (ptx::elect_one()) ptx::mbar_arrive(c.unlisted(seg));
      __syncwarp();
      ++seg;
      base = before;
      before += n;
      idx = pair ? 0 : (int)(tasks & 1) ^ t;
      tasks += n << (int)pair;
      q_loads[0] += pair || buf == 0;
      q_loads[1] += pair || buf == 1;
    }
    k.step = base + idx;
    k.pages = min(kStepPages, n_pages - (j0 + idx) * kStepPages);
    k.buf = pair ? t : buf;
    k.pair = pair;
    k.single = !pair && n == 1;
    k.first = idx < (pair ? 1 : 2);
    idx += pair ? 1 : 2;
    k.last = idx >= n;
    return 1;
  };
  const auto stage_of = [](uint32_t entry) { return (int)(entry % C::kStages); };
  const auto phase_of = [](uint32_t entry) { return entry / C::kStages & 1; };
  // one elected lane
  const auto scores = [&](const Task& k, uint64_t dq, uint64_t dk) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
      ptx::mma_bf16(s_tmem, dq + (off >> 4), dk + (off >> 4), kDescQK, kk > 0);
    }
    ptx::mma_commit(c.s_full(t));
    // a buffer is free when both halves are done with it
    ptx::mma_commit(c.empty(stage_of(2 * k.step)));
    if (!k.pair) ptx::mma_commit(c.empty(stage_of(2 * k.step)));
    if (k.last) {
      ptx::mma_commit(c.q_empty(k.buf));
      if (k.pair || k.single) ptx::mma_commit(c.q_empty(k.buf));
    }
  };
  const auto wait_entry = [&](uint32_t entry) {
    return wait_issued(c, p.status, c.kv_issued(), entry + 1) && wait<1>(c, p.status, c.full(stage_of(entry)), phase_of(entry));
  };
  const auto wait_for_scores = [&](const Task& k) {
    if (!wait_entry(2 * k.step)) return false;
    if (!k.first) return true;
    const uint32_t loads = k.buf ? q_loads[1] : q_loads[0];
    return wait_issued(c, p.status, c.q_issued(k.buf), loads) && wait<1>(c, p.status, c.q_full(k.buf), (loads - 1) & 1);
  };
  // whether it would not wait
  const auto can_score = [&](const Task& k) {
    bool can = (int32_t)(issued_of(c.kv_issued()) - (2 * k.step + 1)) >= 0 &&
               ptx::mbar_test_wait(c.full(stage_of(2 * k.step)), phase_of(2 * k.step));
    if (can && k.first) {
      const uint32_t loads = k.buf ? q_loads[1] : q_loads[0];
      can = (int32_t)(issued_of(c.q_issued(k.buf)) - loads) >= 0 && ptx::mbar_test_wait(c.q_full(k.buf), (loads - 1) & 1);
    }
    return (bool)__all_sync(0xffffffffu, can);
  };
  const auto desc_of_q = [&](const Task& k) { return desc_q + (uint32_t)(k.buf * C::kQBytes >> 4); };
  const auto desc_of = [&](uint64_t desc, uint32_t entry) { return desc + (uint32_t)(stage_of(entry) * C::kStageBytes >> 4); };

  Task now{}, next{};
  int have = next_task(now);
  bool ok = have >= 0, issued = false;
  if (have > 0) {
    ok = wait_for_scores(now);
    if (ok) {
      ptx::tc_fence_after();
      if (ptx::elect_one()) scores(now, desc_of_q(now), desc_of(desc_k, 2 * now.step));
      __syncwarp();
      issued = true;
    }
  }
  uint32_t done = 0, o_read = 0;
  while (ok && have > 0) {
    const int more = next_task(next);
    if (more < 0) {
      ok = false;
      break;
    }
    const uint64_t dq = desc_of_q(next), dk = desc_of(desc_k, 2 * next.step), dv = desc_of(desc_v, 2 * now.step + 1);
    const int v_stage = stage_of(2 * now.step + 1);
    ok = wait_entry(2 * now.step + 1);
    // the first P V of a segment overwrites O: the last one's must have been read
    if (ok && now.first) {
      if (o_read) ok = wait<1>(c, p.status, c.o_empty(t), (o_read - 1) & 1);
      ++o_read;
    }
    if (ok) ok = wait<1>(c, p.status, c.p_full(t), done++ & 1);
    if (!ok) break;
    const bool together = more && can_score(next);
    ptx::tc_fence_after();
    if (ptx::elect_one()) {
      const uint32_t add = now.first ? 0 : 1;
      if (now.pages == kStepPages) {  // 16 tokens: 8 columns of P
#pragma unroll
        for (int b = 0; b < kStepPages; ++b)
          ptx::mma_bf16_ts(o_tmem, s_tmem + b * 8, dv + b * (C::kHead >> 4), kDescPV, b > 0 ? 1 : add);
      } else {
        for (int b = 0; b < now.pages; ++b)
          ptx::mma_bf16_ts(o_tmem, s_tmem + b * 8, dv + b * (C::kHead >> 4), kDescPV, b > 0 ? 1 : add);
      }
      ptx::mma_commit(c.empty(v_stage));
      if (!now.pair) ptx::mma_commit(c.empty(v_stage));
      if (now.last) ptx::mma_commit(c.o_full(t));
      if (together) scores(next, dq, dk);
    }
    __syncwarp();
    if (more && !together) {
      ok = wait_for_scores(next);
      if (!ok) break;
      ptx::tc_fence_after();
      if (ptx::elect_one()) scores(next, dq, dk);
      __syncwarp();
    }
    now = next;
    have = more;
  }
  if (!ok && issued) {
    if (ptx::elect_one()) ptx::mma_commit(c.drain(t));
    __syncwarp();
    drain_wait(c.drain(t), 0);
  }
}

// ------------------------------------------------------------- softmax
struct Mask {
  uint32_t w[4];
};
// The nodes above each lane's new token i (none below 0), and i itself: the
// request's parents, four a lane, are handed round as the lanes climb.
__device__ __forceinline__ Mask nodes_above(const ChunkParams& p, int tok0, int n, int i) {
  const int lane = threadIdx.x & 31;
  int up[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int node = k * 32 + lane;
    up[k] = node < n ? p.parents[tok0 + node] : -1;
    if (up[k] < -1 || up[k] >= node) {
      if (p.status) atomicOr(p.status, kBatchBadInput);
      up[k] = -1;
    }
  }
  Mask m{};
  int at = i;
  while (__any_sync(0xffffffffu, at >= 0)) {
    int next = -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = __shfl_sync(0xffffffffu, up[k], at & 31);
      if (at >> 5 == k) {
        m.w[k] |= 1u << (at & 31);
        next = x;
      }
    }
    at = next;
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

template <int kColumns>
__device__ __forceinline__ void load_columns(uint32_t tmem, float (&o)[kColumns]) {
#pragma unroll
  for (int k = 0; k < kColumns; k += 32) ptx::tmem_ld32(tmem + k, *reinterpret_cast<float(*)[32]>(o + k));
}

template <int D, bool kHalf, bool kTree>
__device__ void softmax_rows(const ChunkArgs& a, const Cta<D>& c, uint32_t tmem, int t) {
  using C = Cfg<D>;
  constexpr float kBase = kHalf ? kFp16Base : 0.f;  // m is that much below the largest score
  const ChunkParams& p = a.p;
  const int tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t s_tmem = tmem + lanes + t * 128;
  const uint32_t o_tmem0 = tmem + lanes + 256, o_tmem = o_tmem0 + t * 128;
  const int in_tile = tid / p.gqa, in_group = tid - in_tile * p.gqa;  // the row's token and head
  uint32_t task = 0;  // of the whole run
  uint32_t done = 0, joins = 0;
  uint32_t o_phase = 0;  // of each half's O, a bit each
  Mask above{};
  int above_b = -1, above_tok = 0;  // the block (request, row's token) that `above` was made for
  bool ok = true;
  for (uint32_t seg = 0;; ++seg) {
    ok = wait<0>(c, p.status, c.listed(seg), c.round(seg));
    const Segment& s = *c.segment(seg);
    const int n = s.j1 - s.j0;
    if (!ok || n == 0) break;
    const bool pair = s.pair(), alone = pair || n == 1;  // a half has the rows' O to itself
    const uint32_t f = task & 1;                         // the half of the segment's first task
    const uint32_t o_now = o_phase;
    task += s.tasks();
    o_phase ^= pair || n > 1 ? 3u : 1u << f;
    const auto let_go = [&]() {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(c.unlisted(seg));
    };
    if (!pair && n == 1 && t != (int)f) {
      let_go();
      continue;
    }
    const int i0 = pair ? t * a.tile_tokens : 0;      // the tile's first token in the block
    const int rows = min(s.tokens - i0, a.tile_tokens) * p.gqa;
    const bool there = tid < rows, act = tid - lane < rows;  // the row, the warp's rows
    const int i = s.first + i0 + in_tile;               // the row's new token
    if (kTree && act && s.j1 * kTileTokens > s.base &&
        (above_b != s.b || __any_sync(0xffffffffu, there && above_tok != i))) {
      above = nodes_above(p, s.tok - s.first, s.len - s.base, there ? i : -1);
      above_b = s.b;
      above_tok = i;
    }
    // keys before `clear` are seen by this row
    const int clear = there ? (kTree ? s.base : s.base + i + 1) : INT32_MAX;
    const int j0 = s.j0;
    float m = -INFINITY, l = 0.f;
    bool first = true;
    for (int j = pair ? 0 : (int)(f ^ t); j < n; j += pair ? 1 : 2) {
      ok = wait<0>(c, p.status, c.s_full(t), done++ & 1);
      if (!ok) break;
      ptx::tc_fence_after();
      if (act) {
        float v[128];
        load_columns(s_tmem, v);
        ptx::tmem_wait_ld();
        const int key0 = (j0 + j) * kTileTokens;
        if (__any_sync(0xffffffffu, clear < key0 + kTileTokens)) {
          const int in = clear - key0;  // seen keys of the step, a tree's aside
          Mask see = first_bits(in);
          if (kTree && in < kTileTokens && in > -kTileTokens) {
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
        // The halves take turns with their exponentials: side by side on the same
        // schedulers both take as long as one behind the other, and the tensor cores
        // then wait for both (16384 tokens of 64 heads: 3.24 ms, in turns 3.04).
        const uint32_t turn = 2 * done - 3 + t;  // the task before this one (done counts it already)
        if (done + t > 1) {
          const uint32_t bar = c.p_full(t ^ 1), parity = turn >> 1 & 1;
          bool there = ptx::mbar_test_wait(bar, parity);  // (in line: a call would spill the scores)
          for (int tries = 0; !there && tries < kTurnTries; ++tries) there = ptx::mbar_test_wait(bar, parity);
          // (where it never comes, the waits behind this one give up)
        }
        l *= alpha;
        // the S that was waited for was issued behind the half's last P V: O holds it
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
    // This half's last P V first, then the exchange: the segment's first P V was issued
    // once O of the half's last segment had been read, by both halves where they shared
    // it, and they read it after each other's {m, l}.  Without it the next segment's
    // could overwrite what a late warp of the other half has still to read.  (Two sets of
    // {m, l} by turns instead: 115 us against 107 for 64 trees of drafts.)
    ok = wait<0>(c, p.status, c.o_full(t), o_now >> t & 1);
    if (!ok) break;
    float a0 = 1.f, a1 = 0.f;  // factors of this half's and the other's O
    if (!alone) {
      c.ml()[t * 128 + tid] = make_float2(m, l);
      ptx::mbar_arrive(c.joined());
      ok = wait<0>(c, p.status, c.joined(), joins++ & 1);
      if (!ok) break;
      const float2 o = c.ml()[(t ^ 1) * 128 + tid];
      const float top = fmaxf(m, o.x);
      a0 = m == -INFINITY ? 0.f : ptx::ex2(m - top);
      a1 = o.x == -INFINITY ? 0.f : ptx::ex2(o.x - top);
      l = a0 * l + a1 * o.y;
      m = top;
    }
    if (!alone) ok = wait<0>(c, p.status, c.o_full(t ^ 1), o_now >> (t ^ 1) & 1);
    if (!ok) break;
    ptx::tc_fence_after();
    const bool whole = s.whole();
    const float inv = !whole ? 1.f : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    a0 *= inv;
    a1 *= inv;
    // Both halves' warps have the same rows' lanes: joined, each takes half the columns.
    const long long at = (long long)(s.tok + i0 + in_tile) * p.hq + s.head * p.gqa + in_group;
    const long long slot = (2ll * blockIdx.x + (s.j0 == 0 ? 1 : 0)) * a.piece_rows + (pair ? t * kTile : 0) + tid;
    const int columns = alone ? D : D / 2, c0 = alone ? 0 : t * (D / 2);
    const uint32_t o_other = o_tmem0 + (t ^ 1) * 128;
    const auto o_is_read = [&]() {
      ptx::tc_fence_before();
      if (alone) {
        ptx::mbar_arrive_n(c.o_empty(t), 2);
      } else {
        ptx::mbar_arrive(c.o_empty(0));
        ptx::mbar_arrive(c.o_empty(1));
      }
    };
    if (act) {
      constexpr int kChunk = D / 2;
      for (int k = c0; k < c0 + columns; k += kChunk) {
        float o[kChunk];
        load_columns(o_tmem + k, o);
        if (alone) {
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kChunk; ++e) o[e] *= a0;
        } else {
          float o2[kChunk];
          load_columns(o_other + k, o2);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < kChunk; ++e) o[e] = fmaf(o2[e], a1, o[e] * a0);
        }
        if (k + kChunk == c0 + columns) o_is_read();
        if (there && whole) {
          uint16_t* dst = p.out + at * D + k;
#pragma unroll
          for (int e = 0; e < kChunk; e += 16)
            ptx::st_global_v8(dst + e, pack2<kHalf>(o[e], o[e + 1]), pack2<kHalf>(o[e + 2], o[e + 3]),
                              pack2<kHalf>(o[e + 4], o[e + 5]), pack2<kHalf>(o[e + 6], o[e + 7]),
                              pack2<kHalf>(o[e + 8], o[e + 9]), pack2<kHalf>(o[e + 10], o[e + 11]),
                              pack2<kHalf>(o[e + 12], o[e + 13]), pack2<kHalf>(o[e + 14], o[e + 15]));
        } else if (there) {
          float* dst = a.piece_o + slot * D + k;
#pragma unroll
          for (int e = 0; e < kChunk; e += 8)
            ptx::st_global_v8(dst + e, __float_as_uint(o[e]), __float_as_uint(o[e + 1]), __float_as_uint(o[e + 2]),
                              __float_as_uint(o[e + 3]), __float_as_uint(o[e + 4]), __float_as_uint(o[e + 5]),
                              __float_as_uint(o[e + 6]), __float_as_uint(o[e + 7]));
        }
      }
      if (there && (alone || t == 0)) {
        if (!whole)
          a.piece_ml[slot] = make_float2(m, l);
        else if (p.lse)
          p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    } else {
      o_is_read();
    }
    let_go();
  }
}

template <int D, bool kHalf, bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tile_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const ChunkArgs a) {
  using C = Cfg<D>;
  const ChunkParams& p = a.p;
  const Cta<D> c{};
  uint8_t* const smem = chunk_smem;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::kOffWords);
  const int warp = threadIdx.x >> 5;
  Place& s_place = *reinterpret_cast<Place*>(smem + C::kOffPlace);
  long long* s_sums = reinterpret_cast<long long*>(smem + C::kOffMl);  // (before it holds anything else)
  if (c.base() & 1023) {  // the swizzled layouts need it
    if (threadIdx.x == 0) {
      if (p.status) atomicOr(p.status, kBatchTimeout);
      a.cuts[blockIdx.x].pieces = a.cuts[blockIdx.x].broken = 0;
    }
    return;
  }
  // the merge may set itself up where there is room
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      ptx::mbar_init(c.full(s), 1);
      ptx::mbar_init(c.empty(s), 2);
      ptx::mbar_init(c.land(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      ptx::mbar_init(c.q_full(t), 1);
      ptx::mbar_init(c.q_empty(t), 2);
      ptx::mbar_init(c.drain(t), 1);
      ptx::mbar_init(c.s_full(t), 1);
      ptx::mbar_init(c.p_full(t), 128);
      ptx::mbar_init(c.o_full(t), 1);
      ptx::mbar_init(c.o_empty(t), 256);
    }
    for (int i = 0; i < C::kListed; ++i) {
      ptx::mbar_init(c.listed(i), 1);
      ptx::mbar_init(c.unlisted(i), kReaders);
    }
    ptx::mbar_init(c.joined(), 256);
    *c.abort_flag() = 0;
    publish_issued(c.kv_issued(), 0);
    publish_issued(c.q_issued(0), 0);
    publish_issued(c.q_issued(1), 0);
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(c.base() + C::kOffWords, kTmemCols);
    ptx::tmem_relinquish();
  }
  // Each thread sums up some requests, and the one whose requests hold the run's
  // start says which.
  const int per = (p.n_req + kThreads - 1) / kThreads;
  const int b0 = min((int)threadIdx.x * per, p.n_req), b1 = min(b0 + per, p.n_req);
  int bad = 0;
  long long mine = 0, total;
  Chunk only{};  // where a thread has one request
  for (int b = b0; b < b1; ++b) {
    only = checked(p, raw_of(p, b), bad);
    mine += cost_of_request(a, only);
  }
  // offsets out of order leave no request any tokens; told with the sum, which stays below
  constexpr long long kBroken = 1ll << 48;
  const long long before = scan_block(mine + (bad & kBadOffsets ? kBroken : 0ll), s_sums, total) - mine;
  const bool broken = total >= kBroken;
  if (broken) total = 0;
  if (blockIdx.x == 0 && bad && p.status) atomicOr(p.status, bad & ~kBadOffsets);
  const long long run = max(quotient(total + a.grid - 1, a.grid), 1ll);
  const long long x0 = min(run * blockIdx.x, total), x1 = min(x0 + run, total);
  if (x0 < x1 && x0 >= before && x0 < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const Chunk r = per == 1 ? only : checked(p, raw_of(p, b), bad);
      const long long cost = per == 1 ? mine : cost_of_request(a, r);
      if (x0 < at + cost) {
        s_place = Place{x0 - at, b, r};
        break;
      }
      at += cost;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk walk{};
  if (warp == 10) walk = start_of_run(a, s_place, x0, x1, run, broken);  // (its calls need the registers of the launch)
  if (warp < 8) {
    ptx::setmaxnreg_inc<kSoftmaxRegs>();
    softmax_rows<D, kHalf, kTree>(a, c, tmem, warp >> 2);
  } else {
    ptx::setmaxnreg_dec<kIssueRegs>();
    if (warp == 8)
      stream_kv<D>(&tmk, &tmv, a, c);
    else if (warp == 10)
      list_segments<D>(&tmq, a, c, walk);
    else
      issue_products<D, kHalf>(p, c, tmem, warp == 9 ? 0 : 1);
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
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
  const int blocks = gridDim.x * gridDim.y, block = blockIdx.y * gridDim.x + blockIdx.x;
  const int all = blocks * blockDim.x, mine = block * blockDim.x + thread;
  if (broken || p.n_req == 0) return fill_tokens(p, 0, p.n_tokens, mine, all);
  if (p.cu) {
    fill_tokens(p, 0, p.cu[0], mine, all);
    fill_tokens(p, p.cu[p.n_req], p.n_tokens, mine, all);
  }
  for (int b = block; b < p.n_req; b += blocks) {
    const Raw raw = raw_of(p, b);
    int bad = 0;
    const Chunk r = checked(p, raw, bad);
    const int n = raw.last - raw.first;
    fill_tokens(p, raw.first, raw.first + (r.n < n ? n : min(max(r.n - r.len, 0), n)), thread, blockDim.x);
  }
}

// ------------------------------------------------------------- merge
// A warp four rows of a segment that was cut; blockIdx.x is the run where it ends.
// And the rows that see nothing.  Bound by the loads that depend on one another
// (the cut, its pieces' sums, the pieces) and, where many segments are cut, by
// reading the pieces: 152 of two pieces of 256 rows at d = 128, 40 MB in 10 us (18
// with one row a warp).  Rows that no segment has are read with the others.
constexpr int kMergeWarps = 8, kMergeRows = 4;

template <int D, bool kHalf>
__global__ void __launch_bounds__(kMergeWarps * 32) chunk_merge_kernel(const ChunkArgs a) {
  constexpr int E = D / 32;  // columns of a lane
  const ChunkParams& p = a.p;
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = a.cuts[blockIdx.x];
  fill_empty(p, a.cuts[0].broken, threadIdx.x);
  const int row0 = (blockIdx.y * kMergeWarps + (threadIdx.x >> 5)) * kMergeRows;
  if (cut.pieces == 0 || row0 >= a.piece_rows) return;
  const auto there = [&](int row) {
    const int in_tile = (row & (kTile - 1)) / p.gqa;
    return row < a.piece_rows && in_tile < a.tile_tokens && row / kTile * a.tile_tokens + in_tile < cut.tokens;
  };
  const auto slot = [&](int k, int row) { return (2ll * (cut.first + k) + (k == 0 ? 1 : 0)) * a.piece_rows + row; };
  // lane i has row i & 3 of piece i >> 2, eight pieces at a time
  const int mine = row0 + (lane & 3);
  const bool have = there(mine);
  const auto ml_of = [&](int k) {
    return have && k < cut.pieces ? a.piece_ml[slot(k, mine)] : make_float2(-INFINITY, 0.f);
  };
  float m = -INFINITY;
  for (int k0 = 0; k0 < cut.pieces; k0 += 8) m = fmaxf(m, ml_of(k0 + (lane >> 2)).x);
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.f, acc[kMergeRows][E] = {};
  for (int k0 = 0; k0 < cut.pieces; k0 += 8) {
    const float2 ml = ml_of(k0 + (lane >> 2));
    const float w = ml.x == -INFINITY ? 0.f : ptx::ex2(ml.x - m);
    l = fmaf(w, ml.y, l);
    const int count = min(cut.pieces - k0, 8);
#pragma unroll 2
    for (int k = 0; k < count; ++k) {
      float v[kMergeRows][E];
#pragma unroll
      for (int r = 0; r < kMergeRows; ++r) {
        const float* src = a.piece_o + slot(k0 + k, row0 + r) * D + lane * E;
        if (row0 + r >= a.piece_rows) {  // (rows there in no segment are not read into a result)
#pragma unroll
          for (int e = 0; e < E; ++e) v[r][e] = 0.f;
        } else if constexpr (E == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          v[r][0] = x.x, v[r][1] = x.y, v[r][2] = x.z, v[r][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          v[r][0] = x.x, v[r][1] = x.y;
        }
      }
#pragma unroll
      for (int r = 0; r < kMergeRows; ++r) {
        const float wk = __shfl_sync(0xffffffffu, w, k * 4 + r);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[r][e] = fmaf(wk, v[r][e], acc[r][e]);
      }
    }
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
#pragma unroll
  for (int r = 0; r < kMergeRows; ++r) {
    const int row = row0 + r;
    const float inv_r = __shfl_sync(0xffffffffu, inv, r);
    if (!there(row)) continue;
    const int in_tile = (row & (kTile - 1)) / p.gqa, tok = row / kTile * a.tile_tokens + in_tile;
    const long long at = (long long)(cut.tok + tok) * p.hq + cut.head * p.gqa + (row & (kTile - 1)) % p.gqa;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + at * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack2<kHalf>(acc[r][e] * inv_r, acc[r][e + 1] * inv_r);
    if (lane == r && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// Sizes of a run, and where its workspace lies.
size_t lay_out(const ChunkParams& p, uint8_t* work, ChunkArgs* a) {
  a->p = p;
  a->tile_tokens = kTile / p.gqa;
  a->block_tokens = 2 * a->tile_tokens;
  a->block_shift = -1;
  for (int e = 0; e <= 8; ++e)
    if (a->block_tokens == 1 << e) a->block_shift = e;
  const long long blocks = ((long long)p.n_tokens / a->block_tokens + std::min(p.n_req, p.n_tokens)) * p.hkv;
  a->grid = (int)std::max(1ll, std::min<long long>(p.num_sms, blocks * (p.width ? p.width / kStepPages + 1 : p.num_sms)));
  a->piece_rows = p.n_tokens > a->tile_tokens ? 2 * kTile : p.n_tokens * p.gqa;
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
  const auto kernel = p.parents ? chunk_tile_kernel<D, kHalf, true> : chunk_tile_kernel<D, kHalf, false>;
  CUtensorMap mq, mk, mv;
  cudaError_t e = make_query_map(&mq, p.q, D, p.hq, p.n_tokens, std::max<long long>(p.q_stride, (long long)p.hq * D),
                                 p.gqa, a.tile_tokens);
  if (e != cudaSuccess) return e;
  e = make_page_map(&mk, p.k_pages, D, p.hkv, p.num_pages, false);
  if (e != cudaSuccess) return e;
  e = make_page_map(&mv, p.v_pages, D, p.hkv, p.num_pages, true);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::kSmem;
  cfg.stream = s;
  e = cudaLaunchKernelEx(&cfg, kernel, mq, mk, mv, a);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.grid, (a.piece_rows + kMergeWarps * kMergeRows - 1) / (kMergeWarps * kMergeRows));
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
