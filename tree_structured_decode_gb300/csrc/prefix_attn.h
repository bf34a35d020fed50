// Structures shared by the kernels of the shared-prefix attention.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "batch.h"

namespace ta {

constexpr int kTileTokens = 128;  // keys of a step of the tensor-core tiles
constexpr int kLineWarps = 12;    // of a CTA of the line kernel

// What the kernels know of a request, checked: its first token and row count
// lie in the batch, its pages in the table.
struct Request {  // 24 bytes
  long long p0;  // steps in the line before it
  int len, n, tok0, np;  // tokens held, queries, the first one, steps of a segment
};

// One division; most are of 32-bit numbers, which takes a third of the time.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// One line of segments (a tile of query rows of one kv head against one
// request's keys), cut into equal runs of steps: the requests' own tokens, or
// the prefix as a request of its own whose rows are all tokens'.
struct Line {
  Request* req;       // (own tokens)
  long long* sizes;   // (own tokens) [0] steps in the line, [1] a run; the prefix's Runs: [2] longer, [3] shorter, [4] n_longer
  float* piece_o;     // [2 * runs][tile_rows][d]
  float2* piece_ml;   // [2 * runs][tile_rows]: {m, l}
  float* row_o;       // [tokens * hq][d]: segments in one run
  float2* row_ml;
  int tile_rows, tile_shift;  // tile_rows = 1 << tile_shift
  int step;           // keys
  int runs;           // warps (or CTAs) that the line is cut for
};

struct Args {
  PrefixParams p;
  Line line[2];  // own tokens, prefix
  int32_t* request_of;  // [tokens] (of tokens that are some request's)
  int mixed;          // the prefix (of few rows) stands in the own tokens' line, before them
  int self;           // the line kernel's CTAs check and sum up the requests themselves
  int tiles;          // the prefix goes to the tensor cores
  int join;           // own segments in one run are final
};

__device__ __forceinline__ int tiles_of(const Request& r, int gqa, const Line& L) {
  return (r.n * gqa + L.tile_rows - 1) >> L.tile_shift;
}

// A line's runs: n_longer of one length, then those of another.
struct Runs {
  long long longer, shorter, n_longer;
  __device__ __forceinline__ long long start(long long w) const {
    return w <= n_longer ? w * longer : n_longer * longer + (w - n_longer) * shorter;
  }
  __device__ __forceinline__ long long of(long long x) const {
    const long long in = x - n_longer * longer;
    return in < 0 || shorter == 0 ? quotient(x, longer) : n_longer + quotient(in, shorter);
  }
};

// The prefix as one request of all queries.  Tokens of no request (the padding
// of a batch of fixed size) are not counted.
struct Cuts {
  Request one;
  long long total;
};
__device__ __forceinline__ Cuts prefix_cuts(const Args& a) {
  const PrefixParams& p = a.p;
  const Line& L = a.line[1];
  Cuts c;
  c.one.p0 = 0;
  c.one.len = p.prefix_len;
  c.one.tok0 = 0;
  c.one.n = p.cu ? min(max(p.cu[p.n_req], 0), p.n_tokens) : p.n_tokens;
  c.one.np = L.step == kPage ? (p.prefix_len + kPage - 1) / kPage : (p.prefix_len + kTileTokens - 1) / kTileTokens;
  c.total = (long long)tiles_of(c.one, p.gqa, L) * p.hkv * c.one.np;
  return c;
}

// How the SMs are shared.  The tiles are bound by arithmetic, the line kernel by
// memory, so that half the SMs take the line nearly as fast (512 requests of 64
// heads, 240 tokens each: 114 us on 76, 103 on 152).  The others go to the tiles
// alone; those of the line take shorter runs of tiles behind it: 458 us instead
// of 483 in all.  (A quarter, 478: 203 us for the line next to the tiles.)  A
// step of the tiles lasts as long as kStepCost pages of the line there.
// All SMs take the line first where it has much more to do than the tiles (256
// requests of 300 tokens behind 200: 69 us, on half the SMs 74), and from fewer
// pages on where its rows are in tiles of 16, so that it is not bound by memory
// alone (128 requests of four drafts: 39 us on 152, 59 on 76, the whole 91 against
// 100; 64 requests of 300 tokens, four drafts, behind 500: 43 against 34).
constexpr int kStepCost = 13;
constexpr int kFewPages = 12;  // of a warp
constexpr int kLateSteps = 2;  // what a CTA that starts behind the line loses
struct Split {
  int line_ctas;
  Runs runs;  // of tiles
};
__device__ __forceinline__ Split split_of(const Args& a, const Cuts& prefix, long long pages) {
  const int sms = a.line[1].runs;
  const long long steps = prefix.total;
  const int warps = sms / 2 * kLineWarps;
  const bool half = pages <= warps * kFewPages + (a.line[0].tile_rows == 8 ? 4 * kStepCost * steps : 0);
  const int behind = half ? sms / 2 : 0;
  const int alone = sms - behind;
  Split s{sms, Runs{0, 0, alone}};
  if (behind > 0) {
    s.line_ctas = behind;
    const long long each = quotient(kStepCost * steps + pages, sms) - quotient(pages, behind);
    s.runs.shorter = max(quotient(max(each, 0ll), kStepCost) - kLateSteps, 0ll);
  }
  long long run = max(quotient(steps - s.runs.shorter * behind + alone - 1, alone), 1ll);
  if (s.runs.shorter == 0 && run < prefix.one.np) {
    // a few steps more where no run has two segments then: one costs about 5
    const int n = prefix.one.np, k = (int)quotient(n, run), even = n / k;
    if (even * k == n && even - run <= 4) run = even;
  }
  s.runs.longer = run;
  return s;
}
// The own tokens' line (with the prefix before them, if mixed) on so many CTAs.
__device__ __forceinline__ long long own_run(const Args& a, long long total, int ctas) {
  const long long warps = (long long)ctas * kLineWarps;
  return max(quotient(total + warps - 1, warps), 1ll);
}
// What the kernels after it need.
__device__ __forceinline__ void publish_sizes(const Args& a, long long total, const Split& s) {
  long long* to = a.line[0].sizes;
  to[0] = total;
  to[1] = own_run(a, total, s.line_ctas);
  to[2] = s.runs.longer;
  to[3] = s.runs.shorter;
  to[4] = s.runs.n_longer;
}
__device__ __forceinline__ Runs own_runs(const Args& a) {
  return Runs{a.line[0].sizes[1], 0, a.line[0].runs};
}
__device__ __forceinline__ Runs prefix_runs(const Args& a) {
  const long long* from = a.line[0].sizes;
  return a.mixed ? own_runs(a) : Runs{from[2], from[3], from[4]};
}

// Where a line's pieces of one query row lie: n of them (0: the line has no
// keys for it), piece k in o(k) and ml(k).
struct Pieces {
  const Line* L;
  long long w0, row;
  int n, in;
  __device__ __forceinline__ long long slot(int k) const {
    return (2 * (w0 + k) + (k == 0 ? 1 : 0)) * L->tile_rows + in;
  }
  __device__ __forceinline__ const float* o(int k, int d) const {
    return n == 1 ? L->row_o + row * d : L->piece_o + slot(k) * d;
  }
  __device__ __forceinline__ float2 ml(int k) const {
    return __ldcg(n == 1 ? L->row_ml + row : L->piece_ml + slot(k));
  }
};
// Pieces of token tok's q head h (of kv head kvh, its in-th) in line L, whose
// request there is r.
__device__ __forceinline__ Pieces pieces_of(const Line& L, const Request& r, const Runs& runs,
                                            const PrefixParams& p, int tok, int kvh, int in_head) {
  Pieces q{&L, 0, (long long)tok * p.hq + kvh * p.gqa + in_head, 0, 0};
  if (r.np == 0) return q;
  const int in = (tok - r.tok0) * p.gqa + in_head;
  const long long seg = (long long)kvh * tiles_of(r, p.gqa, L) + (in >> L.tile_shift);
  const long long first = r.p0 + seg * r.np;
  q.w0 = runs.of(first);
  const long long last = first + r.np - 1;
  q.n = last < runs.start(q.w0 + 1) ? 1 : (int)(runs.of(last) - q.w0) + 1;
  q.in = in & (L.tile_rows - 1);
  return q;
}

// A request, checked.  Offsets out of order (kBadOffsets, beside the status bit)
// could give tokens to many requests and make the line any length: then no
// request has queries.
constexpr int kBadOffsets = 256;
__device__ __forceinline__ Request checked(const PrefixParams& p, int b, int& bad) {
  Request r;
  const int len = p.lens[b];
  int first = b, last = b + 1;
  if (p.cu) first = p.cu[b], last = p.cu[b + 1];
  if (len < 0 || len > p.width * kPage) bad |= kBatchBadInput;
  if (first < 0 || last < first || last > p.n_tokens) bad |= kBatchBadInput | kBadOffsets;
  r.len = min(max(len, 0), p.width * kPage);
  r.tok0 = min(max(first, 0), p.n_tokens);
  r.n = min(max(last, r.tok0), p.n_tokens) - r.tok0;
  r.np = (r.len + kPage - 1) / kPage;
  r.p0 = 0;
  return r;
}
__device__ __forceinline__ long long steps_of(const Args& a, const Request& r) {
  return (long long)tiles_of(r, a.p.gqa, a.line[0]) * r.np * a.p.hkv;
}
// What the merge reads of it.
__device__ __forceinline__ void publish(const Args& a, int b, const Request& r) {
  a.line[0].req[b] = r;
  if (a.p.cu)
    for (int t = r.tok0; t < r.tok0 + r.n; ++t) a.request_of[t] = b;
}
// Inclusive scan over a block; s_warp holds a word per warp, total is the sum.
__device__ __forceinline__ long long scan_block(long long mine, long long* s_warp, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long v = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += o;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  total = 0;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    if (w == warp) v += total;
    total += s_warp[w];
  }
  return v;
}

// Weights P = 2^(s - m) are rounded to the queries' type for the product with V,
// whose operands are of one type; the sums l add them before that.  Half a step
// of the type each (2^-8 or 2^-11 of the weight), of either sign: the output's
// error grows by 40 %, root mean square 0.0023 of the output's in bf16 and 0.00029
// in fp16 behind 32768 tokens, where its own rounding alone gives 0.0017 and
// 0.00021.  P as a pair of 16-bit parts would double P V.
// fp16 ends at 2^-24, so m is held kFp16Base below the largest score there and P
// goes up to 2^(8 + 7): a weight loses at most 2^-32 of the largest.  (With P up to
// 2^8 it was 2^-25, and thousands of small weights together were lost by more than
// the output's rounding.)
constexpr float kFp16Base = 7.f;

// Most query rows of a tile of the tensor-core prefix kernel: two of 128.
constexpr int kTileRows = 256;
// The prefix's pieces by tcgen05 (a.line[1] cut in steps of kTileTokens keys).
cudaError_t launch_prefix_tiles(const Args& a, const CUtensorMap& mk_half, const CUtensorMap& mv,
                                cudaStream_t s);

}  // namespace ta
