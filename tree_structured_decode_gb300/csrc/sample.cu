// Sampling with temperature, top-k, top-p and min-p from given random numbers
// (sm_103a).
//
// The token of a row is a comparison of running sums with u times their total,
// so a sum that is off in its last bits gives another token.  The weights are
// therefore whole numbers,
//   w_i = round(2^42 exp((l_i - max) / T)),
// off by at most 0.67 units (below exp(kLeast) they are 0), and every sum of them
// is exact: the result does not depend on the order or the grid, and is that of
// exact weights except where a border lies within vocab * 0.67 * 2^-42 (4e-8 at
// 262144 logits, all off in one direction) of the largest weight.
//
// A row belongs to one CTA, or to a cluster of two or four where rows are few or long;
// what the CTAs of a cluster have to tell one another goes through distributed
// shared memory.  A part that fits lies in shared memory; a larger one is read
// again, by then from L2.  The passes:
//   1  the largest logit (and NaNs);
//   2  with top-k or top-p: the bins, a histogram of counts and weights over the
//      weight's exponent (2048 bins down to 2^-16 or 2^-24; a second one for what
//      is below where the first does not suffice), and the row's weight.  The
//      bin where the kept prefix of the order (logit descending, index ascending)
//      ends follows by a scan;
//   3  for each such bin, the sums of what lies above it, segment by segment in
//      index order, and a list of the bin's values, which one CTA compares all
//      with all.  (A bin of more values is cut further by the float's bits.)
// What is kept is then: bits above `key`, or equal and index at most `last`.
// A draw finds its segment by the segments' running sums and walks through it.
// Bound by instructions: about 150 a logit in all passes, 42 of them a weight's.
// 256 rows of 128000 fp32 logits with top-p take 220 us (131 MB: 0.6 TB/s).  A
// histogram without its atomics saves 6 us, two weights at a time in packed
// arithmetic nothing.  One row is bound by the barriers between its passes.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "batch.h"
#include "ptx.cuh"

namespace ta {
namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kNumWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kSegments = 256;     // of a CTA's part, at most
// A segment of the longest part has 1024 logits, 32 a lane, whose two sums (of up
// to 2^20 and 2^21 each) stay in 32 bits.
static_assert(kMaxVocab <= kSegments * 1024, "a lane's sums of a segment");
// Bytes of logits held in shared memory, where two CTAs share an SM and where
// each has one for itself.
constexpr int kHeld = 61440, kHeldAlone = 163840;
template <bool kAlone>
constexpr int held_most = kAlone ? kHeldAlone : kHeld;
constexpr int kFew = 384;          // values of a bin that are compared all with all (at most the threads of a CTA)
// The first histogram's range of exponents: down to 2^-16 for top-k, which need
// not look at more than the largest logits, and to 2^-24 for top-p alone, which
// weighs all of them anyway (256 rows of 128000, top-p 0.7 to 1: with 2^-16 a
// third of the rows needed a second one, 76 us for the slowest).
constexpr float kNearK = 11.0903549f, kNearP = 16.6355323f;
constexpr int kSafe = 1023;            // values of a bin whose two 32-bit sums cannot overflow
constexpr int kMaxRanks = 4;
constexpr u64 kOne = 1ull << 42;   // the weight of the largest logit
constexpr float kLeast = -30.498476f;  // below exp(this) = 2^-44 a weight rounds to 0

// 2^(i / 32) and 2^(i / 1024), i = 0..31, in units of 2^-62
__constant__ u64 kCoarse[32] = {
    0x4000000000000000ull, 0x4166c34c5615d0ecull, 0x42d561b3e6243d8aull, 0x444c0740496d4294ull,
    0x45cae0f1f545eb73ull, 0x47521cc5a2e6a9e0ull, 0x48e1e9b9d588e19bull, 0x4a7a77d47f7b84b1ull,
    0x4c1bf828c6dc54b8ull, 0x4dc69cdceaa72a9cull, 0x4f7a993048d088d7ull, 0x513821818624b40cull,
    0x52ff6b54d8a89c75ull, 0x54d0ad5a753e077cull, 0x56ac1f752150a563ull, 0x5891fac0e95612c8ull,
    0x5a827999fcef3242ull, 0x5c7dd7a3b17dcf75ull, 0x5e8451cfac061b5full, 0x6096266533384a2bull,
    0x62b39508aa836d6full, 0x64dcdec3371793d1ull, 0x6712460a8fc24072ull, 0x69540ec8f895722dull,
    0x6ba27e656b4eb57aull, 0x6dfddbcbed791babull, 0x70666f76154a7089ull, 0x72dc8373be41a454ull,
    0x75606373ee921c97ull, 0x77f25ccdee6d7ae6ull, 0x7a92be8a92436616ull, 0x7d41d96db915019dull,
};
__constant__ u64 kFine[32] = {
    0x4000000000000000ull, 0x400b18178ba33b14ull, 0x4016321b687027a8ull, 0x40214e0bebbe0c77ull,
    0x402c6be96af2fb58ull, 0x40378bb43b83d3d8ull, 0x4042ad6cb2f445c2ull, 0x404dd11326d6d3b5ull,
    0x4058f6a7ecccd5b6ull, 0x40641e2b5a867bc0ull, 0x406f479dc5c2d058ull, 0x407a72ff844fbb1full,
    0x4085a050ec0a036aull, 0x4090cf9252dd52cfull, 0x409c00c40ec437beull, 0x40a733e675c82816ull,
    0x40b268f9de0183baull, 0x40bd9ffe9d979724ull, 0x40c8d8f50ac09dffull, 0x40d413dd7bc1c5bcull,
    0x40df50b846ef302bull, 0x40ea8f85c2abf60eull, 0x40f5d046456a29b8ull, 0x410112fa25aad99eull,
    0x410c57a1b9fe12f6ull, 0x41179e3d5902e44dull, 0x4122e6cd59676024ull, 0x412e315211e89f86ull,
    0x41397dcbd952c4a6ull, 0x4144cc3b0680fd7aull, 0x41501c9ff05d8654ull, 0x415b6efaede1ac83ull,
};
// ln 2 / 1024 = hi + lo, hi a multiple of 2^-34 (n hi is exact where it is subtracted)
constexpr float kStepHi = 0x1.62e43p-11f, kStepLo = -0x1.05c61p-39f;
constexpr float kSteps = 0x1.715476p+10f;  // 1024 / ln 2

// Order-preserving bits of a float (no NaN); -0 and 0 have the same.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

// A row's weights.  With c = 1 / T as a pair of floats, the exponent
//   t = (x - max) c
// is a pair (th, tl): the difference's rounding error is exact (two-sum), the
// product's too (fma).  With n the integer next to 1024 t / ln 2,
//   exp(t) = 2^(n/1024) exp(r),  r = t - n ln2/1024,  |r| <= 2^-11.5:
// a table gives 2^(j/1024) as a pair, exp(r) = 1 + r + r^2/2 + r^3/6 (r^4/24 is
// below 2^-50).  The product is rounded to a multiple of 2^-20 by adding 12 (an
// ulp there is 2^-20) and what is left of it to one of 2^-42 in the same way, so
// two integers come out of a float's bits without a conversion.  0.67 units off
// at most over 4 million samples (a half is the rounding), 0.28 in the mean
// square; 42 instructions.
struct Weights {
  float top, ch, cl;
  const float2* table;  // shared: 2^(j/1024) as a pair

  // th: the float next to t (monotone in x); the bins go by it
  __device__ __forceinline__ float coarse(float x) const { return __fmul_rn(x - top, ch); }

  __device__ __forceinline__ void exponent(float x, float& th, float& tl) const {
    const float s = x - top;
    const float bb = s - x;
    const float err = (x - (s - bb)) + (-top - bb);
    th = __fmul_rn(s, ch);
    tl = fmaf(s, cl, fmaf(err, ch, fmaf(s, ch, -th)));
  }

  // The weight is hi 2^22 + lo.  Returns th.
  __device__ __forceinline__ float parts(float x, int& hi, int& lo) const {
    float th, tl;
    exponent(x, th, tl);
    // 1.5 * 2^23: the sum's low bits are the integer; 127 * 1024: the exponent's bias
    const float magic = 12582912.f + 127 * 1024;
    const float fm = fmaf(th, kSteps, magic);
    const int bits = __float_as_int(fm);
    const float n = fm - magic;
    const float r = fmaf(n, -kStepHi, th);  // exact
    const float rl = fmaf(n, -kStepLo, tl);  // as large as r's last bits, or larger
    const float q = r + rl;
    const float y = fmaf(q * q, fmaf(q, 1.f / 6.f, 0.5f), rl - (q - r));
    const float2 f = table[bits & 1023];
    const float scale = __int_as_float((bits << 13) & 0xFF800000);  // 2^floor(n/1024)
    const float s1 = fmaf(f.x, q, f.x);
    const float e1 = fmaf(f.x, q, f.x - s1);
    const float low = fmaf(f.x, y, fmaf(f.y, q, f.y + e1));
    const float a = fmaf(s1, scale, 12.f);
    const float rem = fmaf(s1, scale, -(a - 12.f));
    const float b = fmaf(low, scale, rem) + 1.5f / 524288.f;
    const bool some = th > kLeast;  // not where the exponent is no number either (-inf times 0)
    hi = some ? __float_as_int(a) - __float_as_int(12.f) : 0;
    lo = some ? __float_as_int(b) - __float_as_int(1.5f / 524288.f) : 0;
    return th;
  }
  __device__ __forceinline__ u64 operator()(float x) const {
    int hi, lo;
    parts(x, hi, lo);
    return (u64)((long long)hi * (1 << 22) + lo);
  }
};

struct CountWeight {
  u64 w;
  int n;
};
__device__ __forceinline__ CountWeight operator+(const CountWeight& a, const CountWeight& b) {
  return {a.w + b.w, a.n + b.n};
}
__device__ __forceinline__ CountWeight scan_warp(CountWeight v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const CountWeight o{__shfl_up_sync(0xffffffffu, v.w, off), __shfl_up_sync(0xffffffffu, v.n, off)};
    if (lane >= off) v = v + o;
  }
  return v;
}

// The end of a prefix of the order: every logit of bits above key, and those
// of key itself up to index last.
struct Cut {
  uint32_t key;
  int last;
  __device__ __forceinline__ bool has(uint32_t k, int index) const {
    return k > key || (k == key && index <= last);
  }
};

// What a CTA shows the others of its cluster.
struct Shown {
  float top;         // its largest logit, and (greedy) the first index that has it
  int first, bad;
  uint32_t kmin[2], kmax[2];  // bits of a bin's values: for top-k and for top-p
  CountWeight before;
  int bin, bin_n;
  int ties;
  u64 kept, whole;   // of what is kept; of the row
  int few[2];        // values gathered (in the first CTA's lists)
  Cut cut;
  u64 weight;        // of the prefix up to the cut
};

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }


constexpr float kMostFinite = 3.402823466e38f;

template <typename T>
struct Row {
  cg::cluster_group cluster;
  const T* global;   // this CTA's part of the row
  const T* held;     // the same in shared memory, or null
  bool vector;       // `global` may be read four logits at a time
  uint32_t *hn, *hlo, *hhi;
  uint32_t* few_key; // [2][kFew]: for top-k and for top-p
  int* few_at;       // [2][kFew] index
  u64* few_w;        // [kFew]
  u64* seg_sum;      // [kSegments]
  Shown* shown;
  CountWeight* warp_sum;  // [32]
  float* queue;      // [64] this warp's, and the places
  int* queue_at;
  CountWeight bins[kBins / kThreads];  // this thread's of the whole cluster's
  float near_to;     // the first histogram's range
  bool safe;         // how the bins hold their sums, see put()
  bool infinite;     // the largest logit is +inf
  bool summed_up;    // `bins` are those of the first histogram, if that is there
  int rank, ranks, v0, size, seg;  // seg: logits of a segment, a multiple of 128
  Weights weight;

  __device__ Shown& peer(int r) { return *cluster.map_shared_rank(shown, r); }
  __device__ void sync() {
    if (ranks > 1)
      cluster.sync();
    else
      __syncthreads();
  }

  // Logits i .. i + 3 (i a multiple of 4), -inf past the part's end; all: there
  // are four.  Past pass 1, in a row that has +inf, it counts as the largest
  // finite number and all else as -inf: its weight is exp(-inf).
  __device__ __forceinline__ void load4(int i, float (&v)[4], bool all) const {
    T y[4];
    if (held) {
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(held + i);
      else
        *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(held + i);
    } else if (vector && (all || i + 4 <= size)) {
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<uint4*>(y) = __ldg(reinterpret_cast<const uint4*>(global + i));
      else
        *reinterpret_cast<uint2*>(y) = __ldg(reinterpret_cast<const uint2*>(global + i));
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] = global[min(i + k, size - 1)];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = to_float<T>(y[k]);
    if (!all) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = i + k < size ? v[k] : -INFINITY;
    }
    if (infinite) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = v[k] == INFINITY ? kMostFinite : -INFINITY;
    }
  }

  // f(i, four logits) over the CTA's part by whole warps, end(s) after each
  // segment: a warp takes every 16th segment, a lane four logits of 128, kAhead
  // loads in flight (one where each logit has much to do: two took 6 % longer).
  template <int kAhead, class F, class End>
  __device__ __forceinline__ void each(F f, End end) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int s = warp; s * seg < size; s += kNumWarps) {
      const int e = min((s + 1) * seg, size);
      for (int i0 = s * seg; i0 < e; i0 += 128 * kAhead) {
        float v[kAhead][4];
        if (i0 + 128 * kAhead <= e) {
#pragma unroll
          for (int k = 0; k < kAhead; ++k) load4(i0 + 128 * k + 4 * lane, v[k], true);
        } else {
#pragma unroll
          for (int k = 0; k < kAhead; ++k)
            if (i0 + 128 * k < e) load4(i0 + 128 * k + 4 * lane, v[k], false);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (i0 + 128 * k < e) f(i0 + 128 * k + 4 * lane, v[k]);
      }
      end(s);
    }
  }

  // Collects some lanes' logits (and their places) until a warp is full of them,
  // so that what is done with a few of many is done by whole warps.
  struct Queue {
    float* at;
    int* place;
    int n;
    template <class F>
    __device__ __forceinline__ void push(bool take, float v, int i, F f) {
      const unsigned who = __ballot_sync(0xffffffffu, take);
      if (who == 0) return;
      const int lane = threadIdx.x & 31;
      const int to = n + __popc(who & ((1u << lane) - 1));
      if (take) at[to] = v, place[to] = i;
      n += __popc(who);
      __syncwarp();
      if (n >= 32) {
        f(at[lane], place[lane]);
        n -= 32;
        const float rest = at[32 + lane];
        const int rest_at = place[32 + lane];
        __syncwarp();
        if (lane < n) at[lane] = rest, place[lane] = rest_at;
        __syncwarp();
      }
    }
    template <class F>
    __device__ __forceinline__ void flush(F f) {
      const int lane = threadIdx.x & 31;
      if (lane < n) f(at[lane], place[lane]);
      n = 0;
      __syncwarp();
    }
  };

  // A logit at or below which no exponent is above th (row values: a little
  // lower than the exact one).
  __device__ __forceinline__ float below(float th) const {
    const float d = -th / weight.ch;
    return weight.top - d - 2e-6f * (fabsf(weight.top) + d);
  }

  __device__ void clear() {
    for (int i = threadIdx.x; i < kBins; i += kThreads) hn[i] = hlo[i] = hhi[i] = 0;
    __syncthreads();
  }
  // A bin's count and 64-bit sum of weights.  The sums of hi (up to 2^20) and lo
  // (to +-2^21) by themselves, exact for up to kSafe values of a bin; or, safe,
  // in two words with the low one's carry to the high one, for any number.
  __device__ __forceinline__ void put(int bin, int hi, int lo) {
    atomicAdd(hn + bin, 1u);
    if (!safe) {
      atomicAdd(hhi + bin, (uint32_t)hi);
      atomicAdd(hlo + bin, (uint32_t)lo);
    } else {
      const u64 w = (u64)((long long)hi * (1 << 22) + lo);
      const uint32_t old = atomicAdd(hlo + bin, (uint32_t)w);
      const uint32_t up = (uint32_t)(w >> 32) + (old + (uint32_t)w < old ? 1u : 0u);
      if (up) atomicAdd(hhi + bin, up);
    }
  }

  // Finds the bin in which `before` plus the cluster's bins so far first reaches
  // the target.  kNever where none does (before is then the sum of all), kFull
  // where the sums may have overflowed; else before is what lies above the bin.
  // Every CTA sums up all bins for itself: one cluster barrier behind the
  // filling, and none for a second target.
  enum Crossing { kNever, kFound, kFull };
  __device__ Crossing cross(bool by_weight, u64 target, CountWeight& before, int& bin, int& bin_n, bool again = false) {
    constexpr int kPer = kBins / kThreads;
    static_assert(kPer == 4, "a thread reads 16 bytes of a histogram");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    CountWeight (&sum)[kPer] = bins, all{0, 0};
    int most = 0;
    if (!again) {
#pragma unroll
      for (int k = 0; k < kPer; ++k) sum[k] = {0, 0};
    }
#pragma unroll 2
    for (int r = again ? ranks : 0; r < ranks; ++r) {
      const uint4 n4 = reinterpret_cast<const uint4*>(cluster.map_shared_rank(hn, r))[tid];
      const uint4 l4 = reinterpret_cast<const uint4*>(cluster.map_shared_rank(hlo, r))[tid];
      const uint4 h4 = reinterpret_cast<const uint4*>(cluster.map_shared_rank(hhi, r))[tid];
      const uint32_t n[4] = {n4.x, n4.y, n4.z, n4.w}, lo[4] = {l4.x, l4.y, l4.z, l4.w}, hi[4] = {h4.x, h4.y, h4.z, h4.w};
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        sum[k] = sum[k] + CountWeight{safe ? ((u64)hi[k] << 32) + lo[k] : ((u64)hi[k] << 22) + (u64)(long long)(int)lo[k], (int)n[k]};
        most = max(most, (int)n[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) all = all + sum[k];
    const CountWeight in = scan_warp(all, lane);
    if (lane == 31) warp_sum[warp] = in;
    if (tid == 0) shown->bin = -1;
    const bool full = __syncthreads_or(!safe && most > kSafe);
    CountWeight c{before.w + in.w - all.w, before.n + in.n - all.n}, total = before;
    for (int k = 0; k < kNumWarps; ++k) {
      if (k < warp) c = c + warp_sum[k];
      total = total + warp_sum[k];
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const CountWeight next = c + sum[k];
      const u64 lo = by_weight ? c.w : (u64)c.n, hi = by_weight ? next.w : (u64)next.n;
      if (lo < target && hi >= target) {
        shown->before = c;
        shown->bin = kPer * tid + k;
        shown->bin_n = sum[k].n;
      }
      c = next;
    }
    __syncthreads();
    bin = shown->bin;
    bin_n = shown->bin_n;
    const CountWeight above = shown->before;
    __syncthreads();  // warp_sum and the result may be set again
    if (full) return kFull;
    if (bin < 0) {
      before = total;
      return kNever;
    }
    before = above;
    return kFound;
  }

  // The bins' range of exponents: (-to, -from].
  struct Range {
    float from, to;
    __device__ __forceinline__ bool has(float th) const { return th > -to && th <= -from; }
    __device__ __forceinline__ int bin(float th) const {  // rounded: monotone as well
      const float scale = kBins / (to - from), magic = 12582912.f;
      return min(max(__float_as_int(fmaf(-th - from, scale, magic)) - 0x4B400000, 0), kBins - 1);
    }
  };

  // Pass 2.  With `sum`, also this lane's sum of all weights.
  __device__ u64 fill(Range range, bool sum) {
    clear();
    long long all_hi = 0, all_lo = 0;
    int seg_hi = 0, seg_lo = 0;  // at most 32 of 2^20 and 2^21
    if (sum) {
      each<1>(
          [&](int, const float (&v)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              int hi, lo;
              const float th = weight.parts(v[k], hi, lo);
              seg_hi += hi;
              seg_lo += lo;
              if (range.has(th)) put(range.bin(th), hi, lo);
            }
          },
          [&](int) { all_hi += seg_hi, all_lo += seg_lo, seg_hi = seg_lo = 0; });
    } else {
      Queue q{queue, queue_at, 0};
      const float low = below(-range.to);
      auto bin = [&](float v, int) {
        int hi, lo;
        const float th = weight.parts(v, hi, lo);
        if (range.has(th)) put(range.bin(th), hi, lo);
      };
      each<1>(
          [&](int i, const float (&v)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) q.push(v[k] >= low, v[k], i + k, bin);
          },
          [](int) {});
      q.flush(bin);
    }
    return (u64)(all_hi * (1 << 22) + all_lo);
  }
  // The cluster's sum of v.
  __device__ u64 total_of(u64 v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    __syncthreads();
    if (lane == 0) warp_sum[warp].w = v;
    __syncthreads();
    if (threadIdx.x == 0) {
      v = 0;
      for (int w = 0; w < kNumWarps; ++w) v += warp_sum[w].w;
      shown->whole = v;
    }
    sync();
    v = 0;
    for (int r = 0; r < ranks; ++r) v += peer(r).whole;
    return v;
  }

  __device__ void store_segment(int s, int hi, int lo) {
    u64 v = (u64)((long long)hi * (1 << 22) + lo);
#pragma unroll
    for (int off = 16; off; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) seg_sum[s] = v;
  }

  // The segments' sums of what the cut keeps.
  __device__ void sum_kept(const Cut& cut) {
    int hi_sum = 0, lo_sum = 0;
    auto add = [&](float v, int) {
      int hi, lo;
      weight.parts(v, hi, lo);
      hi_sum += hi;
      lo_sum += lo;
    };
    if (cut.key == 0) {  // all: no need to collect them
      each<1>(
          [&](int, const float (&v)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) add(v[k], 0);
          },
          [&](int s) { store_segment(s, hi_sum, lo_sum), hi_sum = lo_sum = 0; });
      return;
    }
    Queue q{queue, queue_at, 0};
    each<1>(
        [&](int i, const float (&v)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) q.push(cut.has(key_of(v[k]), v0 + i + k), v[k], i + k, add);
        },
        [&](int s) { q.flush(add), store_segment(s, hi_sum, lo_sum), hi_sum = lo_sum = 0; });
  }

  // The shortest prefix of the order that has `target` elements, or weight:
  // its cut and weight.  near: the bins hold the first range (on return as
  // well).  With `sums`, the segments' sums of it (of what has bits least or
  // above) are taken on the way; summed says whether they could be.
  __device__ bool select(bool by_weight, u64 target, uint32_t least, bool sums, Cut& cut, u64& cut_weight,
                         bool& near, bool& summed) {
    CountWeight before{0, 0};
    int bin, bin_n;
    Range range{0.f, near_to};
    auto refill = [&](bool direct) {
      sync();  // every CTA has read the bins
      fill(range, direct);
      sync();
    };
    const bool again = near && summed_up;  // the sums of all bins are there from the last target
    if (!near) refill(false), near = true;
    Crossing got = cross(by_weight, target, before, bin, bin_n, again);
    summed_up = true;
    if (got == kFull) {
      safe = true;
      refill(false);
      got = cross(by_weight, target, before, bin, bin_n);
    }
    if (got == kNever) {  // below it: what is above are all of the first bins
      range = {near_to, -kLeast};
      refill(true);  // most logits lie there: they are not collected
      near = false;
      got = cross(by_weight, target, before, bin, bin_n);
      if (got == kFull) {
        safe = true;
        refill(true);
        got = cross(by_weight, target, before, bin, bin_n);
      }
      if (got == kNever) return false;
    }
    const bool few = bin_n <= kFew;
    sums &= few;
    // pass 3
    uint32_t kmin = 0xffffffffu, kmax = 0;
    Shown& lead = peer(0);
    const int which = by_weight ? 1 : 0;  // lists of their own: some CTA may still read the first
    uint32_t* my_key = few_key + which * kFew;
    int* my_at = few_at + which * kFew;
    uint32_t* list_key = cluster.map_shared_rank(my_key, 0);
    int* list_at = cluster.map_shared_rank(my_at, 0);
    int hi_sum = 0, lo_sum = 0;
    Queue q{queue, queue_at, 0};
    auto sort = [&](float v, int i) {
      const float th = weight.coarse(v);
      const int b = th > -range.from ? -1 : th > -range.to ? range.bin(th) : kBins;
      const uint32_t key = key_of(v);
      if (b == bin) {
        kmin = min(kmin, key);
        kmax = max(kmax, key);
        if (few) {
          const int n = atomicAdd(&lead.few[which], 1);
          list_key[n] = key;
          list_at[n] = v0 + i;
        }
      } else if (sums && b < bin && key >= least) {
        int hi, lo;
        weight.parts(v, hi, lo);
        hi_sum += hi;
        lo_sum += lo;
      }
    };
    // the bin's lower end, or the logit of bits least where that is higher
    const float low = below(-(range.from + (bin + 1) * ((range.to - range.from) / kBins)));
    each<1>(
        [&](int i, const float (&v)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) q.push(v[k] >= low, v[k], i + k, sort);
        },
        [&](int s) {
          if (sums) q.flush(sort), store_segment(s, hi_sum, lo_sum), hi_sum = lo_sum = 0;
        });
    q.flush(sort);
    if (few) {
      sync();  // the list is complete; every CTA works it out
      const int t = threadIdx.x;
      uint32_t key = 0;
      int at = 0;
      u64 w = 0;
      if (t < bin_n) {
        key = list_key[t];
        at = list_at[t];
        w = weight(of_key(key));
        if (rank) my_key[t] = key, my_at[t] = at;
        few_w[t] = w;
      }
      __syncthreads();
      if (t < bin_n) {
        CountWeight above = before;
        int same = 0, lower = 0;  // values equal to this, those of lower index
        for (int j = 0; j < bin_n; ++j) {
          const uint32_t k = my_key[j];
          if (k > key) above = above + CountWeight{few_w[j], 1};
          same += k == key;
          lower += k == key && my_at[j] < at;
        }
        const u64 lo = by_weight ? above.w : (u64)above.n;
        const u64 hi = by_weight ? above.w + same * w : (u64)above.n + same;
        if (lo < target && hi >= target) {  // the prefix ends among the values equal to this
          const u64 need = by_weight ? (target - lo + w - 1) / w : target - lo;
          if ((u64)lower + 1 == need) {
            shown->cut = {key, at};
            shown->weight = above.w + need * w;
          }
        }
      }
      __syncthreads();
      cut = shown->cut;
      cut_weight = shown->weight;
      if (sums) {  // the bin's kept values
        if (t < bin_n && key >= least && cut.has(key, at) && at >= v0 && at - v0 < size)
          atomicAdd(seg_sum + (at - v0) / seg, w);
        summed = true;
      }
      return true;
    }
    // many values: cut the range of bits until one is left.  (Bounds of their own,
    // as the lists: where the bin's values are all equal and top-k ends at the last
    // of them, no barrier stands between the reads here and top-p's.)
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (threadIdx.x == 0) shown->kmin[which] = 0xffffffffu, shown->kmax[which] = 0;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      atomicMin(&shown->kmin[which], kmin);
      atomicMax(&shown->kmax[which], kmax);
    }
    sync();
    for (int r = 0; r < ranks; ++r) {
      kmin = min(kmin, peer(r).kmin[which]);
      kmax = max(kmax, peer(r).kmax[which]);
    }
    while (kmin != kmax) {
      const uint32_t span = kmax - kmin;
      const int shift = max(0, 32 - __clz(span) - 11);
      sync();  // every CTA has read the bins
      clear();
      near = false;
      safe = true;
      each<1>(
          [&](int, const float (&v)[4]) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t key = key_of(v[k]);
              int hi, lo;
              if (key >= kmin && key <= kmax) weight.parts(v[k], hi, lo), put((int)((kmax - key) >> shift), hi, lo);
            }
          },
          [](int) {});
      sync();
      if (cross(by_weight, target, before, bin, bin_n) != kFound) return false;
      kmax -= (uint32_t)bin << shift;
      const uint32_t width = (1u << shift) - 1;
      kmin = kmax - kmin > width ? kmax - width : kmin;
    }
    const u64 w = weight(of_key(kmax));
    const u64 need = by_weight ? (target - before.w + w - 1) / w : target - (u64)before.n;
    cut = {kmax, need < (u64)bin_n ? index_of(kmax, (int)need) : 0x7fffffff};
    cut_weight = before.w + min(need, (u64)bin_n) * w;
    return true;
  }

  // The index of the n-th logit (from 1) of these bits.
  __device__ int index_of(uint32_t key, int n) {
    int count = 0;
    each<1>(
        [&](int, const float (&v)[4]) {
#pragma unroll
          for (int k = 0; k < 4; ++k) count += key_of(v[k]) == key;
        },
        [&](int s) {
          count = (int)__reduce_add_sync(0xffffffffu, (unsigned)count);
          if ((threadIdx.x & 31) == 0) seg_sum[s] = count;
          count = 0;
        });
    __syncthreads();
    if (threadIdx.x == 0) {
      int all = 0;
      for (int s = 0; s * seg < size; ++s) all += (int)seg_sum[s];
      shown->ties = all;
    }
    sync();
    for (int r = 0; r < rank; ++r) n -= peer(r).ties;
    const bool mine = n > 0 && n <= shown->ties;
    if (mine && threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int s = 0;
      for (; n > (int)seg_sum[s]; ++s) n -= (int)seg_sum[s];
      for (int i = s * seg + 4 * lane; n > 0; i += 128) {
        float v[4];
        load4(min(i, (size - 1) / 4 * 4), v, false);
        int c = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) c += i + k < size && key_of(v[k]) == key;
        int upto = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += o;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        if (upto >= n && upto - c < n) {
          int left = n - (upto - c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (i + k < size && key_of(v[k]) == key && --left == 0) shown->cut.last = v0 + i + k;
        }
        n -= all;
      }
    }
    if (threadIdx.x == 0) shown->bin = mine;
    sync();
    int at = 0x7fffffff;
    for (int r = 0; r < ranks; ++r)
      if (peer(r).bin) at = peer(r).cut.last;
    sync();
    return at;
  }
};

// kAlone: no more CTAs than SMs, and twice the registers, which hold all of a
// row's state.  (L2 flushed, launch included: a row of 32000 fp32 on four CTAs 42 us
// against 49 with the registers for two an SM, 100 rows of 50257 bf16 on one each 77
// against 91.  With more CTAs than SMs two an SM are as fast or faster: 256 rows of
// 50257 122 against 122, of 128000 on two each 238 against 274.)
template <typename T, bool kAlone>
__global__ void __launch_bounds__(kThreads, kAlone ? 1 : 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shown s_shown;
  __shared__ CountWeight s_warp[32];
  __shared__ float s_top[32];
  __shared__ int s_bad;
  __shared__ double s_c, s_least;  // 1 / T, T ln(min_p)
  __shared__ float s_queue[kNumWarps][64];
  __shared__ int s_queue_at[kNumWarps][64];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2* table = reinterpret_cast<float2*>(smem);
  u64* seg_sum = reinterpret_cast<u64*>(table + 1024);
  u64* few_w = seg_sum + kSegments;
  uint32_t* few_key = reinterpret_cast<uint32_t*>(few_w + kFew);
  int* few_at = reinterpret_cast<int*>(few_key + 2 * kFew);
  uint32_t* hist = reinterpret_cast<uint32_t*>(few_at + 2 * kFew);
  T* held = reinterpret_cast<T*>(hist + 3 * kBins);
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / ranks;
  const int v0 = min(rank * p.slice, p.vocab), size = min(p.slice, p.vocab - v0);
  const T* global = reinterpret_cast<const T*>(p.logits) + row * p.stride + v0;
  Row<T> R{cluster, global, nullptr, (reinterpret_cast<uintptr_t>(global) & (4 * sizeof(T) - 1)) == 0,
           hist, hist + kBins, hist + 2 * kBins, few_key, few_at, few_w, seg_sum, &s_shown, s_warp,
           s_queue[warp], s_queue_at[warp], {}, 0.f, false, false, false, rank, ranks, v0, size, 128 * ((p.slice + 128 * kSegments - 1) / (128 * kSegments)), {}};
  // segments of up to 512 logits, of fewer where a warp would have none
  R.seg = max(R.seg, min(512, 128 * ((p.slice + 128 * kNumWarps - 1) / (128 * kNumWarps))));
  const float temperature = p.temperature ? p.temperature[row] : p.temperature_all;
  const float min_p = p.min_p ? p.min_p[row] : p.min_p_all;
  if (tid == 0) {  // 64-bit arithmetic is slow here: once a CTA
    s_bad = 0;
    s_shown.few[0] = s_shown.few[1] = 0;
    s_c = 1.0 / (double)temperature;
    s_least = min_p > 0.f ? (double)temperature * log((double)fminf(min_p, 1.f)) : 0.0;
  }
  for (int j = tid; j < 1024; j += kThreads) {
    const u64 v = __umul64hi(kCoarse[j >> 5], kFine[j & 31]);  // units of 2^-60
    const float hi = (float)v;
    table[j] = make_float2(hi * 0x1p-60f, (float)(long long)(v - (u64)hi) * 0x1p-60f);
  }

  // ---- pass 1: the largest logit, and whether one is not a number
  float top = -INFINITY;
  bool nan = false;
  R.template each<4>(
      [&](int i, const float (&v)[4]) {
        if (p.held) {
          T y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = T(v[k]);  // exact: it came from a T
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<uint4*>(held + i) = *reinterpret_cast<const uint4*>(y);
          else
            *reinterpret_cast<uint2*>(held + i) = *reinterpret_cast<const uint2*>(y);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          nan |= v[k] != v[k];
          top = fmaxf(top, v[k]);
        }
      },
      [](int) {});
  if (p.held) R.held = held;
#pragma unroll
  for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  if (nan) s_bad = 1;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kNumWarps; ++w) top = fmaxf(top, s_top[w]);
    s_shown.top = top;
    s_shown.bad = s_bad;
  }
  R.sync();
  int bad = 0;
  top = -INFINITY;
  for (int r = 0; r < ranks; ++r) {
    bad |= R.peer(r).bad;
    top = fmaxf(top, R.peer(r).top);
  }
  int32_t* tokens = p.tokens + (long long)row * p.draws;
  float* logprobs = p.logprobs ? p.logprobs + (long long)row * p.draws : nullptr;
  const bool none = bad || top == -INFINITY;
  R.infinite = top == INFINITY;
  if (none || !(temperature > 0.f)) {  // nothing to draw from, or the first of the largest
    int first = 0x7fffffff;
    if (!none) {
      const float most = R.infinite ? kMostFinite : top;
      R.template each<4>(
          [&](int i, const float (&v)[4]) {
#pragma unroll
            for (int k = 3; k >= 0; --k)
              if (v[k] == most) first = min(first, v0 + i + k);
          },
          [](int) {});
    }
    first = __reduce_min_sync(0xffffffffu, first);
    if (tid == 0) s_shown.first = 0x7fffffff;
    __syncthreads();
    if (lane == 0) atomicMin(&s_shown.first, first);
    R.sync();
    for (int r = 0; r < ranks; ++r) first = min(first, R.peer(r).first);
    if (rank == 0)
      for (int j = tid; j < p.draws; j += kThreads) {
        tokens[j] = none ? -1 : first;
        if (logprobs) logprobs[j] = none ? NAN : 0.f;
      }
    R.sync();  // this CTA's words may still be read
    return;
  }
  top = fminf(top, kMostFinite);
  const double c = s_c;
  R.weight.top = top;
  R.weight.ch = fminf((float)c, kMostFinite);
  R.weight.cl = R.weight.ch == kMostFinite ? 0.f : (float)(c - (double)R.weight.ch);
  R.weight.table = table;

  // ---- the kept prefix of the order
  Cut cut{0, 0x7fffffff};  // everything
  if (min_p > 0.f && temperature < INFINITY) {
    // w >= min_p * w_max is x >= top + T ln(min_p): the least float that is
    float f = top;
    if (lane == 0) {
      const double least = (double)top + s_least;
      f = (float)least;
      if ((double)f < least) f = nextafterf(f, INFINITY);
      f += 0.f;
      if (isnan(f) || f > top) f = top;
    }
    f = __shfl_sync(0xffffffffu, f, 0);
    cut.key = key_of(f);
  }
  const uint32_t least = cut.key;
  auto shorten = [&](const Cut& o) {
    if (o.key > cut.key || (o.key == cut.key && o.last < cut.last)) cut = o;
  };
  const int top_k = p.top_k ? p.top_k[row] : p.top_k_all;
  const float top_p = p.top_p ? p.top_p[row] : p.top_p_all;
  const bool use_k = top_k > 0 && top_k < p.vocab, use_p = top_p < 1.f;
  bool summed = false;
  R.near_to = use_k ? kNearK : kNearP;
  if (use_k || use_p) {
    u64 total = R.fill({0.f, R.near_to}, !use_k);
    if (use_k)
      R.sync();  // every histogram is complete
    else
      total = R.total_of(total);  // as well
    bool near = true;
    Cut o;
    u64 w = 0;
    if (use_k && R.select(false, (u64)top_k, least, !use_p, o, w, near, summed)) shorten(o);
    if (use_p) {
      if (use_k && w == 0) {  // fewer than k have a weight: all of it counts
        R.summed_up = false;
        R.sync();
        total = R.total_of(R.fill({0.f, R.near_to}, true));
        near = true;
      }
      if (w) total = w;
      u64 want = 0;
      if (lane == 0) want = max((u64)ceil((double)fmaxf(top_p, 0.f) * (double)total), 1ull);
      want = __shfl_sync(0xffffffffu, want, 0);
      if (R.select(true, want, least, true, o, w, near, summed)) shorten(o);
    }
  }
  if (!summed) R.sum_kept(cut);
  __syncthreads();

  // ---- running sums over the segments
  u64 mine = tid < kSegments && tid * R.seg < size ? seg_sum[tid] : 0;
  const CountWeight upto = scan_warp({mine, 0}, lane);
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  u64 before = 0, cta = 0;
  for (int k = 0; k < kNumWarps; ++k) {
    if (k == warp) before = cta;
    cta += s_warp[k].w;
  }
  if (tid < kSegments) seg_sum[tid] = before + upto.w;  // up to and with segment tid
  if (tid == 0) s_shown.kept = cta;
  R.sync();
  u64 total = 0, start = 0;
  for (int r = 0; r < ranks; ++r) {
    if (r == rank) start = total;
    total += R.peer(r).kept;
  }

  // ---- the draws whose place lies in this CTA's part, a warp each
  const float whole = logf((float)((double)total * (1.0 / (double)kOne)));
  for (int j = warp; j < p.draws; j += kNumWarps) {
    const float u = p.u[(long long)row * p.draws + j];
    const double place = (u > 0.f ? fmin((double)u, 1.0) : 0.0) * (double)total;
    u64 target = min((u64)place, total - 1);
    if (target < start || target - start >= cta) continue;
    target -= start;
    int s = 0;  // segments that end at or before the target
#pragma unroll
    for (int k = 0; k < kSegments / 32; ++k) s += seg_sum[32 * k + lane] <= target;
    s = __reduce_add_sync(0xffffffffu, s);
    u64 at = s ? seg_sum[s - 1] : 0;
    const int end = min((s + 1) * R.seg, size);
    for (int i = s * R.seg + 4 * lane; i - 4 * lane < end; i += 128) {
      u64 w[4] = {0, 0, 0, 0}, sum = 0;
      float v[4];
      if (i < end) {
        R.load4(i, v, false);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (cut.has(key_of(v[k]), v0 + i + k)) w[k] = R.weight(v[k]);
          sum += w[k];
        }
      }
      const u64 with = at + scan_warp({sum, 0}, lane).w;
      const unsigned past = __ballot_sync(0xffffffffu, with > target);
      if (past) {
        if (lane == __ffs(past) - 1) {
          u64 c_i = with - sum;
          int hit = 3;
#pragma unroll
          for (int k = 3; k >= 0; --k) {  // the first k whose running sum passes the target
            u64 run = c_i;
#pragma unroll
            for (int q = 0; q < 4; ++q) run += q <= k ? w[q] : 0;
            if (run > target) hit = k;
          }
          const float x = hit == 0 ? v[0] : hit == 1 ? v[1] : hit == 2 ? v[2] : v[3];
          tokens[j] = v0 + i + hit;
          if (logprobs) {
            float th, tl;
            R.weight.exponent(x, th, tl);
            logprobs[j] = (th - whole) + tl;
          }
        }
        break;
      }
      at = __shfl_sync(0xffffffffu, with, 31);
    }
  }
  R.sync();  // this CTA's words may still be read
}

template <typename T, bool kAlone>
cudaError_t run(SampleParams p, int ranks, cudaStream_t s) {
  constexpr int kTables = 1024 * 8 + kSegments * 8 + kFew * 24 + 3 * kBins * 4;
  p.slice = ((p.vocab + ranks - 1) / ranks + 127) / 128 * 128;
  p.held = p.slice * sizeof(T) <= held_most<kAlone>;
  const size_t smem = kTables + (p.held ? p.slice * sizeof(T) : 0);
  // The limit is the kernel's, for all threads of the process: always the most
  // that any call asks for, not this call's, which would fail another's launch.
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T, kAlone>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kTables + held_most<kAlone>);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * ranks);
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
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, kAlone>, p);
}
template <typename T>
cudaError_t run(const SampleParams& p, int ranks, cudaStream_t s) {
  return (long long)p.rows * ranks <= p.num_sms ? run<T, true>(p, ranks, s) : run<T, false>(p, ranks, s);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, cudaStream_t s) {
  if (p.rows == 0 || p.draws == 0) return cudaSuccess;
  // Few rows: more CTAs a row, as long as each has an SM for itself.  (us on 1, 2, 4,
  // L2 flushed and launch included: a row of 32000 52, 45, 42; 8 of 128000 143, 85, 54;
  // 32 of 50257 76, 50, 42.  Two an SM: 64 of 50257 on four each 51 against 50, 76 of
  // 32000 71 against 48, 128 of 50257 on two each 74 against 74; faster where a part
  // does not fit shared memory, which this rule leaves: 150 of 128000 136 against 180.
  // So do 38 rows of 32000, whose clusters of four do not find all 152 SMs free: 60
  // against 49 on two each.)
  int ranks = 1;
  while (ranks < kMaxRanks && 2ll * p.rows * ranks <= p.num_sms && p.vocab / ranks > 4096) ranks *= 2;
  // Many rows: two a row where it is long, which evens out what the SMs have.  (On 1
  // and 2 each, fp32 with top-p / bf16 with all filters:
  //              160 rows              256 rows              1000 rows
  //    50257     106, 106 / 114, 106   121, 129 / 121, 121   317, 384 / 338, 363
  //    60000     129, 112 / 108, 100   135, 131 / 139, 121   352, 391 / 375, 375
  //    65537     138, 118 / 126, 122   148, 146 / 141, 151   392, 427 / 391, 451
  //    80000     161, 134 / 152, 136   174, 162 / 168, 164   450, 462 / 446, 495
  //   100000     189, 147 / 175, 157   215, 199 / 201, 205   589, 581 / 549, 599
  //   128000     204, 169 / 195, 174   272, 239 / 247, 233   716, 676 / 655, 670
  // The border follows the few hundred rows; it costs a thousand up to 18 %.)
  if (p.rows > p.num_sms && p.vocab > 65536) ranks = 2;
  if (p.dtype == kFp32) return run<float>(p, ranks, s);
  if (p.dtype == kBf16) return run<__nv_bfloat16>(p, ranks, s);
  return run<__half>(p, ranks, s);
}

}  // namespace ta
