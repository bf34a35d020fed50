// Sampling with temperature, top-k, top-p and min-p from given random numbers
// (sm_103a).
//
// The token of a row is a comparison of running sums with u times their total,
// so a sum that is off in its last bits gives another token.  The weights are
// therefore whole numbers,
//   w_i = round(2^42 exp((l_i - max) / T)),
// computed to about that last unit, and every sum of them is exact: the result
// does not depend on the order or the grid, and agrees with 64-bit arithmetic
// except where u lies within about 2^-42 of a border.
//
// A cluster of up to eight CTAs holds a row in shared memory, so that logits are
// read from DRAM once; the passes over them work there, and what the CTAs have
// to tell one another goes through distributed shared memory.
//   top-k / top-p   a prefix of the order (logit descending, index ascending).
//                   One histogram over the exponent of the weight (2048 bins of
//                   1/128 of a power of two, and a second for what is below
//                   2^-16) gives the bin in which it ends.  A bin of one value
//                   is done; the values of a small one are compared all with
//                   all by one CTA; a large one is cut further by the float's
//                   bits until one value is left.
//   min-p           a least logit.
//   draw            per-warp sums in index order, their scan, and one walk
//                   through the 32-element groups of the warp that holds u S.
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
constexpr int kSlice = 16384;      // two CTAs fit an SM: one loads while the other computes
constexpr int kFew = 256;          // values of a bin that are compared all with all
constexpr float kNear = 16.f;      // the first histogram's range of exponents
constexpr int kMaxRanks = 8;
constexpr u64 kOne = 1ull << 42;   // the weight of the largest logit
constexpr float kLeast = -44.f;    // below 2^-44 a weight rounds to 0

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
constexpr float kLn2Hi = 0x1.62e4300000000p-1f, kLn2Lo = -0x1.05c6100000000p-29f;  // ln 2 = hi + lo to 2^-50

// Order-preserving bits of a float (no NaN, no -0).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}

// A row's weights.  With c = log2(e) / T as a pair of floats, the exponent
//   t = (x - max) c
// is a pair (th, tl): the difference's rounding error is exact (two-sum), the
// product's too (fma).  2^t = 2^e 2^(j/1024) 2^r with |r| <= 2^-11: the table
// gives the second factor as a pair, 2^r = 1 + q + q^2/2 + q^3/6 with q = r ln 2
// as a pair; q^4/24 is below 2^-50.  The product is rounded to a multiple of
// 2^-20 by adding 12 (an ulp there is 2^-20) and what is left of it to one of
// 2^-42 in the same way, so two integers come out of a float's bits without a
// conversion: 0.67 units off at most over 4 million samples (a half is the
// rounding), 0.29 in the mean square.
struct Weights {
  float top, ch, cl;
  const float2* table;  // shared: 2^(j/1024) as a pair

  // th: the float next to t (monotone in x); the bins go by it
  __device__ __forceinline__ float coarse(float x) const { return x == top ? 0.f : __fmul_rn(x - top, ch); }

  __device__ __forceinline__ void exponent(float x, float& th, float& tl) const {
    const float s = x - top;
    const float bb = s - x;
    const float err = (x - (s - bb)) + (-top - bb);
    th = __fmul_rn(s, ch);
    tl = fmaf(s, ch, -th) + fmaf(s, cl, err * ch);
  }

  // The weight is hi 2^22 + lo.  Returns th.
  __device__ __forceinline__ float parts(float x, int& hi, int& lo) const {
    float th, tl;
    exponent(x, th, tl);
    const float magic = 12582912.f;  // 1.5 * 2^23: the sum's low bits are the rounded integer
    const float fm = fmaf(th, 1024.f, magic);
    const int bits = __float_as_int(fm);
    const float r = fmaf(fm - magic, -1.f / 1024.f, th);  // exact
    const float qh = __fmul_rn(r, kLn2Hi);  // not contracted: its error is added below
    const float ql = fmaf(r, kLn2Hi, -qh) + fmaf(r, kLn2Lo, tl * kLn2Hi);
    const float q = qh + ql;  // tl may be as large as r's last bits
    const float y = fmaf(q * q, fmaf(q, 1.f / 6.f, 0.5f), ql - (q - qh));
    const float2 f = table[bits & 1023];
    const float scale = __int_as_float(0x3F800000 + ((bits << 13) & 0xFF800000));  // 2^e
    const float p = __fmul_rn(f.x, q);
    const float low = fmaf(f.y, q, fmaf(f.x, y, fmaf(f.x, q, -p))) + f.y;
    const float s1 = __fadd_rn(f.x, p);
    const float e1 = p - (s1 - f.x);
    const float a = fmaf(s1, scale, 12.f);
    const float rem = fmaf(s1, scale, -(a - 12.f));
    const float b = fmaf(e1 + low, scale, rem) + 1.5f / 524288.f;
    hi = __float_as_int(a) - __float_as_int(12.f);
    lo = __float_as_int(b) - __float_as_int(1.5f / 524288.f);
    const bool some = th > kLeast;  // not where the exponent is no number either (-inf times 0)
    if (!some) hi = lo = 0;
    if (x == top) hi = 1 << 20, lo = 0, th = 0.f;
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

// The end of a prefix of the order: every logit above key (weight above), then
// the first m of those at key, each of weight w.
struct Cut {
  uint32_t key;
  int m;
  u64 above, w;
};

// What a CTA shows the others of its cluster.
struct Shown {
  float top;         // its largest logit, and the first index that has it
  int first, bad;
  uint32_t kmin, kmax;
  CountWeight total; // of the bins that it sums up
  CountWeight before;
  int bin, bin_n;
  int ties;          // final pass
  u64 kept;
  int few;           // values gathered (in the first CTA's list)
  Cut cut;
};

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float<__half>(__half v) { return __half2float(v); }

template <typename T>
struct Row {
  const SampleParams& p;
  cg::cluster_group cluster;
  float* x;          // this CTA's logits
  uint32_t *hn, *hlo, *hhi;
  uint32_t* few_key; // [kFew]
  u64* few_w;        // [kFew]
  Shown* shown;
  CountWeight* warp_sum;  // [32]
  int rank, ranks, v0, size;
  Weights weight;

  __device__ Shown& peer(int r) { return *cluster.map_shared_rank(shown, r); }

  __device__ void clear() {
    for (int i = threadIdx.x; i < kBins; i += kThreads) hn[i] = hlo[i] = hhi[i] = 0;
    __syncthreads();
  }
  // A 64-bit sum in two 32-bit words: the low word's carry goes to the high
  // one, so the pair is exact whatever the order of the additions.
  __device__ void put(int bin, u64 w) {
    atomicAdd(hn + bin, 1u);
    const uint32_t lo = (uint32_t)w;
    const uint32_t old = atomicAdd(hlo + bin, lo);
    const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
    if (hi) atomicAdd(hhi + bin, hi);
  }

  // Sums the cluster's histograms, each CTA a share of the bins, and finds the
  // bin in which `before` plus the bins so far first reaches the target.
  // Returns false where it never does; else before is what lies above the bin.
  __device__ bool cross(bool by_weight, u64 target, CountWeight& before, int& bin, int& bin_n) {
    cluster.sync();  // every histogram is complete
    const int share = kBins / ranks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (share + kThreads - 1) / kThreads;  // bins of a thread: 1, 2 or 4
    const int first = rank * share + threadIdx.x * per;
    const bool mine = (int)threadIdx.x * per < share;
    CountWeight sum[4], all{0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = {0, 0};
    if (mine) {
      for (int r = 0; r < ranks; ++r) {
        const uint32_t *n = cluster.map_shared_rank(hn, r), *lo = cluster.map_shared_rank(hlo, r),
                       *hi = cluster.map_shared_rank(hhi, r);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < per)
            sum[k] = sum[k] + CountWeight{((u64)hi[first + k] << 32) + lo[first + k], (int)n[first + k]};
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) all = all + sum[k];
    }
    CountWeight in = scan_warp(all, lane);
    if (lane == 31) warp_sum[warp] = in;
    __syncthreads();
    CountWeight at{in.w - all.w, in.n - all.n}, total{0, 0};
    for (int k = 0; k < kNumWarps; ++k) {
      if (k == warp) at = at + total;
      total = total + warp_sum[k];
    }
    if (threadIdx.x == 0) shown->total = total;
    cluster.sync();
    int owner = -1;
    CountWeight sofar = before;
    for (int r = 0; r < ranks; ++r) {
      const CountWeight next = sofar + peer(r).total;
      if ((by_weight ? next.w : (u64)next.n) >= target) {
        owner = r;
        break;
      }
      sofar = next;
    }
    if (owner == rank && mine) {
      CountWeight c = sofar + at;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < per) {
          const CountWeight next = c + sum[k];
          const u64 lo = by_weight ? c.w : (u64)c.n, hi = by_weight ? next.w : (u64)next.n;
          if (lo < target && hi >= target) {
            shown->before = c;
            shown->bin = first + k;
            shown->bin_n = sum[k].n;
          }
          c = next;
        }
    }
    cluster.sync();
    if (owner < 0) return false;
    before = peer(owner).before;
    bin = peer(owner).bin;
    bin_n = peer(owner).bin_n;
    return true;
  }

  // The part of the row whose exponent lies in (-to, -from], in the bins.  With
  // `sum`, also this lane's sum of all weights.
  __device__ u64 fill(float from, float to, bool sum) {
    clear();
    const float scale = kBins / (to - from);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int c0, c1;
    chunk(warp, c0, c1);
    int all_hi = 0, all_lo = 0;  // at most 64 of 2^20 and 2^21
    for (int i = c0 + lane; i < c1; i += 32) {
      const float v = x[i];
      if (!sum && !(weight.coarse(v) > -to)) continue;
      int hi, lo;
      const float th = weight.parts(v, hi, lo);
      all_hi += hi;
      all_lo += lo;
      if (th > -to && th <= -from)
        put(min((int)((-th - from) * scale), kBins - 1), (u64)((long long)hi * (1 << 22) + lo));
    }
    return (u64)((long long)all_hi * (1 << 22) + all_lo);
  }

  // A warp's share of the CTA's logits.
  __device__ void chunk(int warp, int& c0, int& c1) const {
    const int n = ((size + kThreads - 1) / kThreads) * 32;
    c0 = min(warp * n, size);
    c1 = min(c0 + n, size);
  }

  // The shortest prefix of the order that has `target` elements, or weight.
  // near: the bins hold the part up to kNear; they do again on return, or
  // near is false.
  __device__ bool select(bool by_weight, u64 target, Cut& cut, bool& near) {
    CountWeight before{0, 0};
    int bin, bin_n;
    float from = 0.f, to = kNear;
    if (!near) fill(from, to, false), near = true;
    if (!cross(by_weight, target, before, bin, bin_n)) {
      // below it: what is above are all of the first bins
      for (int r = 0; r < ranks; ++r) before = before + peer(r).total;
      from = kNear, to = -kLeast;
      cluster.sync();
      fill(from, to, false);
      near = false;
      if (!cross(by_weight, target, before, bin, bin_n)) return false;
    }
    // the values in that bin
    const float scale = kBins / (to - from);
    uint32_t kmin = 0xffffffffu, kmax = 0;
    Shown& lead = peer(0);
    uint32_t* list = cluster.map_shared_rank(few_key, 0);
    for (int i = threadIdx.x; i < size; i += kThreads) {
      const float th = weight.coarse(x[i]);
      if (th > -to && th <= -from && min((int)((-th - from) * scale), kBins - 1) == bin) {
        const uint32_t k = key_of(x[i]);
        kmin = min(kmin, k);
        kmax = max(kmax, k);
        if (bin_n <= kFew) list[atomicAdd(&lead.few, 1)] = k;
      }
    }
    kmin = __reduce_min_sync(0xffffffffu, kmin);
    kmax = __reduce_max_sync(0xffffffffu, kmax);
    if (threadIdx.x == 0) shown->kmin = 0xffffffffu, shown->kmax = 0;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
      atomicMin(&shown->kmin, kmin);
      atomicMax(&shown->kmax, kmax);
    }
    cluster.sync();
    for (int r = 0; r < ranks; ++r) {
      kmin = min(kmin, peer(r).kmin);
      kmax = max(kmax, peer(r).kmax);
    }
    if (kmin != kmax && bin_n <= kFew) {
      if (rank == 0) {
        if ((int)threadIdx.x < bin_n) few_w[threadIdx.x] = weight(of_key(few_key[threadIdx.x]));
        __syncthreads();
        if ((int)threadIdx.x < bin_n) {
          const uint32_t key = few_key[threadIdx.x];
          CountWeight above = before;
          int same = 0;
          for (int j = 0; j < bin_n; ++j) {
            if (few_key[j] > key) above = above + CountWeight{few_w[j], 1};
            same += few_key[j] == key;
          }
          const u64 w = few_w[threadIdx.x];
          const u64 lo = by_weight ? above.w : (u64)above.n;
          const u64 hi = by_weight ? above.w + same * w : (u64)above.n + same;
          if (lo < target && hi >= target)  // one value: its threads write the same
            shown->cut = end_at(by_weight, target, key, above, same, w);
        }
        if (threadIdx.x == 0) shown->few = 0;
      }
      cluster.sync();
      cut = lead.cut;
      return true;
    }
    if (rank == 0 && threadIdx.x == 0) shown->few = 0;
    while (kmin != kmax) {
      const uint32_t span = kmax - kmin;
      const int shift = max(0, 32 - __clz(span) - 11);
      clear();
      near = false;
      for (int i = threadIdx.x; i < size; i += kThreads) {
        const uint32_t k = key_of(x[i]);
        if (k >= kmin && k <= kmax) put((int)((kmax - k) >> shift), weight(x[i]));
      }
      if (!cross(by_weight, target, before, bin, bin_n)) return false;
      kmax -= (uint32_t)bin << shift;
      const uint32_t width = (1u << shift) - 1;
      kmin = kmax - kmin > width ? kmax - width : kmin;
    }
    cut = end_at(by_weight, target, kmax, before, bin_n, weight(of_key(kmax)));
    return true;
  }

  __device__ static Cut end_at(bool by_weight, u64 target, uint32_t key, const CountWeight& above,
                               int same, u64 w) {
    const u64 need = by_weight ? (target - above.w + w - 1) / w : target - (u64)above.n;
    return {key, (int)min(need, (u64)same), above.w, w};
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Shown s_shown;
  __shared__ CountWeight s_warp[32];
  __shared__ float s_top[32];
  __shared__ int s_first[32], s_bad;
  __shared__ double s_c, s_least;  // log2(e) / T, T ln(min_p)
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float2* table = reinterpret_cast<float2*>(smem);
  uint32_t* hist = reinterpret_cast<uint32_t*>(table + 1024);
  u64* few_w = reinterpret_cast<u64*>(hist + 3 * kBins);
  uint32_t* few_key = reinterpret_cast<uint32_t*>(few_w + kFew);
  float* x = reinterpret_cast<float*>(few_key + kFew);
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / ranks;
  const int v0 = min(rank * p.slice, p.vocab), size = min(p.slice, p.vocab - v0);
  Row<T> R{p, cluster, x, hist, hist + kBins, hist + 2 * kBins, few_key, few_w, &s_shown, s_warp, rank, ranks, v0, size, {}};
  const float temperature = p.temperature ? p.temperature[row] : p.temperature_all;
  const float min_p = p.min_p ? p.min_p[row] : p.min_p_all;
  if (tid == 0) {  // 64-bit arithmetic is slow here: once a CTA
    s_bad = 0;
    s_shown.few = 0;
    s_c = 1.4426950408889634074 / (double)temperature;
    s_least = min_p > 0.f ? (double)temperature * log((double)fminf(min_p, 1.f)) : 0.0;
  }
  for (int j = tid; j < 1024; j += kThreads) {
    const u64 v = __umul64hi(kCoarse[j >> 5], kFine[j & 31]);  // units of 2^-60
    const float hi = (float)v;
    table[j] = make_float2(hi * 0x1p-60f, (float)(long long)(v - (u64)hi) * 0x1p-60f);
  }

  // ---- the logits, their largest, and whether one is not a number
  const T* src = reinterpret_cast<const T*>(p.logits) + row * p.stride + v0;
  float top = -INFINITY;
  int first = p.vocab;
  bool nan = false;
  auto take = [&](int i, T y) {
    const float v = to_float<T>(y) + 0.f;  // -0 becomes 0: equal logits have equal bits
    x[i] = v;
    nan |= v != v;
    if (v > top) top = v, first = v0 + i;
  };
  constexpr int kVec = 16 / sizeof(T);
  int done = 0;
  if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {  // 16 bytes a load, four in flight
    done = size / kVec * kVec;
    for (int i0 = tid * kVec; i0 < done; i0 += 4 * kThreads * kVec) {
      uint4 raw[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i0 + k * kThreads * kVec < done)
          raw[k] = __ldg(reinterpret_cast<const uint4*>(src + i0 + k * kThreads * kVec));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i0 + k * kThreads * kVec < done) {
          T y[kVec];
          memcpy(y, &raw[k], 16);
#pragma unroll
          for (int j = 0; j < kVec; ++j) take(i0 + k * kThreads * kVec + j, y[j]);
        }
    }
  }
  for (int i0 = done + tid; i0 < size; i0 += 8 * kThreads) {
    T y[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i0 + k * kThreads < size) y[k] = src[i0 + k * kThreads];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i0 + k * kThreads < size) take(i0 + k * kThreads, y[k]);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, top, off);
    const int f = __shfl_xor_sync(0xffffffffu, first, off);
    if (o > top || (o == top && f < first)) top = o, first = f;
  }
  if (lane == 0) s_top[warp] = top, s_first[warp] = first;
  __syncthreads();
  if (nan) s_bad = 1;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kNumWarps; ++w)
      if (s_top[w] > top || (s_top[w] == top && s_first[w] < first)) top = s_top[w], first = s_first[w];
    s_shown.top = top;
    s_shown.first = first;
    s_shown.bad = s_bad;
  }
  cluster.sync();
  int bad = 0;
  top = -INFINITY;
  first = p.vocab;
  for (int r = 0; r < ranks; ++r) {
    const Shown& o = R.peer(r);
    bad |= o.bad;
    if (o.top > top || (o.top == top && o.first < first)) top = o.top, first = o.first;
  }
  int32_t* tokens = p.tokens + (long long)row * p.draws;
  float* logprobs = p.logprobs ? p.logprobs + (long long)row * p.draws : nullptr;
  const bool none = bad || top == -INFINITY;
  if (none || !(temperature > 0.f)) {  // nothing to draw from, or the largest
    if (rank == 0)
      for (int j = tid; j < p.draws; j += kThreads) {
        tokens[j] = none ? -1 : first;
        if (logprobs) logprobs[j] = none ? NAN : 0.f;
      }
    cluster.sync();  // this CTA's words may still be read
    return;
  }
  const double c = s_c;
  R.weight.top = top;
  R.weight.ch = (float)c;
  R.weight.cl = isinf(R.weight.ch) ? 0.f : (float)(c - (double)R.weight.ch);
  R.weight.table = table;

  // ---- the kept prefix of the order
  Cut cut{0, 0x7fffffff, 0, 0};  // everything
  const int top_k = p.top_k ? p.top_k[row] : p.top_k_all;
  const float top_p = p.top_p ? p.top_p[row] : p.top_p_all;
  auto shorten = [&](const Cut& o) {
    if (o.key > cut.key || (o.key == cut.key && o.m < cut.m)) cut = o;
  };
  const bool use_k = top_k > 0 && top_k < p.vocab, use_p = top_p < 1.f;
  if (use_k || use_p) {
    // one pass: the bins, and with top-p alone the whole row's weight
    u64 sum = R.fill(0.f, kNear, !use_k);
    bool near = true;
    if (!use_k) {
#pragma unroll
      for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) s_warp[warp].w = sum;
      __syncthreads();
      if (tid == 0) {
        sum = 0;
        for (int w = 0; w < kNumWarps; ++w) sum += s_warp[w].w;
        s_shown.kept = sum;
      }
      __syncthreads();
    }
    u64 total = 0;
    Cut o;
    if (use_k) {
      if (R.select(false, (u64)top_k, o, near)) shorten(o), total = o.above + (u64)o.m * o.w;
    }
    if (use_p) {
      cluster.sync();
      if (use_k && total == 0) {  // fewer than k have a weight: all of it counts
        sum = R.fill(0.f, kNear, true);
        near = true;
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) s_warp[warp].w = sum;
        __syncthreads();
        if (tid == 0) {
          sum = 0;
          for (int w = 0; w < kNumWarps; ++w) sum += s_warp[w].w;
          s_shown.kept = sum;
        }
        cluster.sync();
      }
      if (total == 0)
        for (int r = 0; r < ranks; ++r) total += R.peer(r).kept;
      u64 want = 0;
      if (lane == 0) want = max((u64)ceil((double)fmaxf(top_p, 0.f) * (double)total), 1ull);
      want = __shfl_sync(0xffffffffu, want, 0);
      if (R.select(true, want, o, near)) shorten(o);
    }
  }
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
    shorten({key_of(f), 0x7fffffff, 0, 0});
  }

  // ---- sums of the kept weights, warp by warp in index order
  int c0, c1;
  R.chunk(warp, c0, c1);
  int hi_sum = 0, lo_sum = 0, ties = 0;
  for (int i = c0 + lane; i < c1; i += 32) {
    const uint32_t k = key_of(x[i]);
    if (k > cut.key) {
      int hi, lo;
      R.weight.parts(x[i], hi, lo);
      hi_sum += hi;
      lo_sum += lo;
    }
    ties += k == cut.key;
  }
  u64 sum = (u64)((long long)hi_sum * (1 << 22) + lo_sum);
  const float tie_x = of_key(cut.key);
  const u64 w_tie = tie_x == tie_x ? R.weight(tie_x) : 0;
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    ties += __shfl_xor_sync(0xffffffffu, ties, off);
  }
  if (lane == 0) s_warp[warp] = {sum, ties};
  __syncthreads();
  int ties_before = 0, all_ties = 0;
  for (int w = 0; w < kNumWarps; ++w) {
    if (w == warp) ties_before = all_ties;
    all_ties += s_warp[w].n;
  }
  if (tid == 0) s_shown.ties = all_ties;
  cluster.sync();
  int cta_ties = 0;
  for (int r = 0; r < rank; ++r) cta_ties += R.peer(r).ties;
  auto kept_of = [&](int before, int n) { return max(0, min(n, cut.m - before)); };
  u64 before = 0, cta = 0, own = 0;
  {
    int t = cta_ties;
    for (int w = 0; w < kNumWarps; ++w) {
      const u64 s = s_warp[w].w + (u64)kept_of(t, s_warp[w].n) * w_tie;
      if (w == warp) before = cta, own = s;
      cta += s;
      t += s_warp[w].n;
    }
  }
  if (tid == 0) s_shown.kept = cta;
  cluster.sync();
  u64 total = 0;
  for (int r = 0; r < ranks; ++r) {
    if (r == rank) before += total;
    total += R.peer(r).kept;
  }
  ties_before += cta_ties;

  // ---- the draws whose place lies in this warp's part
  if (own > 0) {
    const float whole = log2f((float)((double)total * (1.0 / (double)kOne)));
    for (int j = 0; j < p.draws; ++j) {
      const float u = p.u[(long long)row * p.draws + j];
      const double place = (u > 0.f ? fmin((double)u, 1.0) : 0.0) * (double)total;
      const u64 target = min((u64)place, total - 1);
      if (target < before || target - before >= own) continue;
      u64 at = before;
      int tie = ties_before;
      for (int i0 = c0; i0 < c1; i0 += 32) {
        const int i = i0 + lane;
        u64 w = 0;
        bool is_tie = false;
        if (i < c1) {
          const uint32_t k = key_of(x[i]);
          if (k > cut.key) w = R.weight(x[i]);
          is_tie = k == cut.key;
        }
        const unsigned t = __ballot_sync(0xffffffffu, is_tie);
        if (is_tie && tie + __popc(t & ((1u << lane) - 1)) < cut.m) w = w_tie;
        tie += __popc(t);
        const u64 c_i = at + scan_warp({w, 0}, lane).w;
        const unsigned past = __ballot_sync(0xffffffffu, c_i > target);
        if (past) {
          if (lane == __ffs(past) - 1) {
            tokens[j] = v0 + i;
            if (logprobs) {
              float th = 0.f, tl = 0.f;
              if (x[i] != R.weight.top) R.weight.exponent(x[i], th, tl);
              logprobs[j] = ((th - whole) + tl) * kLn2Hi;
            }
          }
          break;
        }
        at = __shfl_sync(0xffffffffu, c_i, 31);
      }
    }
  }
  cluster.sync();  // this CTA's words may still be read
}

template <typename T>
cudaError_t run(SampleParams p, int ranks, cudaStream_t s) {
  p.slice = ((p.vocab + ranks - 1) / ranks + 31) / 32 * 32;
  const size_t smem = 1024 * 8 + 3 * kBins * 4 + kFew * 12 + (size_t)p.slice * 4;
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
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
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace

cudaError_t launch_sample(const SampleParams& p, cudaStream_t s) {
  if (p.rows == 0 || p.draws == 0) return cudaSuccess;
  int ranks = 1;
  while (ranks < kMaxRanks && (p.vocab + ranks - 1) / ranks > kSlice) ranks *= 2;
  // few rows: more CTAs a row while SMs are free
  while (ranks < kMaxRanks && (long long)p.rows * ranks * 2 <= p.num_sms && p.vocab / ranks > 2048) ranks *= 2;
  if (p.dtype == kFp32) return run<float>(p, ranks, s);
  if (p.dtype == kBf16) return run<__nv_bfloat16>(p, ranks, s);
  return run<__half>(p, ranks, s);
}

}  // namespace ta
