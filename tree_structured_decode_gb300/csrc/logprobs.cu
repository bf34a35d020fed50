// Log probabilities of given tokens, entropy and the likeliest tokens of rows of
// logits (sm_103a), in one pass over them.
//
// With c = log2(e) / T, a thread's logits x, its largest so far m and t = (x - m) c:
//   S = sum 2^t,  H' = sum 2^t (-t),
// and where m grows by g / c, S becomes 2^-g S and H' 2^-g (H' + g S).  Threads
// are joined by the same rule, and
//   ln p_i = (x_i - max) / T - ln 2 log2 S,  entropy = ln 2 (log2 S + H' / S):
// no term is negative, so nothing cancels.  Sums are in 32 bits, a thread's of its
// own 1/128 or less of a row, then a tree.
//
// The likeliest k: a thread whose round's largest logit is above a threshold notes
// the round's logits in shared memory.  When many are noted, those of the k threads
// with the largest (no others can hold one) join a list of the k best so far, by
// all-with-all comparison, whose last is the next threshold.  The first threshold
// is taken from the lanes' largest.  Order is by (logit, index), one 64-bit key.
// (Logits put in the list one by one, where they are found: 70 us instead of 57 at
// 1664 rows of 50257 bf16, k = 8.)
//
// A row belongs to a CTA, or to a cluster of up to eight where rows are few; their
// sums and lists meet in the first one's shared memory.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "drafts.h"
#include "ptx.cuh"

namespace ta {
namespace {

namespace cg = cooperative_groups;
typedef unsigned long long u64;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLowest = -3.402823466e38f, kLargest = 3.402823466e38f;
constexpr float kNone = -200.f;  // 2^t of this or less counts as 0
constexpr int kMaxCluster = 8;

// Order-preserving bits of a float (no NaN); -0 and 0 have the same.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ u64 key_at(float x, int i) { return (u64)key_of(x) << 32 | (uint32_t)~i; }

__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <class T>
struct Type;
template <>
struct Type<float> {
  static constexpr int kVec = 4, kVectors = 4;  // elements of a 16-byte load, loads of a thread and round
  static constexpr uint32_t kNothing = 0xff800000u;  // -inf
  static __device__ __forceinline__ void split(uint32_t w, float* v) { v[0] = __uint_as_float(w); }
};
template <>
struct Type<__nv_bfloat16> {
  static constexpr int kVec = 8, kVectors = 2;
  static constexpr uint32_t kNothing = 0xff80ff80u;
  static __device__ __forceinline__ void split(uint32_t w, float* v) {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
};
template <>
struct Type<__half> {
  static constexpr int kVec = 8, kVectors = 2;
  static constexpr uint32_t kNothing = 0xfc00fc00u;
  static __device__ __forceinline__ void split(uint32_t w, float* v) {
    const float2 f = ptx::unpack_f16(w);
    v[0] = f.x, v[1] = f.y;
  }
};

struct Sums {
  float m, s, h;
};
// b's logits counted with a's.
__device__ __forceinline__ Sums joined(const Sums& a, const Sums& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float ga = fminf((m - a.m) * c, -kNone), gb = fminf((m - b.m) * c, -kNone);
  const float fa = ptx::ex2(-ga), fb = ptx::ex2(-gb);
  return Sums{m, fmaf(a.s, fa, b.s * fb), fmaf(fmaf(ga, a.s, a.h), fa, fmaf(gb, b.s, b.h) * fb)};
}
__device__ __forceinline__ Sums joined_warp(Sums x, float c) {
#pragma unroll
  for (int o = 16; o; o >>= 1)
    x = joined(x, Sums{__shfl_xor_sync(0xffffffffu, x.m, o), __shfl_xor_sync(0xffffffffu, x.s, o),
                       __shfl_xor_sync(0xffffffffu, x.h, o)}, c);
  return x;
}

// The likeliest so far, and what has come above them since.
template <int kThreads, int kGroup>
struct List {
  static constexpr int kRoom = kMaxTop + kMaxTop * kGroup;  // what is kept, and the logits of k threads
  // threads noted before the list is made anew (8: 60 us at 1664 rows, k = 8, and 91 at
  // 1216, k = 64; 32: 57 and 80; 64 takes 1 and 4 % more)
  static constexpr int kLook = 32;
  struct __align__(16) Noted {
    union {
      float x[kLook + kThreads][kGroup];  // (a round adds one a thread)
      u64 best[kMaxCluster * kMaxTop];    // selected ones, when the logits have been looked at
    };
    u64 most[kLook + kThreads];         // the largest of them
    int index[kLook + kThreads];        // of the first of them
    int n;
  } noted;
  u64 key[kRoom];
  // Keys up to it are left out: one less than a key that k are known to reach, so that
  // the logit of (threshold + 1) is that key's, whatever its index.  0: fewer are known.
  u64 threshold;
  int n;
};

// The k largest of from[0..n) to to[0..k), in order (0 where there are fewer).
template <int kThreads>
__device__ __forceinline__ void select_largest(const u64* from, int n, u64* to, int k) {
  for (int i = threadIdx.x; i < k; i += kThreads)
    if (i >= n) to[i] = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const u64 mine = from[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += from[j] > mine;
    if (rank < k) to[rank] = mine;
  }
}

// The noted threads' logits join the list.
template <int kThreads, int kVec, int kGroup>
__device__ __forceinline__ void add_noted(List<kThreads, kGroup>& s, int k) {
  const int tid = threadIdx.x, n = s.noted.n;
  const auto index = [&](int from, int e) {
    return s.noted.index[from] + (e / kVec) * (kThreads * kVec) + e % kVec;
  };
  for (int i = tid; i < n; i += kThreads) {
    float most = s.noted.x[i][0];
    int first = 0;
#pragma unroll
    for (int e = 1; e < kGroup; ++e)
      if (s.noted.x[i][e] > most) most = s.noted.x[i][e], first = e;
    s.noted.most[i] = key_at(most, index(i, first));
  }
  __syncthreads();
  if (n > k) {  // the k-th of the threads' largest is reached by k logits, and by k threads only
    for (int i = tid; i < n; i += kThreads) {
      const u64 mine = s.noted.most[i];
      int above = 0;
      for (int j = 0; j < n; ++j) above += s.noted.most[j] > mine;
      if (above == k - 1 && mine - 1 > s.threshold) s.threshold = mine - 1;
    }
    __syncthreads();
  }
  const u64 low = s.threshold;
  for (int i = tid; i < n * kGroup; i += kThreads) {
    const int from = i / kGroup, e = i % kGroup;
    if (s.noted.most[from] <= low) continue;
    const float x = s.noted.x[from][e];
    const u64 key = key_at(x, index(from, e));
    if (x > -INFINITY && key > low) s.key[atomicAdd(&s.n, 1)] = key;
  }
  __syncthreads();
  const int have = s.n;
  if (have > k) {
    select_largest<kThreads>(s.key, have, s.noted.best, k);
    __syncthreads();
    for (int i = tid; i < k; i += kThreads) s.key[i] = s.noted.best[i];
    // (the k-th itself does not come again)
    if (tid == 0) s.n = k, s.threshold = s.noted.best[k - 1] - 1;
  }
  if (tid == 0) s.noted.n = 0;
  __syncthreads();
}

template <class T, int kThreads, bool kTop>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) scores_kernel(const ScoreParams p) {
  constexpr int kVec = Type<T>::kVec, kVectors = Type<T>::kVectors, kGroup = kVectors * kVec;
  constexpr int kWarps = kThreads / 32, kRound = kVectors * kThreads;
  using Keys = List<kThreads, kGroup>;
  __shared__ Keys s_list;
  __shared__ Sums s_sums[kWarps], s_rank[kMaxCluster];
  __shared__ uint32_t s_mth[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / ranks;
  const T* row = static_cast<const T*>(p.logits) + r * p.stride;
  const float heat = p.temperature ? p.temperature[r] : p.temperature_all;
  const bool greedy = !(heat > 0.f);
  const float inv = greedy ? 1.f : 1.f / heat;
  // (finite, and not 0: -inf stays below everything; the least there is, so that a
  // temperature of +inf weighs all other logits alike)
  const float c = fminf(fmaxf(inv * kLog2e, 1.40129846e-45f), kLargest);
  const int k = kTop ? (greedy ? max(p.top, 1) : p.top) : 0;

  // the row as 16-byte vectors; `shift` elements of the first lie before it
  const int shift = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  const T* base = row - shift;
  const int vectors = (shift + p.vocab + kVec - 1) / kVec, per = (vectors + ranks - 1) / ranks;
  const int v0 = min(rank * per, vectors), v1 = min(v0 + per, vectors);
  auto load = [&](int at, uint4 (&x)[kVectors]) {
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const int v = at + u * kThreads + tid;
      const int i0 = v * kVec - shift;
      if (v < v1 && i0 >= 0 && i0 + kVec <= p.vocab) {
        x[u] = load16(base + (long long)v * kVec);
      } else {
        uint32_t w[4] = {Type<T>::kNothing, Type<T>::kNothing, Type<T>::kNothing, Type<T>::kNothing};
        if (v < v1) {
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            if (i0 + e < 0 || i0 + e >= p.vocab) continue;
            if constexpr (sizeof(T) == 4) {
              w[e] = reinterpret_cast<const uint32_t*>(row)[i0 + e];
            } else {
              const uint32_t h = reinterpret_cast<const uint16_t*>(row)[i0 + e];
              w[e / 2] = e & 1 ? (w[e / 2] & 0xffffu) | h << 16 : (w[e / 2] & 0xffff0000u) | h;
            }
          }
        }
        x[u] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };

  // a given token's logit, asked for now
  const auto given_at = [&](int g) {
    const int i = p.given[(long long)r * p.n_given + g];
    return i >= 0 && i < p.vocab ? i : -1;
  };
  const int given_i = rank == 0 && tid < p.n_given ? given_at(tid) : -1;
  const float given_x = given_i >= 0 ? (float)row[given_i] : 0.f;

  if (kTop) {
    if (tid == 0) s_list.n = 0, s_list.threshold = 0, s_list.noted.n = 0;
    __syncthreads();
  }
  Sums sum{kLowest, 0.f, 0.f};
  const uint64_t c2 = ptx::f2(c, c);
  uint4 ahead[kVectors];
  load(v0, ahead);
  // (shared memory of another CTA may be written once that CTA has started: waited
  // for where the row's sums go to the first one, so that it costs no time here)
  if (ranks > 1) ptx::cluster_arrive();
  for (int at = v0; at < v1; at += kRound) {
    float x[kGroup];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
      const uint32_t w[4] = {ahead[u].x, ahead[u].y, ahead[u].z, ahead[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) Type<T>::split(w[e], x + u * kVec + e * (kVec / 4));
    }
    if (at + kRound < v1) load(at + kRound, ahead);
    float most = x[0];
#pragma unroll
    for (int e = 1; e + 1 < kGroup; e += 2) most = ptx::max3(most, x[e], x[e + 1]);
    most = fmaxf(most, x[kGroup - 1]);
    if (most > sum.m) {
      const float g = fminf((most - sum.m) * c, -kNone), f = ptx::ex2(-g);
      sum.h = fmaf(g, sum.s, sum.h) * f;
      sum.s *= f;
      sum.m = most;
    }
    {
      const uint64_t low = ptx::f2(-sum.m, -sum.m);
      uint64_t s2[2] = {0ull, 0ull}, h2[2] = {0ull, 0ull};
#pragma unroll
      for (int e = 0; e < kGroup; e += 2) {
        float t0, t1;
        ptx::f2_split(ptx::fma_f32x2(ptx::add_f32x2(ptx::f2(x[e], x[e + 1]), low), c2, 0ull), t0, t1);
        t0 = max_nan(t0, kNone), t1 = max_nan(t1, kNone);
        const uint64_t w = ptx::f2(ptx::ex2(t0), ptx::ex2(t1));
        s2[e / 2 & 1] = ptx::add_f32x2(s2[e / 2 & 1], w);
        h2[e / 2 & 1] = ptx::fma_f32x2(w, ptx::f2(t0, t1), h2[e / 2 & 1]);
      }
      float a, b;
      ptx::f2_split(ptx::add_f32x2(s2[0], s2[1]), a, b);
      sum.s += a + b;
      ptx::f2_split(ptx::add_f32x2(h2[0], h2[1]), a, b);
      sum.h -= a + b;
    }
    if (kTop && k > 0) {
      u64 low = s_list.threshold;
      const bool open = !low;
      if (open) {  // of each warp's lanes the m-th largest, of these the least, has k threads' largest at or above it
        uint32_t left = key_of(most), mth = 0;
        for (int m = (k + kWarps - 1) / kWarps; m > 0; --m) {
          mth = __reduce_max_sync(0xffffffffu, left);
          if (lane == __ffs(__ballot_sync(0xffffffffu, left == mth)) - 1) left = 0;
        }
        if (lane == 0) s_mth[warp] = mth;
        __syncthreads();
        mth = s_mth[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mth = min(mth, s_mth[w]);
        if (of_key(mth) > -INFINITY) {
          low = ((u64)mth << 32) - 1;
          if (tid == 0) s_list.threshold = low;  // (read again behind a barrier)
        }
      }
      // (what equals the k-th of earlier rounds comes behind it)
      const float least = low ? of_key((uint32_t)((low + 1) >> 32)) : kLowest;
      bool many = open;
      if (open ? most >= least : most > least) {
        const int to = atomicAdd(&s_list.noted.n, 1);
        s_list.noted.index[to] = (at + tid) * kVec - shift;
#pragma unroll
        for (int e = 0; e < kGroup; e += 4)
          *reinterpret_cast<float4*>(s_list.noted.x[to] + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        many |= to + 1 >= Keys::kLook;
      }
      if (__syncthreads_or(many || at + kRound >= v1)) add_noted<kThreads, kVec, kGroup>(s_list, k);
    }
  }

  // ---- the row's sums and list
  sum = joined_warp(sum, c);
  if (lane == 0) s_sums[warp] = sum;
  __syncthreads();
  if (ranks > 1) ptx::cluster_wait();
  if (warp == 0) {
    Sums x = lane < kWarps ? s_sums[lane] : Sums{kLowest, 0.f, 0.f};
    x = joined_warp(x, c);
    if (lane == 0) *cluster.map_shared_rank(&s_rank[rank], 0) = x;
  }
  if (kTop) {
    __syncthreads();
    select_largest<kThreads>(s_list.key, s_list.n, s_list.noted.best, k);
    __syncthreads();
    if (ranks > 1) {  // (the first one's keys are its own list's until all have been ranked)
      u64* to = cluster.map_shared_rank(s_list.key, 0);
      cluster.sync();
      for (int i = tid; i < k; i += kThreads) to[rank * k + i] = s_list.noted.best[i];
    }
  }
  if (ranks > 1)
    cluster.sync();
  else
    __syncthreads();
  if (rank) return;
  if (kTop && ranks > 1) {
    select_largest<kThreads>(s_list.key, ranks * k, s_list.noted.best, k);
  }
  Sums all = s_rank[0];
  for (int i = 1; i < ranks; ++i) all = joined(all, s_rank[i], c);
  int broken = !(all.s > 0.f);  // nothing above -inf
  int infinite = 0;             // +inf shares the row
  if (all.s != all.s) {
    int nan = 0;
    for (int i = tid; i < p.vocab; i += kThreads) {
      const float x = (float)row[i];
      nan |= x != x;
      infinite += x == INFINITY;
    }
    broken = __syncthreads_or(nan);
#pragma unroll
    for (int o = 16; o; o >>= 1) infinite += __shfl_xor_sync(0xffffffffu, infinite, o);
    if (lane == 0) s_sums[warp].s = (float)infinite;
    __syncthreads();
    infinite = 0;
    for (int w = 0; w < kWarps; ++w) infinite += (int)s_sums[w].s;
  }
  __syncthreads();
  if (infinite) all = Sums{INFINITY, (float)infinite, 0.f};
  const int first = kTop ? (int)~(uint32_t)s_list.noted.best[0] : 0;
  const float log_s = greedy ? 0.f : log2f(all.s) * kLn2;
  const auto logprob = [&](float x, int i) {
    if (broken) return NAN;
    if (greedy) return i == first ? 0.f : -INFINITY;
    const float y = x - all.m;
    return (x == all.m ? 0.f : y > -INFINITY ? y * inv : -INFINITY) - log_s;  // (inv may be 0)
  };
  if (tid == 0 && p.entropy) p.entropy[r] = broken ? NAN : greedy ? 0.f : fmaf(all.h / all.s, kLn2, log_s);
  for (int g = tid; g < p.n_given; g += kThreads) {
    const int i = g == tid ? given_i : given_at(g);
    p.given_logprobs[(long long)r * p.n_given + g] = i < 0 ? NAN : logprob(g == tid ? given_x : (float)row[i], i);
  }
  if (kTop)
    for (int e = tid; e < p.top; e += kThreads) {
      const u64 key = s_list.noted.best[e];
      const long long to = (long long)r * p.top + e;
      p.top_tokens[to] = broken || !key ? -1 : (int)~(uint32_t)key;
      p.top_logprobs[to] = broken ? NAN : key ? logprob(of_key((uint32_t)(key >> 32)), (int)~(uint32_t)key) : -INFINITY;
    }
}

template <class T, int kThreads>
cudaError_t run(const ScoreParams& p, bool top, int ranks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
  return top ? cudaLaunchKernelEx(&cfg, scores_kernel<T, kThreads, true>, p)
             : cudaLaunchKernelEx(&cfg, scores_kernel<T, kThreads, false>, p);
}

template <class T>
cudaError_t pick(const ScoreParams& p, cudaStream_t s) {
  // a row whose temperature is not above 0 needs its largest logit's place
  const bool top = p.top > 0 || p.temperature || !(p.temperature_all > 0.f);
  const long long bytes = (long long)p.vocab * sizeof(T);
  // Half the threads where rows are short, or too many for all their CTAs of 256 to be
  // on the SMs at once: 900 rows of 50257 bf16 with 8 alternatives take 32 us (with 256
  // threads 37), 1664 58 (61), with 64 110 (108), 2048 rows of 128000 fp32 151 (158),
  // with 8 172 (174); 272 rows of 28510, all at once either way, 18 (13).  (64 threads:
  // 1664 rows 56, but 900 46 and with 64 alternatives 161.)
  if (bytes <= 8192 || p.rows > 4 * p.num_sms) return run<T, 128>(p, top, 1, s);
  // Few rows are split while that leaves at most three parts an SM and the parts are
  // long: one row of 32000 fp32 takes 6.3 us in eight (whole 11.1), 100 of 50257 bf16
  // 11.9 in four (in two 13.3, whole 14.7), 225 of 128000 fp32 27.8 in two (whole 35.8);
  // with more parts, 150 of 128000 fp32 28.5 in four (in two 22.6), 250 of 50257 bf16
  // 17.3 in two (whole 16.7).
  int ranks = 1;
  while (ranks < kMaxCluster && (long long)p.rows * ranks * 2 <= 3 * p.num_sms && bytes / ranks > 16384) ranks *= 2;
  return run<T, 256>(p, top, ranks, s);
}

}  // namespace

cudaError_t launch_token_logprobs(const ScoreParams& p, cudaStream_t s) {
  if (p.dtype == kFp32) return pick<float>(p, s);
  return p.dtype == kFp16 ? pick<__half>(p, s) : pick<__nv_bfloat16>(p, s);
}

}  // namespace ta
