// Acceptance of drafts against sampled target tokens: temperature, top-k,
// top-p and min-p from given random numbers.
//
// The order of a row's tokens (largest logit first, equal logits by lowest
// index) makes top-k and top-p prefixes of one order, so no row is sorted: a
// prefix is a threshold key (the logit's ordered bits) and the number of tokens
// with exactly that key that belong to it.  The weights are whole numbers (32
// bits of exp), their sums exact in 64 bits, so atomics and any split of the row
// give the same sums, and the drawn token does not depend on either.
//
// sample_kernel: a cluster of 1 to 8 blocks per verify row.  Each block stages
//   its slice of the row in shared memory (the logits are read from HBM once)
//   and keeps the maximum of each thread's elements.
//   - a small top_k: the k-th largest thread maximum is a bound that at least k
//     tokens reach, and few more do.  Those are appended to one list in the first
//     block, which sorts it and finishes alone: no other pass over the row.
//   - otherwise (or if more tokens than a list holds reach the bound): a histogram
//     of weight sums (top-p) or counts (a large top_k) over kBins equal steps of the
//     logit below the maximum finds the step that holds the prefix' end, and
//     8-bit digits of the keys inside that step find the key.  Equal steps, not
//     the keys' own leading digits, spread the bulk of the logits over the bins,
//     so few lanes of a warp add to the same one.  The kept weights are then
//     summed in index order and the draw located.
//   Bound by instructions and by the chain of steps between cluster barriers, not by
//   HBM.  Rows of 151936 bf16, 64 of them (19.4 MB, 2.9 us of HBM): greedy 10 us, a small
//   top_k 18, weights without a filter 34 (exp of every token, twice), top-p 63 (and the
//   shared-memory atomics of the histogram), a large top_k 68.  One row of 32000 in 32
//   bits: 4, 9, 8, 17 and 29.  Of a row with a small top_k (12 us of the call's 18) the
//   slices take 3.4 us, the bound 2.3, the list 3.5, the first block's two sorts, two
//   scans and draw 2.7.
// accept_kernel: one warp per request; where there are no drafts (R = 1) the rows'
//   blocks write the accept lengths, 0, themselves.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdnhybrid.h"

namespace gdnsample {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
constexpr int kList = kThreads;  // candidates that the first block can hold, a thread each
constexpr int kMaxSlice = 49152;  // elements a block stages: 192 KB in 32 bits; sums of 16-bit halves fit 32 bits
static_assert(kMaxSlice * kMaxCluster == GDN_SAMPLE_MAX_V, "a row is staged by one cluster");
static_assert(kThreads == 256, "a digit, and a word of a sorted list, is a thread");
constexpr int kScratch = 2048;  // words: the thread maxima, a histogram, or the list and its sort
static_assert(kMaxCluster * kThreads <= kScratch && 2 * kBins <= kScratch && 2 * (kList + 2 * kThreads) <= kScratch, "each fits");

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

using u64 = unsigned long long;

// bits that order as the values do; 0 for NaN, which takes no part.  -0 equals +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return x != x ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// a row's weights: w = exp((l - max) / T), and W = rint(2^31 w) as a whole number
struct Weight {
  float top, inv_t;
  __device__ float w(float x) const { return x == top ? 1.f : expf((x - top) * inv_t); }
  __device__ uint32_t whole(float x) const { return __float2uint_rn(w(x) * 2147483648.f); }
};

__device__ __forceinline__ u64 shift_mul(u64 total, u64 frac) {
  return (total >> 24) * frac + (((total & 0xffffff) * frac) >> 24);
}

// floor(x * 2^24) of x clamped to [0, most]; NaN as 0
__device__ __forceinline__ u64 fraction(float x, float most) { return (u64)(fminf(fmaxf(x, 0.f), most) * 16777216.f); }

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
  return v;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void put(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void put(uint32_t at, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t get(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint4 get4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t add_at(uint32_t at, uint32_t v) {
  uint32_t old;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(at), "r"(v) : "memory");
  return old;
}
__device__ __forceinline__ void min_at(uint32_t at, uint32_t v) {
  asm volatile("red.shared::cluster.min.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// kN equal steps of the distance from the largest logit, a monotonous map whatever the range: adding 2^23 rounds to a
// whole number without a conversion (those, like exp, run at a quarter of the rate of additions).  A distance of NaN
// (both infinite) is 0, and so is every distance where the range is infinite.
template <int kN>
struct Steps {
  float scale;
  __device__ explicit Steps(float range) : scale(fminf(kN / range, 3e38f)) {}
  __device__ int of(float distance) const {
    const float s = fminf(fmaxf(distance * scale, 0.f), (float)(kN - 1));
    return (int)(__float_as_uint(s + 8388608.f) & (2 * kN - 1));
  }
};

struct Ends {
  uint32_t most, least;
  int count;
};
// the block's largest and smallest word and its count's sum
__device__ __forceinline__ Ends block_ends(uint32_t most, uint32_t least, int count, u64* part) {
  const uint32_t m = __reduce_max_sync(kFull, most), l = __reduce_min_sync(kFull, least);
  const int c = __reduce_add_sync(kFull, count);
  Ends* const words = reinterpret_cast<Ends*>(part);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = {m, l, c};
  __syncthreads();
  Ends e = {0, 0xffffffffu, 0};
  for (int w = 0; w < kWarps; ++w) {
    e.most = max(e.most, words[w].most);
    e.least = min(e.least, words[w].least);
    e.count += words[w].count;
  }
  return e;
}

// inclusive prefix over the block's threads
__device__ __forceinline__ u64 block_scan(u64 v, u64* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 o = __shfl_up_sync(kFull, v, off);
    if (lane >= off) v += o;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) v += part[w];
  __syncthreads();
  return v;
}

template <typename T>
struct Unit {  // the elements of 16 bytes
  static constexpr int kN = 16 / sizeof(T);
  float x[kN];
  __device__ explicit Unit(const uint4& w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      } else {
        x[i] = __uint_as_float(u[i]);
      }
    }
  }
};

struct News {  // what the first block tells the others
  u64 left;
  uint32_t top_key, bound, low, digit;  // low: the smallest thread maximum
};

// Descending order of kWords (a power of two up to kThreads) words, one a thread: neighbours up to 16 apart compare by
// shuffles, others through `places` (two halves in turn, one barrier each).
template <int kWords>
__device__ __forceinline__ u64 sort_descending(u64 v, u64* places) {
  const int tid = threadIdx.x;
  int half = 0;
#pragma unroll
  for (int k = 2; k <= kWords; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) {
      u64 other;
      if (j < 32) {
        other = __shfl_xor_sync(kFull, v, j);
      } else {
        places[half * kThreads + tid] = v;
        __syncthreads();
        other = places[half * kThreads + (tid ^ j)];
        half ^= 1;
      }
      const bool larger = ((tid & j) == 0) == ((tid & k) == 0);
      v = (other > v) == larger ? other : v;
    }
  }
  return v;
}

__device__ __forceinline__ u64 sort_descending(u64 v, int n, u64* places) {
  return n <= 64 ? sort_descending<64>(v, places) : n <= 128 ? sort_descending<128>(v, places) : sort_descending<256>(v, places);
}

// The rest of a row whose m candidates (key << 32 | ~index, in any order) lie in `list`; the first c of them in order are
// the top-k tokens.  A candidate is a thread's, sorted twice (by logit for the prefixes, by index for the draw).
__device__ __forceinline__ void finish(const gdn_sample_args& p, size_t at, const u64* list, u64* places, int m, int c,
                                              float top_p, float floor_w, u64 u, const Weight& weight, u64* part) {
  __shared__ u64 total_s;
  __shared__ uint32_t drawn_s;
  const int tid = threadIdx.x;
  const u64 word = sort_descending(tid < m ? list[tid] : 0, m, places);
  const float w = tid < c ? weight.w(of_key(word >> 32)) : 0.f;
  const uint32_t W = __float2uint_rn(w * 2147483648.f);
  u64 upto = block_scan(W, part);
  if (tid == kThreads - 1) total_s = upto;
  __syncthreads();
  const u64 limit = top_p < 1.f ? shift_mul(total_s, fraction(top_p, 1.f)) : ~0ull;
  const bool kept = tid < c && (upto - W < limit || tid == 0) && w >= floor_w;
  const u64 by_index = sort_descending(kept ? word << 32 | W : 0, m, places);
  const uint32_t V = (uint32_t)by_index;
  upto = block_scan(V, part);  // its first barrier is behind every read of total_s
  if (tid == kThreads - 1) total_s = upto;
  __syncthreads();
  const u64 drawn = shift_mul(total_s, u);
  if (upto - V <= drawn && drawn < upto) drawn_s = (uint32_t)(by_index >> 32);
  __syncthreads();
  if (kept && (uint32_t)word == drawn_s) {
    p.target[at] = (int)~drawn_s;
    if (p.prob) p.prob[at] = w * 2147483648.f / (float)total_s;
  }
}

struct Place {  // a block's kept weight above the threshold, and its tokens on it
  u64 sum, equal;
};

// kPerSm: blocks an SM holds at least, by registers.  Six instead of four hide more of the others' waits where the call has
// more blocks than fit, but the fewer registers spill: 1152 rows of 50001 with a top-k take 88 us, with four 101; 64 rows
// of 151936 (512 blocks) take 17.8 with four, 18.5 with six.
template <typename T, int kPerSm>
__global__ void __launch_bounds__(kThreads, kPerSm) sample_kernel(const gdn_sample_args p, int blocks, int slice_units) {
  constexpr int kN = Unit<T>::kN;
  extern __shared__ uint4 slice[];                      // [slice_units], then the scratch below
  uint32_t* const scratch = reinterpret_cast<uint32_t*>(slice + slice_units);
  u64* const list = reinterpret_cast<u64*>(scratch);     // [kList], and twice as many words behind it for the sort
  uint32_t* const lo = scratch;                          // [kBins] sums of the weights' low halves
  uint32_t* const hi = scratch + kBins;                  // [kBins] and high halves
  uint32_t* const maxima = scratch;                      // [blocks][kThreads]
  __shared__ u64 part[2 * kWarps];
  __shared__ News news;
  __shared__ Place places[kMaxCluster], warps[kWarps];
  __shared__ uint32_t count, lowest, all_s, digits[256];
  __shared__ u64 total_s, ranges[kMaxCluster];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int t = blockIdx.x / blocks, b = blockIdx.y;
  pdl_wait();
  pdl_trigger();
  const int n = p.n_rows[b];
  if (t == 0 && rank == 0 && tid == 0) {
    if ((n < 0 || n > p.R) && p.status) atomicOr(p.status, GDN_STATUS_BAD_NROWS);
    if (p.R == 1 && p.accept_len) p.accept_len[b] = 0;
  }
  if (n <= 0 || n > p.R || t >= n) return;  // the whole cluster
  cluster_arrive();  // every block of the cluster runs before any writes to another's shared memory
  const size_t at = (size_t)b * p.R + t;
  const T* const row = static_cast<const T*>(p.logits) + at * p.row_stride;
  const float temp = p.temperature ? p.temperature[b] : 1.f;
  const int k = p.top_k ? p.top_k[b] : 0;
  const float top_p = p.top_p ? p.top_p[b] : 1.f, min_p = p.min_p ? p.min_p[b] : 0.f;
  const u64 u = fraction(p.u[at], 1.f - 1.f / 16777216.f);

  // stage the slice in units of 16 aligned bytes; what is not of the row is NaN
  const int shift = (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
  const int units = (p.V + shift + kN - 1) / kN, per = (units + blocks - 1) / blocks;
  const int u0 = min(units, (int)rank * per), own = min(units, u0 + per) - u0;
  const int first = u0 * kN - shift;  // the row's index of the slice's first element
  const uint4* const src = reinterpret_cast<const uint4*>(row - shift) + u0;
  float top = __uint_as_float(0x7fffffffu);  // NaN: no element yet
  for (int i = tid; i < own; i += kThreads) {
    const int e = first + i * kN;
    if (e >= 0 && e + kN <= p.V) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(slice + i)), "l"(src + i) : "memory");
    } else {
      T x[kN];
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        if constexpr (sizeof(T) == 2) x[c] = e + c >= 0 && e + c < p.V ? row[e + c] : __ushort_as_bfloat16(0x7fff);
        else x[c] = e + c >= 0 && e + c < p.V ? row[e + c] : __uint_as_float(0x7fffffffu);
      }
      slice[i] = *reinterpret_cast<uint4*>(x);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // a thread reads only what it copied itself, so far
#pragma unroll 4
  for (int i = tid; i < own; i += kThreads) {
    const Unit<T> x(slice[i]);
#pragma unroll
    for (int c = 0; c < kN; ++c) top = fmaxf(top, x.x[c]);  // NaN loses
  }
  cluster_wait();
  put(peer(maxima + rank * kThreads + tid, 0), key_of(top));
  if (tid == 0) {
    count = 0;
    lowest = 0xffffffffu;
  }
  cluster_sync();

  // the first block: the row's largest key, and for a top_k that a list can hold a bound just under the k-th largest
  // thread maximum
  // How many tokens reach the bound: about k + k^2 / 2n with n thread maxima, if the order is random.  A list that
  // would overflow costs its pass for nothing.  (64 rows of 151936, k = 200: 21 us, without a list 72.)
  const int n_threads = min(blocks * kThreads, units);
  const bool listed = k > 0 && k < p.V && temp > 0.f && (p.V <= kList || k + k * (int64_t)k / n_threads <= kList - kList / 16);
  if (rank == 0) {
    uint32_t mine[kMaxCluster], best = 0, low = 0xffffffffu;
    int n_maxima = 0;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
      mine[r] = r < blocks ? maxima[r * kThreads + tid] : 0;
      best = max(best, mine[r]);
      if (mine[r] != 0) low = min(low, mine[r]);
      n_maxima += mine[r] != 0;
    }
    digits[tid] = 0;
    const auto ends = block_ends(best, low, n_maxima, part);
    best = ends.most;
    low = ends.least;
    uint32_t bound = 1;  // every key but NaN's: fewer maxima than k
    if (listed && ends.count >= k) {
      // the maxima in 256 equal steps between the ends (the keys' leading digits would be the same few for most of them):
      // the k-th largest lies in the first step that k of them reach
      const float best_x = of_key(best);
      const Steps<256> steps(best_x - of_key(low));
      auto step_of = [&](uint32_t key) { return steps.of(best_x - of_key(key)); };
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (mine[r] != 0) atomicAdd(&digits[step_of(mine[r])], 1u);
      __syncthreads();
      const uint32_t here = digits[tid], upto = (uint32_t)block_scan(here, part);
      if (upto - here < (uint32_t)k && (uint32_t)k <= upto) all_s = tid;
      __syncthreads();
      const int last = (int)all_s;
      uint32_t least = 0xffffffffu;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (mine[r] != 0 && step_of(mine[r]) <= last) least = min(least, mine[r]);
      bound = block_ends(0, least, 0, part).least;
    }
    if (tid < blocks) {
      put(peer(&news.top_key, tid), best);
      put(peer(&news.bound, tid), bound);
      put(peer(&news.low, tid), low);
    }
  }
  cluster_sync();
  const uint32_t top_key = news.top_key;
  const float peak = of_key(top_key);

  if (!(temp > 0.f) || top_key == 0) {  // greedy, or a row of NaN alone
    if (top_key != 0) {
      uint32_t mine = 0xffffffffu;
      for (int i = tid; i < own; i += kThreads) {
        const Unit<T> x(slice[i]);
#pragma unroll
        for (int c = kN - 1; c >= 0; --c)
          if (x.x[c] == peak) mine = min(mine, (uint32_t)(first + i * kN + c));
      }
      mine = __reduce_min_sync(kFull, mine);
      if (lane == 0 && mine != 0xffffffffu) min_at(peer(&lowest, 0), mine);
    }
    cluster_sync();
    if (rank == 0 && tid == 0) {
      p.target[at] = top_key == 0 ? 0 : (int)lowest;
      if (p.prob) p.prob[at] = 1.f;
    }
    return;
  }
  const Weight weight{peak, 1.f / temp};
  const float floor_w = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;

  if (listed) {
    const float bound = of_key(news.bound);
    const bool every = news.bound == 1;
    const uint32_t counter = peer(&count, 0), to = peer(list, 0);
    for (int i = tid; i < own; i += kThreads) {
      const Unit<T> x(slice[i]);
#pragma unroll
      for (int c = 0; c < kN; ++c)
        if (x.x[c] >= bound || (every && x.x[c] == x.x[c])) {
          const uint32_t place = add_at(counter, 1u);
          if (place < kList) put(to + place * 8, (u64)key_of(x.x[c]) << 32 | (uint32_t)~(first + i * kN + c));
        }
    }
    cluster_sync();
    const int found = (int)get(counter);
    if (found <= kList) {
      if (rank != 0) return;
      finish(p, at, list, list + kList, found, min(k, found), top_p, floor_w, u, weight, part);
      cluster_sync();  // the others have read `count`, or have left
      return;
    }
    cluster_sync();  // the list's place is the histogram's
  }

  // ---- the general way.  kept: keys above thr, and the first `ties` tokens (by index) of key thr
  uint32_t thr = 1;
  u64 ties = ~0ull;
  auto narrow = [&](bool weights, float range, u64 want) {
    // the new threshold: the prefix of the kept tokens whose counts, or weights, reach `want` (for weights: that
    // share of their sum)
    const Steps<kBins> steps(range);
    const bool edged = ties != ~0ull;
    const float edge_x = edged ? of_key(thr) : -INFINITY;
    auto within = [&](float x) { return edged ? x > edge_x : x >= edge_x; };  // not NaN; the tied tokens apart
    auto bin_of = [&](float x) { return steps.of(peak - x); };
    auto add = [&](float x, int i) {
      const uint32_t v = weights ? weight.whole(x) : 1u;
      if (v & 0xffff) atomicAdd(&lo[i], v & 0xffff);
      if (v >> 16) atomicAdd(&hi[i], v >> 16);
    };
    const u64 edge = edged ? ties * (weights ? weight.whole(of_key(thr)) : 1u) : 0;  // tokens of key thr, not swept
    const int edge_bin = edged ? bin_of(of_key(thr)) : -1;
    for (int i = tid; i < kBins; i += kThreads) lo[i] = hi[i] = 0;
    __syncthreads();
    for (int i = tid; i < own; i += kThreads) {
      const Unit<T> x(slice[i]);
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        if (within(x.x[c])) add(x.x[c], bin_of(x.x[c]));
      }
    }
    cluster_sync();
    if (rank == 0) {
      u64 s[4] = {0, 0, 0, 0};
      for (int r = 0; r < blocks; ++r) {
        const uint4 l = get4(peer(lo + 4 * tid, r)), h = get4(peer(hi + 4 * tid, r));
        s[0] += l.x + ((u64)h.x << 16);
        s[1] += l.y + ((u64)h.y << 16);
        s[2] += l.z + ((u64)h.z << 16);
        s[3] += l.w + ((u64)h.w << 16);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * tid + i == edge_bin) s[i] += edge;
      u64 upto = block_scan(s[0] + s[1] + s[2] + s[3], part);
      if (tid == kThreads - 1) total_s = upto;
      __syncthreads();
      const u64 limit = weights ? shift_mul(total_s, want) : want;
      upto -= s[0] + s[1] + s[2] + s[3];
      if (limit == 0 || total_s < limit) {
        if (tid < blocks) put(peer(&news.left, tid), 0ull);
        if (tid < blocks) put(peer(&news.digit, tid), limit == 0 ? 0u : 1u);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (upto < limit && limit <= upto + s[i])
            for (int r = 0; r < blocks; ++r) {
              put(peer(&news.left, r), limit - upto);
              put(peer(&news.digit, r), (uint32_t)(4 * tid + i));
            }
          upto += s[i];
        }
      }
    }
    cluster_sync();
    u64 left = news.left;
    if (left == 0) {  // nothing asked for: the first token; or fewer tokens than asked for: all of them
      if (news.digit == 0) {
        thr = top_key;
        ties = 1;
      }
      return;
    }
    const int bin = (int)news.digit;
    // the keys in that step have leading bits in common, often all of them (bf16: a step is seldom wider than a value's)
    uint32_t most = 0, least = 0xffffffffu;
    for (int i = tid; i < own; i += kThreads) {
      const Unit<T> x(slice[i]);
#pragma unroll
      for (int c = 0; c < kN; ++c) {
        if (bin_of(x.x[c]) != bin || !within(x.x[c])) continue;
        most = max(most, key_of(x.x[c]));
        least = min(least, key_of(x.x[c]));
      }
    }
    const auto ends = block_ends(most, least, 0, part);
    if (tid < blocks) put(peer(&ranges[rank], tid), (u64)ends.most << 32 | ends.least);
    cluster_sync();
    most = edge_bin == bin ? thr : 0;
    least = edge_bin == bin ? thr : 0xffffffffu;
    for (int r = 0; r < blocks; ++r) {
      most = max(most, (uint32_t)(ranges[r] >> 32));
      least = min(least, (uint32_t)ranges[r]);
    }
    constexpr int kLast = sizeof(T) == 2 ? 16 : 0;  // a bf16's bits below are all equal
    const int bits = 32 - __clz(most ^ least);
    uint32_t prefix = bits == 32 ? 0 : most >> bits << bits;
    for (int end = bits; end > kLast;) {
      const int s = max(kLast, end - 8);
      const uint32_t digit_bits = (1u << (end - s)) - 1;
      auto fits = [&](uint32_t key) { return end == bits || (key ^ prefix) >> end == 0; };
      for (int i = tid; i < 256; i += kThreads) lo[i] = hi[i] = 0;
      __syncthreads();
      for (int i = tid; i < own; i += kThreads) {
        const Unit<T> x(slice[i]);
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          if (bin_of(x.x[c]) != bin || !within(x.x[c])) continue;
          const uint32_t key = key_of(x.x[c]);
          if (fits(key)) add(x.x[c], key >> s & digit_bits);
        }
      }
      cluster_sync();
      if (rank == 0) {
        const int d = 255 - tid;  // digits from the top
        u64 v = 0;
        for (int r = 0; r < blocks; ++r) v += get(peer(lo + d, r)) + ((u64)get(peer(hi + d, r)) << 16);
        if (edge_bin == bin && fits(thr) && (int)(thr >> s & digit_bits) == d) v += edge;
        const u64 upto = block_scan(v, part);
        if (upto - v < left && left <= upto)
          for (int r = 0; r < blocks; ++r) {
            put(peer(&news.left, r), left - (upto - v));
            put(peer(&news.digit, r), (uint32_t)d);
          }
      }
      cluster_sync();
      left = news.left;
      prefix |= news.digit << s;
      end = s;
    }
    if (sizeof(T) == 2 && !(prefix & 0x80000000u)) prefix |= 0xffff;  // a negative bf16's low bits, turned over
    const u64 W = weights ? weight.whole(of_key(prefix)) : 1;
    const u64 fit = (left + W - 1) / W;  // tokens of the last key before which the sum is still short
    ties = edged && prefix == thr ? min(ties, fit) : fit;
    thr = prefix;
  };
  if (k > 0 && k < p.V) narrow(false, 2.f * (peak - of_key(max(news.low, 1u))), (u64)k);
  if (top_p < 1.f) narrow(true, 22.f * temp, fraction(top_p, 1.f));  // 2^31 exp(-22) < 1/2: weights beyond are 0
  const bool edged = ties != ~0ull;
  const bool thr_in = edged && weight.w(of_key(thr)) >= floor_w;
  const u64 thr_w = thr_in ? weight.whole(of_key(thr)) : 0;

  // index order: each warp has a run of units; its kept weight is that of the keys above thr and of its share of the
  // tied ones
  const int run = (own + kWarps - 1) / kWarps, r0 = min(own, warp * run), r1 = min(own, r0 + run);
  const float edge_x = edged ? of_key(thr) : -INFINITY;
  auto above = [&](float x) -> uint32_t {
    if (!(edged ? x > edge_x : x >= edge_x)) return 0;  // NaN too
    const float w = weight.w(x);
    return w < floor_w ? 0 : __float2uint_rn(w * 2147483648.f);
  };
  u64 sum = 0, equal = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    const Unit<T> x(slice[i]);
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      sum += above(x.x[c]);
      equal += edged && x.x[c] == edge_x;
    }
  }
  sum = warp_sum(sum);
  equal = warp_sum(equal);
  if (lane == 0) warps[warp] = {sum, equal};
  __syncthreads();
  if (tid < blocks) {
    u64 s = 0, e = 0;
    for (int w = 0; w < kWarps; ++w) {
      s += warps[w].sum;
      e += warps[w].equal;
    }
    const uint32_t to = peer(&places[rank], tid);
    put(to, s);
    put(to + 8, e);
  }
  cluster_sync();
  u64 total = 0, seen = 0, before = 0, eq_before = 0;
  auto pass = [&](const Place& q) {
    const u64 take = seen >= ties ? 0 : min(q.equal, ties - seen);
    seen += q.equal;
    return q.sum + take * thr_w;
  };
  for (int r = 0; r < blocks; ++r) {
    if (r == (int)rank) {
      before = total;
      eq_before = seen;
    }
    total += pass(places[r]);
  }
  const u64 drawn = shift_mul(total, u);
  seen = eq_before;
  for (int w = 0; w < warp; ++w) before += pass(warps[w]);
  eq_before = seen;
  const u64 mine = pass(warps[warp]);
  if (!(before <= drawn && drawn < before + mine)) return;
  // the one warp whose run holds the drawn weight walks it
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const int i = i0 + lane;
    u64 W[kN], W_all = 0;
    uint32_t eq = 0;
    uint4 w = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
    if (i < r1) w = slice[i];
    const Unit<T> x(w);
#pragma unroll
    for (int c = 0; c < kN; ++c) eq += edged && x.x[c] == edge_x;
    uint32_t eq_upto = eq;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t o = __shfl_up_sync(kFull, eq_upto, off);
      if (lane >= off) eq_upto += o;
    }
    u64 place = eq_before + eq_upto - eq;
#pragma unroll
    for (int c = 0; c < kN; ++c) {
      W[c] = above(x.x[c]);
      if (edged && x.x[c] == edge_x) W[c] = place++ < ties ? thr_w : 0;
      W_all += W[c];
    }
    u64 upto = W_all;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const u64 o = __shfl_up_sync(kFull, upto, off);
      if (lane >= off) upto += o;
    }
    const unsigned hit = __ballot_sync(kFull, before + upto > drawn);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        u64 s = before + upto - W_all;
#pragma unroll
        for (int c = 0; c < kN; ++c) {
          if (s <= drawn && drawn < s + W[c]) {
            p.target[at] = first + i * kN + c;
            if (p.prob) p.prob[at] = weight.w(x.x[c]) * 2147483648.f / (float)total;
          }
          s += W[c];
        }
      }
      return;
    }
    before += __shfl_sync(kFull, upto, 31);
    eq_before += __shfl_sync(kFull, eq_upto, 31);
  }
}

// as gdn_greedy_accept's: the leading drafts equal to the target's tokens.  A warp per request: every draft is compared at
// once, where a loop that stops at the first difference would wait for a read of each.
__global__ void __launch_bounds__(256) accept_kernel(const gdn_sample_args p) {
  pdl_wait();
  pdl_trigger();
  const int b = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  if (b >= p.B) return;
  const int32_t* d = p.drafts + (size_t)b * (p.R - 1);
  const int32_t* tg = p.target + (size_t)b * p.R;
  const int n = p.n_rows[b];
  int a = 0;
  if (n <= p.R) {  // a bad count was flagged with the rows
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
      const int i = i0 + lane;
      const unsigned differ = __ballot_sync(kFull, i >= n - 1 || d[i] != tg[i]);
      a += differ ? __ffs(differ) - 1 : 32;
      if (differ) break;
    }
  }
  if (lane == 0) p.accept_len[b] = a;
}

template <typename Kernel, typename... Args>
int launch(Kernel kernel, dim3 grid, dim3 block, int cluster, size_t smem, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return GDN_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int check(const gdn_sample_args* a) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->R < 1 || a->V < 1 || a->row_stride < a->V) return GDN_ERR_INVALID_ARG;
  if (a->in_dtype != GDN_DTYPE_BF16 && a->in_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
  const size_t size = a->in_dtype == GDN_DTYPE_BF16 ? 2 : 4;
  if (a->V > GDN_SAMPLE_MAX_V || a->B > 65535 || a->R > 65535) return GDN_ERR_UNSUPPORTED;
  if (a->B == 0) return GDN_OK;
  if (!a->logits || !a->u || !a->n_rows || !a->target || (a->R > 1 && a->accept_len && !a->drafts))
    return GDN_ERR_INVALID_ARG;
  auto al = [](const void* ptr, uintptr_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; };
  const void* words[] = {a->u, a->temperature, a->top_k, a->top_p, a->min_p, a->drafts, a->n_rows,
                         a->target, a->prob, a->accept_len, a->status};
  if (!al(a->logits, size)) return GDN_ERR_MISALIGNED;
  for (const void* w : words)
    if (!al(w, 4)) return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

// Blocks per row: enough that a slice is at most 40 KB (four blocks of 256 threads fit an SM beside their scratch),
// and more, down to slices of 2 KB, while the rows alone do not give every SM two blocks.  Measured: 1152 rows of 50001
// bf16 took 99 us with 40 KB, 133 with 14 or 20, 109 with 60, 142 with 110; 128 rows of 32000 take 15 us with two blocks an
// SM, 26 with one, 18 with four.
int cluster_of(int64_t rows, int64_t bytes) {
  int c = 1;
  while (c < kMaxCluster && bytes > 40 * 1024 * (int64_t)c) c *= 2;
  while (c < kMaxCluster && rows * c < 304 && bytes > 2048 * (int64_t)c) c *= 2;
  return c;
}

template <typename T>
int run(const gdn_sample_args& p, cudaStream_t st) {
  constexpr int kN = Unit<T>::kN;
  const int blocks = cluster_of((int64_t)p.B * p.R, (int64_t)p.V * sizeof(T));
  const int units = (p.V + 2 * (kN - 1)) / kN;  // at the worst alignment
  const int slice_units = (units + blocks - 1) / blocks;
  const int smem = slice_units * 16 + kScratch * 4;
  auto start = [&](auto kernel) {
    // the largest slice's size, so that calls of any V from any thread set the same value
    if (smem > 40 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024) != cudaSuccess)
      return (int)GDN_ERR_LAUNCH;
    return launch(kernel, dim3(p.R * blocks, p.B), dim3(kThreads), blocks, smem, st, p, blocks, slice_units);
  };
  return (int64_t)p.B * p.R * blocks <= 4 * 152 ? start(sample_kernel<T, 4>) : start(sample_kernel<T, 6>);
}

}  // namespace gdnsample

using namespace gdnsample;

extern "C" GDN_API int gdn_sample_accept(const gdn_sample_args* args, void* stream) {
  const int rc = check(args);
  if (rc != GDN_OK || args->B == 0) return rc;
  const gdn_sample_args p = *args;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int r = p.in_dtype == GDN_DTYPE_BF16 ? run<__nv_bfloat16>(p, st) : run<float>(p, st);
  if (r != GDN_OK || !p.accept_len || p.R == 1) return r;
  return launch(accept_kernel, dim3((p.B + 7) / 8), dim3(256), 1, 0, st, p);
}
