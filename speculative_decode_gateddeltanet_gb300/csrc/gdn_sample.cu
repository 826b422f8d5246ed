// Acceptance of drafts against sampled target tokens: temperature, top-k,
// top-p and min-p from given random numbers.
//
// The order of a row's tokens (largest logit first, equal logits by lowest
// index) makes top-k and top-p prefixes of one order, so no sort is needed: a
// prefix is a threshold key and the number of tokens with exactly that key that
// belong to it.  Both are found by radix selection over the logits' ordered
// bits, eight bits a level, with counts (top-k) or weight sums (top-p) per
// digit.  The weights are whole numbers (32 bits of exp), their sums exact in
// 64 bits, so atomics and any split of the row give the same sums, and the
// drawn token does not depend on either.
//
// sample_kernel: one block per verify row.  accept_kernel: one thread per
// request.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdnhybrid.h"

namespace gdnsample {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

using u64 = unsigned long long;

__device__ __forceinline__ float value(const float* p) { return __ldg(p); }
__device__ __forceinline__ float value(const __nv_bfloat16* p) { return __bfloat162float(__ldg(p)); }

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
  __device__ uint32_t whole(float x) const { return (uint32_t)__float2ll_rn(w(x) * 2147483648.f); }
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

__device__ __forceinline__ u64 block_sum(u64 v, u64* part) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  u64 s = 0;
  for (int w = 0; w < kWarps; ++w) s += part[w];
  __syncthreads();
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const gdn_sample_args p) {
  __shared__ u64 hist[256];
  __shared__ u64 part[kWarps], part2[kWarps];
  __shared__ uint32_t s_key;
  __shared__ u64 s_sum;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x, b = blockIdx.y, V = p.V;
  pdl_wait();
  pdl_trigger();
  const int n = p.n_rows[b];
  if (n <= 0 || n > p.R || t >= n) return;
  const size_t at = (size_t)b * p.R + t;
  const T* row = static_cast<const T*>(p.logits) + at * p.row_stride;
  const float temp = p.temperature ? p.temperature[b] : 1.f;
  const int k = p.top_k ? p.top_k[b] : 0;
  const float top_p = p.top_p ? p.top_p[b] : 1.f, min_p = p.min_p ? p.min_p[b] : 0.f;

  // the largest key, lowest index: one 64-bit maximum of (key, ~index)
  u64 best = 0;
  for (int i = tid; i < V; i += kThreads) {
    const u64 c = (u64)key_of(value(row + i)) << 32 | (uint32_t)~i;
    best = c > best ? c : best;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const u64 o = __shfl_xor_sync(kFull, best, off);
    best = o > best ? o : best;
  }
  if (lane == 0) part[warp] = best;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) best = part[w] > best ? part[w] : best;
  __syncthreads();
  const uint32_t top_key = best >> 32;
  if (!(temp > 0.f) || top_key == 0) {  // greedy, or a row of NaN alone
    if (tid == 0) {
      p.target[at] = top_key == 0 ? 0 : (int)~(uint32_t)best;
      if (p.prob) p.prob[at] = 1.f;
    }
    return;
  }
  const Weight weight{of_key(top_key), 1.f / temp};

  // kept: keys above thr, and the first `ties` tokens (by index) of key thr
  uint32_t thr = 1;  // every key but NaN's
  u64 ties = (u64)V;
  if (k > 0 && k < V) {
    uint32_t prefix = 0;
    u64 left = (u64)k;
    bool all = false;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int i = tid; i < V; i += kThreads) {
        const uint32_t key = key_of(value(row + i));
        if (key != 0 && (shift == 24 || (key ^ prefix) >> (shift + 8) == 0)) atomicAdd(&hist[key >> shift & 255], 1ull);
      }
      __syncthreads();
      if (tid == 0) {
        int d = 255;
        u64 above = 0;
        while (d > 0 && above + hist[d] < left) above += hist[d--];
        s_key = d;
        s_sum = above;
        part[0] = hist[d];
      }
      __syncthreads();
      if (shift == 24 && s_sum + part[0] < left) all = true;  // fewer than k tokens that are not NaN
      prefix |= s_key << shift;
      left -= s_sum;
      __syncthreads();
      if (all) break;
    }
    if (!all) {
      thr = prefix;
      ties = left;
    }
  }
  if (top_p < 1.f) {
    u64 sum = 0;
    for (int i = tid; i < V; i += kThreads) {
      const float x = value(row + i);
      if (key_of(x) > thr || (key_of(x) == thr && ties >= (u64)V)) sum += weight.whole(x);
    }
    const u64 edge = ties >= (u64)V ? 0 : ties * weight.whole(of_key(thr));  // the tied tokens' share
    const u64 limit = shift_mul(block_sum(sum, part) + edge, fraction(top_p, 1.f));
    if (limit == 0) {
      thr = top_key;
      ties = 1;
    } else {
      uint32_t prefix = 0;
      u64 left = limit;
      for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < V; i += kThreads) {
          const float x = value(row + i);
          const uint32_t key = key_of(x);
          if ((key > thr || (key == thr && ties >= (u64)V)) && (shift == 24 || (key ^ prefix) >> (shift + 8) == 0)) {
            const uint32_t W = weight.whole(x);
            if (W) atomicAdd(&hist[key >> shift & 255], (u64)W);
          }
        }
        __syncthreads();
        if (tid == 0) {
          if (edge && (shift == 24 || (thr ^ prefix) >> (shift + 8) == 0)) hist[thr >> shift & 255] += edge;
          int d = 255;
          u64 above = 0;
          while (d > 0 && above + hist[d] < left) above += hist[d--];
          s_key = d;
          s_sum = above;
        }
        __syncthreads();
        prefix |= s_key << shift;
        left -= s_sum;
        __syncthreads();
      }
      // tokens of the last key are kept while what came before them is below the limit
      const u64 W = weight.whole(of_key(prefix));
      const u64 fit = (left + W - 1) / W;
      ties = prefix == thr && ties < fit ? ties : fit;
      thr = prefix;
    }
  }
  const float floor_w = min_p > 0.f ? fminf(min_p, 1.f) : 0.f;
  const bool thr_in = weight.w(of_key(thr)) >= floor_w;
  const u64 thr_w = thr_in ? weight.whole(of_key(thr)) : 0;

  // index order: each warp has a run of tokens; its kept weight is that of the
  // keys above thr and of its share of the tied ones
  const int per = ((V + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int i0 = min(V, warp * per), i1 = min(V, i0 + per);
  u64 sum = 0, equal = 0;
  for (int i = i0 + lane; i < i1; i += 32) {
    const float x = value(row + i);
    const uint32_t key = key_of(x);
    if (key > thr && weight.w(x) >= floor_w) sum += weight.whole(x);
    equal += key == thr;
  }
  sum = warp_sum(sum);
  equal = warp_sum(equal);
  if (lane == 0) {
    part[warp] = sum;
    part2[warp] = equal;
  }
  __syncthreads();
  u64 total = 0, seen = 0, before = 0, eq_before = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) {
      before = total;
      eq_before = seen;
    }
    const u64 eq = seen >= ties ? 0 : min(part2[w], ties - seen);
    total += part[w] + eq * thr_w;
    seen += part2[w];
  }
  const u64 own_eq = eq_before >= ties ? 0 : min(equal, ties - eq_before);
  const u64 drawn = shift_mul(total, fraction(p.u[at], 1.f - 1.f / 16777216.f));
  if (!(before <= drawn && drawn < before + sum + own_eq * thr_w)) return;
  // the one warp whose run holds the drawn weight walks it
  for (int i = i0; i < i1; i += 32) {
    float x = 0.f;
    uint32_t key = 0;
    if (i + lane < i1) {
      x = value(row + i + lane);
      key = key_of(x);
    }
    const unsigned eq = __ballot_sync(kFull, key == thr);
    const u64 rank = eq_before + __popc(eq & ((1u << lane) - 1));
    u64 W = key > thr && weight.w(x) >= floor_w ? weight.whole(x) : key == thr && rank < ties ? thr_w : 0;
    u64 inc = W;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const u64 o = __shfl_up_sync(kFull, inc, off);
      if (lane >= off) inc += o;
    }
    const unsigned hit = __ballot_sync(kFull, before + inc > drawn);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        p.target[at] = i + lane;
        if (p.prob) p.prob[at] = weight.w(x) * 2147483648.f / (float)total;
      }
      return;
    }
    before += __shfl_sync(kFull, inc, 31);
    eq_before += __popc(eq);
  }
}

// as gdn_greedy_accept's: the leading drafts equal to the target's tokens
__global__ void __launch_bounds__(256) accept_kernel(const gdn_sample_args p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.B) return;
  const int n = p.n_rows[b];
  int a = 0;
  if (n < 0 || n > p.R) {
    if (p.status) atomicOr(p.status, GDN_STATUS_BAD_NROWS);
  } else {
    const int32_t* d = p.drafts + (size_t)b * (p.R - 1);
    const int32_t* tg = p.target + (size_t)b * p.R;
    while (a < n - 1 && d[a] == tg[a]) ++a;
  }
  p.accept_len[b] = a;
}

template <typename Kernel>
int launch(Kernel kernel, dim3 grid, dim3 block, cudaStream_t st, const gdn_sample_args& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) return GDN_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

int check(const gdn_sample_args* a) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->R < 1 || a->V < 1 || a->row_stride < a->V) return GDN_ERR_INVALID_ARG;
  if (a->in_dtype != GDN_DTYPE_BF16 && a->in_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
  const size_t size = a->in_dtype == GDN_DTYPE_BF16 ? 2 : 4;
  if (a->V > (1 << 20) || a->V * size > GDN_SAMPLE_MAX_STAGED || a->B > 65535 || a->R > 65535) return GDN_ERR_UNSUPPORTED;
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

}  // namespace gdnsample

using namespace gdnsample;

extern "C" GDN_API int gdn_sample_accept(const gdn_sample_args* args, void* stream) {
  const int rc = check(args);
  if (rc != GDN_OK || args->B == 0) return rc;
  const gdn_sample_args p = *args;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 grid(p.R, p.B);
  const int r = p.in_dtype == GDN_DTYPE_BF16 ? launch(sample_kernel<__nv_bfloat16>, grid, dim3(kThreads), st, p)
                                             : launch(sample_kernel<float>, grid, dim3(kThreads), st, p);
  if (r != GDN_OK || !p.accept_len) return r;
  return launch(accept_kernel, dim3((p.B + 255) / 256), dim3(256), st, p);
}
