// Eviction from the paged cache: the choice of tokens that leave, and their moves.
#include <algorithm>
#include <cmath>

#include "attn_common.cuh"
#include "gdnlong.h"

namespace gdnlong {

using gdnattn::Div;
using gdnattn::kFull;
using gdnattn::kMaxIndex;
using gdnattn::launch;
using gdnattn::make_div;
using gdnattn::Params;
using gdnattn::params_of;
using gdnattn::pdl_trigger;
using gdnattn::pdl_wait;
using gdnattn::quotient;
using gdnattn::request;
using gdnattn::Request;

template <typename T>
__device__ __forceinline__ float to_float(T x) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(x);
  else return x;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}

// ---- the choice: a block per request -----------------------------------------------------------------------------------------

constexpr int kSelectThreads = 1024;

// weights as whole numbers in the same order; NaN as -infinity, -0 as 0
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// sums over the block's threads before this one, and in all
__device__ __forceinline__ int block_before(int x, int* part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(kFull, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int before = inc - x, all = 0;
  for (int w = 0; w < kSelectThreads / 32; ++w) {
    if (w < warp) before += part[w];
    all += part[w];
  }
  __syncthreads();
  *total = all;
  return before;
}

__global__ void __launch_bounds__(kSelectThreads) select_simple(const gdn_evict_args p, const Div by_page) {
  __shared__ int part[kSelectThreads / 32], hist[256], found[2], bad_page;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const int L = p.ctx_len[b], budget = max(p.budget[b], 0), pinned = p.pinned ? max(p.pinned[b], 0) : 0;
    const int keep_from = p.keep_from && p.born ? p.keep_from[b] : INT32_MAX;
    const bool bound = p.keep_from && p.born;
    const int32_t* const pages = p.block_table + (size_t)b * p.table_stride;
    __syncthreads();
    if (tid == 0) bad_page = 0;
    __syncthreads();
    const bool bad_length = L < 0 || L > (int64_t)p.max_pages * p.page_size;
    if (!bad_length)
      for (int i = tid; i < (L + p.page_size - 1) / p.page_size; i += kSelectThreads)
        if ((unsigned)pages[i] >= (unsigned)p.n_pages) bad_page = 1;
    __syncthreads();
    if (bad_length || bad_page) {
      if (tid == 0) {
        p.ctx_out[b] = L;
        p.n_moves[b] = 0;
        if (p.status) atomicOr(p.status, bad_length ? GDN_STATUS_BAD_LENGTH : GDN_STATUS_BAD_PAGE);
      }
      continue;
    }
    auto slot_of = [&](int j) {
      const int i = (int)quotient(j, by_page);
      return pages[i] * p.page_size + j - i * p.page_size;
    };
    auto may_go = [&](int j, int slot) { return j >= pinned && (!bound || p.born[slot] < keep_from); };
    int mine = 0, n_may;
    for (int64_t j = tid; j < L; j += kSelectThreads) mine += may_go((int)j, slot_of((int)j));
    block_before(mine, part, &n_may);
    const int go = min(max(L - budget, 0), n_may), K = L - go;
    // the go-th lightest key, eight bits at a time: `low` keys are lighter, and `ties` of those that equal it leave too
    uint32_t key = 0, mask = 0;
    int ties = go;
    for (int shift = 24; shift >= 0 && go > 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelectThreads) hist[i] = 0;
      __syncthreads();
      for (int64_t j = tid; j < L; j += kSelectThreads) {
        const int slot = slot_of((int)j);
        if (!may_go((int)j, slot)) continue;
        const uint32_t k = weight_key(p.weight[slot]);
        if ((k & mask) == key) atomicAdd(&hist[k >> shift & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int i = 0, left = ties;
        while (left > hist[i]) left -= hist[i++];
        found[0] = i;
        found[1] = left;
      }
      __syncthreads();
      key |= (uint32_t)found[0] << shift;
      mask |= 255u << shift;
      ties = found[1];
    }
    int equal = 0, n_equal;
    for (int64_t j = tid; j < L && go > 0; j += kSelectThreads) {
      const int slot = slot_of((int)j);
      equal += may_go((int)j, slot) && weight_key(p.weight[slot]) == key;
    }
    block_before(equal, part, &n_equal);
    int64_t done_equal = 0, gaps = 0, movers = 0;
    // twice: the number of moves first, then the lists
    for (int round = 0; round < 2; ++round) {
      const int64_t moves = gaps;
      if (round == 1 && moves > p.max_moves) break;
      done_equal = gaps = movers = 0;
      for (int64_t j0 = 0; j0 < L && go > 0; j0 += kSelectThreads) {
        const int64_t j = j0 + tid;
        const int slot = j < L ? slot_of((int)j) : 0;
        const bool may = j < L && may_go((int)j, slot);
        const uint32_t k = may ? weight_key(p.weight[slot]) : 0;
        int n;
        const int tie_at = block_before(may && k == key, part, &n);
        const bool goes = may && (k < key || (k == key && done_equal + tie_at >= n_equal - ties));
        done_equal += n;
        const bool gap = goes && j < K, mover = j < L && !goes && j >= K;
        const int gap_at = block_before(gap, part, &n);
        if (round == 1 && gap) p.move_to[(size_t)b * p.max_moves + gaps + gap_at] = slot;
        gaps += n;
        const int mover_at = block_before(mover, part, &n);
        if (round == 1 && mover) p.move_from[(size_t)b * p.max_moves + movers + mover_at] = slot;
        movers += n;
      }
      if (round == 1 || moves > 0) continue;
    }
    const bool full = gaps > p.max_moves;
    __syncthreads();
    if (!full)
      for (int64_t i = tid; i < gaps; i += kSelectThreads) {
        const int from = p.move_from[(size_t)b * p.max_moves + i], to = p.move_to[(size_t)b * p.max_moves + i];
        p.weight[to] = p.weight[from];
        if (p.born) p.born[to] = p.born[from];
      }
    if (tid == 0) {
      p.ctx_out[b] = full ? L : K;
      p.n_moves[b] = full ? 0 : (int)gaps;
      if (full && p.status) atomicOr(p.status, GDN_STATUS_MOVES_FULL);
    }
  }
}

// ---- moves -----------------------------------------------------------------------------------------------------------------

struct MoveParams {
  int B, max_moves, n_slots, chunks, H_kv;
  Div page;
  int page_size;
  const int32_t *from, *to, *n;
  uint4 *k, *v;  // strides in 16-byte chunks
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;
  int32_t* status;
};

__global__ void __launch_bounds__(128) move_simple(const MoveParams p) {
  pdl_wait();
  pdl_trigger();
  for (int b = blockIdx.y; b < p.B; b += gridDim.y) {
    const int n = p.n[b];
    if (n < 0 || n > p.max_moves) {
      if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) atomicOr(p.status, GDN_STATUS_BAD_LENGTH);
      continue;
    }
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
      const int from = p.from[(size_t)b * p.max_moves + i], to = p.to[(size_t)b * p.max_moves + i];
      if ((unsigned)from >= (unsigned)p.n_slots || (unsigned)to >= (unsigned)p.n_slots) {
        if (threadIdx.x == 0 && p.status) atomicOr(p.status, GDN_STATUS_BAD_PAGE);
        continue;
      }
      const int from_page = (int)quotient(from, p.page), from_token = from - from_page * p.page_size;
      const int to_page = (int)quotient(to, p.page), to_token = to - to_page * p.page_size;
      for (int x = threadIdx.x; x < 2 * p.H_kv * p.chunks; x += 128) {
        const bool is_v = x >= p.H_kv * p.chunks;
        const int y = is_v ? x - p.H_kv * p.chunks : x, h = y / p.chunks, c = y - h * p.chunks;
        uint4* const pool = is_v ? p.v : p.k;
        const int64_t page = is_v ? p.v_page : p.k_page, head = is_v ? p.v_head : p.k_head, token = is_v ? p.v_token : p.k_token;
        pool[to_page * page + h * head + to_token * token + c] = pool[from_page * page + h * head + from_token * token + c];
      }
    }
  }
}

// ---- host --------------------------------------------------------------------------------------------------------------------

bool aligned(const void* ptr, uintptr_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; }

}  // namespace gdnlong

using namespace gdnlong;

extern "C" GDN_API int gdn_evict_select(const gdn_evict_args* a, void* stream) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->page_size < 1 || a->n_pages < 1 || a->max_pages < 0 || a->table_stride < a->max_pages || a->max_moves < 0)
    return GDN_ERR_INVALID_ARG;
  if (a->B > 65535 || (int64_t)a->n_pages * a->page_size > INT32_MAX || (int64_t)a->B * a->max_moves > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  if (a->B == 0) return GDN_OK;
  if (!a->block_table || !a->ctx_len || !a->budget || !a->weight || !a->ctx_out || !a->n_moves || (a->max_moves > 0 && (!a->move_from || !a->move_to)))
    return GDN_ERR_INVALID_ARG;
  const void* all[] = {a->block_table, a->ctx_len, a->budget, a->pinned, a->keep_from, a->weight, a->born, a->ctx_out, a->n_moves, a->move_from, a->move_to, a->status};
  for (const void* ptr : all)
    if (!aligned(ptr, 4)) return GDN_ERR_MISALIGNED;
  return launch(select_simple, dim3(a->B), dim3(kSelectThreads), 0, static_cast<cudaStream_t>(stream), *a, make_div((uint32_t)a->page_size));
}

extern "C" GDN_API int gdn_kv_move(const gdn_kv_move_args* a, void* stream) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->max_moves < 0 || a->H_kv < 1 || a->d < 1 || a->page_size < 1 || a->n_pages < 1 || a->reserved != 0) return GDN_ERR_INVALID_ARG;
  if (a->in_dtype != GDN_DTYPE_BF16 && a->in_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
  const int size = a->in_dtype == GDN_DTYPE_BF16 ? 2 : 4, per16 = 16 / size;
  if ((int64_t)a->d * size % 16 != 0 || (int64_t)a->H_kv * (a->d / per16) > INT32_MAX / 2 || (int64_t)a->n_pages * a->page_size > INT32_MAX ||
      a->B > 65535 || (int64_t)a->B * a->max_moves > INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  if (a->B == 0 || a->max_moves == 0) return GDN_OK;
  if (!a->move_from || !a->move_to || !a->n_moves || !a->k_cache || !a->v_cache) return GDN_ERR_INVALID_ARG;
  const int64_t strides[] = {a->k_page_stride, a->k_head_stride, a->k_token_stride, a->v_page_stride, a->v_head_stride, a->v_token_stride};
  for (int64_t s : strides) {
    if (s * size % 16 != 0) return GDN_ERR_MISALIGNED;
    if (s < 0) return GDN_ERR_INVALID_ARG;
  }
  if (!aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !aligned(a->move_from, 4) || !aligned(a->move_to, 4) || !aligned(a->n_moves, 4) ||
      !aligned(a->status, 4))
    return GDN_ERR_MISALIGNED;
  MoveParams p = {};
  p.B = a->B;
  p.max_moves = a->max_moves;
  p.n_slots = a->n_pages * a->page_size;
  p.chunks = a->d / per16;
  p.H_kv = a->H_kv;
  p.page = make_div((uint32_t)a->page_size);
  p.page_size = a->page_size;
  p.from = a->move_from;
  p.to = a->move_to;
  p.n = a->n_moves;
  p.k = static_cast<uint4*>(a->k_cache);
  p.v = static_cast<uint4*>(a->v_cache);
  p.k_page = a->k_page_stride / per16;
  p.k_head = a->k_head_stride / per16;
  p.k_token = a->k_token_stride / per16;
  p.v_page = a->v_page_stride / per16;
  p.v_head = a->v_head_stride / per16;
  p.v_token = a->v_token_stride / per16;
  p.status = a->status;
  return launch(move_simple, dim3(std::min(a->max_moves, 256), std::min(a->B, 1024)), dim3(128), 0, static_cast<cudaStream_t>(stream), p);
}
