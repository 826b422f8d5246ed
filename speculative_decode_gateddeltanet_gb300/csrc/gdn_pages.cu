// The paged cache's bookkeeping for one step: the page map (tables, slots and
// positions from request lengths) and the append of K and V rows to their slots.
//
// page_map_kernel: integer work on a few words per request, bound by latency.
//   Every block forms the three prefix sums (pages taken, pages given back,
//   rows) over all requests by itself, so that one launch with no exchange
//   between blocks does everything; the blocks then share the flat lists of
//   new table entries, returned pages and rows, each finding its request by a
//   binary search of the prefix in shared memory.  A row's page is taken from
//   the old table or straight from the ring, so no block reads what another
//   writes.  16 requests take 3.9 us, 1024 with prompts among them 7.3; an empty
//   launch takes 2.  (More blocks than SMs, or a search per row in global memory,
//   only add to the chain of dependent reads.)
// append_kernel: a copy, bound by HBM.  A thread moves one or four 16-byte chunks,
//   all loads in flight before the first store.  16381 rows of 8 heads of 128 in 32
//   bits take 41.4 us: 6.5 TB/s, 0.96 of a plain copy's rate.
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdnhybrid.h"

namespace gdnpages {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

constexpr int kMaxB = 4096;
constexpr unsigned kFull = 0xffffffffu;

// x / d for 0 <= x < 2^31 by a multiplication and a shift
struct Div {
  uint32_t mul, shift, d;
};

__device__ __forceinline__ uint32_t div(uint32_t x, const Div& k) {
  return k.d == 1 ? x : __umulhi(x, k.mul) >> k.shift;
}

Div make_div(uint32_t d) {
  Div k{0, 0, d};
  if (d == 1) return k;
  uint32_t l = 31 - __builtin_clz(d);
  if ((d & (d - 1)) == 0) l -= 1;  // a power of two: the multiplier is 2^31
  k.shift = l;
  k.mul = (uint32_t)(((uint64_t(1) << (32 + l)) + d - 1) / d);
  return k;
}

// the sums a request's place in the three lists comes from; 64 bits, as the
// demand of requests that are not served counts too
struct Sums {
  long long take, back, rows;
};

__device__ __forceinline__ Sums warp_scan(Sums v, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long a = __shfl_up_sync(kFull, v.take, off), b = __shfl_up_sync(kFull, v.back, off),
                    c = __shfl_up_sync(kFull, v.rows, off);
    if (lane >= off) {
      v.take += a;
      v.back += b;
      v.rows += c;
    }
  }
  return v;
}

// exclusive prefix of v over the block's threads; *total = the whole sum
template <int kThreads>
__device__ __forceinline__ Sums block_scan(Sums v, Sums* part, Sums* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Sums inc = warp_scan(v, lane);
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  Sums before = {inc.take - v.take, inc.back - v.back, inc.rows - v.rows}, all = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const Sums q = part[w];
    if (w == warp) {
      before.take += all.take;
      before.back += all.back;
      before.rows += all.rows;
    }
    all.take += q.take;
    all.back += q.back;
    all.rows += q.rows;
  }
  *total = all;
  __syncthreads();  // part may be used again
  return before;
}

// the last request whose prefix is not above i
__device__ __forceinline__ int find(const int* prefix, int B, int i) {
  int lo = 0, hi = B;  // prefix[lo] <= i < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// kPerThread requests a thread: one where they are few, as then the call is as long as its chain of reads and barriers
template <int kThreads, int kPerThread>
__global__ void __launch_bounds__(kThreads) page_map_kernel(const gdn_page_map_args p, const Div page_div) {
  extern __shared__ int sm[];
  __shared__ Sums part[kThreads / 32];
  int* const take_at = sm;                    // [B+1] prefix of pages taken
  int* const back_at = take_at + p.B + 1;     // [B+1] prefix of pages given back
  int* const row_at = back_at + p.B + 1;      // [B+1] prefix of rows (b*R when padded)
  int* const ctx_s = row_at + p.B + 1;        // [B]
  int* const held_s = ctx_s + p.B;            // [B] pages held before; need is held + taken - given back
  int* const rows_s = held_s + p.B;           // [B] rows served
  pdl_wait();
  pdl_trigger();
  const int N = p.n_pages, P = p.page_size, B = p.B;
  const int head = (int)((((long long)p.free_in[0] % N) + N) % N);
  const int n_free = min(max(p.free_in[1], 0), N);
  const int per = kPerThread == 1 ? 1 : (B + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * per;
  int ctx[kPerThread], n[kPerThread], held[kPerThread], need[kPerThread];
  int status = 0;
  Sums mine = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= per || b0 + i >= B) break;
    const int b = b0 + i;
    ctx[i] = p.ctx_len[b];
    n[i] = p.n_rows[b];
    held[i] = p.held_in[b];
    const long long tokens = (long long)ctx[i] + n[i];
    const long long up = tokens + P - 1, want = up >> 31 ? up / P : div((uint32_t)up, page_div);  // a negative one is refused
    int why = 0;
    if (ctx[i] < 0) why |= GDN_STATUS_BAD_LENGTH;
    if (n[i] < 0 || (p.R > 0 && n[i] > p.R)) why |= GDN_STATUS_BAD_NROWS;
    if (held[i] < 0 || held[i] > min(p.max_pages, N) || (!why && want > p.max_pages)) why |= GDN_STATUS_TABLE_FULL;
    if (why) {
      status |= why;
      n[i] = 0;
      need[i] = held[i];
    } else {
      need[i] = (int)want;
    }
    mine.take += max(need[i] - held[i], 0);
  }
  Sums total;
  Sums at = block_scan<kThreads>(mine, part, &total);
  // a request is served when the demand up to and with it fits the free pages
  Sums place = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= per || b0 + i >= B) break;
    const int want = max(need[i] - held[i], 0);
    at.take += want;
    // never more pages than there are, whatever the counts say: positions stay below 2^31
    if (want > 0 && (at.take > n_free || need[i] > N)) {
      status |= GDN_STATUS_NO_PAGES;
      need[i] = held[i];
      n[i] = 0;
    }
    place.take += max(need[i] - held[i], 0);
    place.back += max(held[i] - need[i], 0);
    place.rows += n[i];
  }
  Sums given;
  place = block_scan<kThreads>(place, part, &given);
  // what the free part leaves of the ring; counts that add up never return more, others are cut there
  const long long most_back = N - n_free;
  given.back = min(given.back, most_back);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (i >= per || b0 + i >= B) break;
    const int b = b0 + i;
    take_at[b] = (int)place.take;
    back_at[b] = (int)min(place.back, most_back);
    place.take += max(need[i] - held[i], 0);
    place.back += max(held[i] - need[i], 0);
    const int counted = n[i];
    const int first = p.R > 0 ? b * p.R : (int)min(place.rows, (long long)INT32_MAX);
    if (p.R == 0 && (p.slot_map || p.positions) && n[i] > 0 && place.rows + n[i] > p.n_slot_rows) {
      status |= GDN_STATUS_ROWS_FULL;
      n[i] = 0;
    }
    row_at[b] = first;
    place.rows += counted;
    ctx_s[b] = ctx[i];
    held_s[b] = held[i];
    rows_s[b] = n[i];
    if (blockIdx.x == 0) {
      p.held_out[b] = need[i];
      p.rows_out[b] = n[i];
      if (p.row_start) p.row_start[b] = first;
    }
  }
  const int end = p.R > 0 ? B * p.R : (int)min(given.rows, (long long)INT32_MAX);
  if (threadIdx.x == 0) {
    take_at[B] = (int)given.take;
    back_at[B] = (int)given.back;
    row_at[B] = end;
    if (blockIdx.x == 0) {
      p.free_out[0] = (int)((head + given.take) % N);
      p.free_out[1] = (int)(n_free - given.take + given.back);
      if (p.row_start) p.row_start[B] = end;
    }
  }
  if (blockIdx.x == 0 && status && p.status) atomicOr(p.status, status);
  __syncthreads();

  // a position of the ring, less than twice round in a state that adds up
  auto wrap = [&](long long x) {
    if (x >= N) x -= N;
    return (int)(x < N ? x : x % N);
  };
  // unsigned: the lists may end less than a step below 2^31
  const uint32_t first = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
  for (uint32_t i = first; i < given.take; i += step) {
    const int b = find(take_at, B, i);
    p.block_table[(size_t)b * p.table_stride + held_s[b] + i - take_at[b]] = p.free_ring[wrap((long long)head + i)];
  }
  // the ring's free part ends where the returned pages go: the two ranges are disjoint
  for (uint32_t i = first; i < given.back; i += step) {
    const int b = find(back_at, B, i);
    const int left = held_s[b] - (back_at[b + 1] - back_at[b]);  // pages kept
    p.free_ring[wrap((long long)head + n_free + i)] = p.block_table[(size_t)b * p.table_stride + left + i - back_at[b]];
  }
  if (!p.slot_map && !p.positions) return;
  for (uint32_t row = first; row < (uint32_t)p.n_slot_rows; row += step) {
    const int r = (int)row;
    int pos = -1, slot = -1;
    if (r < end) {
      const int b = p.R > 0 ? r / p.R : find(row_at, B, r);
      const int t = r - row_at[b];
      if (t < rows_s[b]) {
        pos = ctx_s[b] + t;
        const int i = (int)div(pos, page_div);
        const int page = i < held_s[b] ? p.block_table[(size_t)b * p.table_stride + i]
                                       : p.free_ring[wrap((long long)head + take_at[b] + i - held_s[b])];
        if ((unsigned)page < (unsigned)N) slot = page * P + pos - i * P;
        else if (p.status) atomicOr(p.status, GDN_STATUS_BAD_PAGE);
      }
    }
    if (p.slot_map) p.slot_map[r] = slot;
    if (p.positions) p.positions[r] = pos;
  }
}

struct AppendParams {
  int rows, n_slots, chunks;  // chunks of 16 bytes per (row, head)
  Div per_row, per_head, page;
  const uint4 *k, *v;  // strides below in 16-byte chunks
  int64_t k_row, k_head, v_row, v_head;
  const int32_t* slots;
  uint4 *kc, *vc;
  int64_t kc_page, kc_head, kc_token, vc_page, vc_head, vc_token;
  int32_t* status;
};

constexpr int kCopyThreads = 256;
// One chunk a thread where they are few, as the call is then as long as one thread's chain of reads (64 rows of 8 heads of
// 128 bf16: 1.8 us, with four chunks a thread 2.5; 2048 rows 3.8 and 4.5); four where HBM is the bound (4096 rows 6.2 and
// 6.1, 16384 rows 24.6 and 22.9).
constexpr uint32_t kOneEach = 1 << 18;

template <int kUnroll>
__global__ void __launch_bounds__(kCopyThreads) append_kernel(const AppendParams p) {
  pdl_wait();
  pdl_trigger();
  const bool is_v = blockIdx.y != 0;
  const uint4* src = is_v ? p.v : p.k;
  uint4* dst = is_v ? p.vc : p.kc;
  const int64_t s_row = is_v ? p.v_row : p.k_row, s_head = is_v ? p.v_head : p.k_head;
  const int64_t d_page = is_v ? p.vc_page : p.kc_page, d_head = is_v ? p.vc_head : p.kc_head,
                d_token = is_v ? p.vc_token : p.kc_token;
  const uint32_t total = (uint32_t)p.rows * p.per_row.d;
  const uint32_t base = blockIdx.x * (kCopyThreads * kUnroll) + threadIdx.x;
  uint4 val[kUnroll];
  int64_t to[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t i = base + u * kCopyThreads;
    to[u] = -1;
    if (i >= total) continue;
    const uint32_t row = div(i, p.per_row), in_row = i - row * p.per_row.d;
    const uint32_t head = div(in_row, p.per_head), c = in_row - head * p.per_head.d;
    const int slot = p.slots[row];
    val[u] = __ldcs(src + row * s_row + head * s_head + c);  // read once
    if (slot >= 0 && slot < p.n_slots) {
      const uint32_t page = div(slot, p.page), token = slot - page * p.page.d;
      to[u] = page * d_page + head * d_head + token * d_token + c;
    } else if (slot >= 0 && !is_v && in_row == 0 && p.status) {
      atomicOr(p.status, GDN_STATUS_BAD_PAGE);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (to[u] >= 0) dst[to[u]] = val[u];
}

template <typename Kernel, typename... Args>
int launch(Kernel kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return GDN_ERR_LAUNCH;
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_LAUNCH;
}

bool aligned(const void* ptr, uintptr_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

int check(const gdn_page_map_args* a) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->R < 0 || a->page_size < 1 || a->n_pages < 1 || a->max_pages < 0 || a->table_stride < a->max_pages ||
      a->n_slot_rows < 0 || a->reserved != 0)
    return GDN_ERR_INVALID_ARG;
  if (a->B > kMaxB || (int64_t)a->n_pages * a->page_size > INT32_MAX || (int64_t)a->B * a->R > INT32_MAX)
    return GDN_ERR_UNSUPPORTED;
  if (a->R > 0 && (a->slot_map || a->positions) && a->n_slot_rows != a->B * a->R) return GDN_ERR_INVALID_ARG;
  if (a->B == 0 && !a->free_in && !a->free_out) return GDN_OK;
  if (!a->free_in || !a->free_out) return GDN_ERR_INVALID_ARG;
  if (a->B > 0 && (!a->ctx_len || !a->n_rows || !a->held_in || !a->free_ring || !a->block_table || !a->held_out || !a->rows_out))
    return GDN_ERR_INVALID_ARG;
  const void* all[] = {a->ctx_len, a->n_rows, a->held_in, a->free_ring, a->free_in, a->block_table, a->held_out,
                       a->free_out, a->rows_out, a->row_start, a->slot_map, a->positions, a->status};
  for (const void* ptr : all)
    if (!aligned(ptr, 4)) return GDN_ERR_MISALIGNED;
  const size_t nb = (size_t)a->B * 4;
  const void* in[] = {a->ctx_len, a->n_rows, a->held_in};
  const void* out[] = {a->held_out, a->rows_out};
  for (const void* o : out) {
    for (const void* i : in)
      if (overlap(o, nb, i, nb)) return GDN_ERR_INVALID_ARG;
    if (overlap(o, nb, a->free_in, 8)) return GDN_ERR_INVALID_ARG;
  }
  if (overlap(a->free_out, 8, a->free_in, 8)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

int check(const gdn_kv_append_args* a) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->rows < 0 || a->H_kv < 1 || a->d < 1 || a->page_size < 1 || a->n_pages < 1) return GDN_ERR_INVALID_ARG;
  if (a->in_dtype != GDN_DTYPE_BF16 && a->in_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
  const int size = a->in_dtype == GDN_DTYPE_BF16 ? 2 : 4;
  const int64_t per_row = (int64_t)a->H_kv * ((int64_t)a->d * size / 16);  // chunks; below 2^60
  if ((int64_t)a->d * size % 16 != 0 || (int64_t)a->n_pages * a->page_size > INT32_MAX ||
      (a->rows > 0 && per_row > INT32_MAX / a->rows))
    return GDN_ERR_UNSUPPORTED;
  if (a->rows == 0) return GDN_OK;
  if (!a->k || !a->v || !a->slot_map || !a->k_cache || !a->v_cache) return GDN_ERR_INVALID_ARG;
  const int64_t strides[] = {a->k_row_stride, a->k_head_stride, a->v_row_stride, a->v_head_stride,
                             a->k_page_stride, a->k_cache_head_stride, a->k_token_stride,
                             a->v_page_stride, a->v_cache_head_stride, a->v_token_stride};
  for (int64_t s : strides)
    if (s * size % 16 != 0) return GDN_ERR_MISALIGNED;
  for (int i = 4; i < 10; ++i)  // the pools': a negative offset is a row that is not written
    if (strides[i] < 0) return GDN_ERR_INVALID_ARG;
  if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) ||
      !aligned(a->slot_map, 4) || !aligned(a->status, 4))
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

}  // namespace gdnpages

using namespace gdnpages;

extern "C" GDN_API int gdn_page_map(const gdn_page_map_args* args, void* stream) {
  const int rc = check(args);
  if (rc != GDN_OK || !args->free_out) return rc;
  const gdn_page_map_args p = *args;
  const size_t smem = (size_t)(6 * p.B + 3) * sizeof(int);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&](auto kernel, int threads) {
    // what a block gets without asking, 48 KB, holds the kernel's static part too
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (6 * kMaxB + 3) * sizeof(int)) != cudaSuccess)
      return (int)GDN_ERR_LAUNCH;
    const int blocks = (int)min(max(((int64_t)p.n_slot_rows + threads - 1) / threads, (int64_t)1), (int64_t)152);
    return launch(kernel, dim3(blocks), dim3(threads), smem, st, p, make_div((uint32_t)p.page_size));
  };
  // a thread per request and few warps to scan where they suffice: 16 requests 3.8 us, with 512 threads 4.8; 128 4.1 and 5.2
  return p.B <= 128 ? run(page_map_kernel<128, 1>, 128) : run(page_map_kernel<512, 8>, 512);
}

extern "C" GDN_API int gdn_kv_append(const gdn_kv_append_args* a, void* stream) {
  const int rc = check(a);
  if (rc != GDN_OK || a->rows == 0) return rc;
  const int per16 = a->in_dtype == GDN_DTYPE_BF16 ? 8 : 4;
  AppendParams p;
  p.rows = a->rows;
  p.n_slots = a->n_pages * a->page_size;
  p.chunks = a->d / per16;
  p.per_row = make_div((uint32_t)(a->H_kv * p.chunks));
  p.per_head = make_div((uint32_t)p.chunks);
  p.page = make_div((uint32_t)a->page_size);
  p.k = static_cast<const uint4*>(a->k);
  p.v = static_cast<const uint4*>(a->v);
  p.k_row = a->k_row_stride / per16;
  p.k_head = a->k_head_stride / per16;
  p.v_row = a->v_row_stride / per16;
  p.v_head = a->v_head_stride / per16;
  p.slots = a->slot_map;
  p.kc = static_cast<uint4*>(a->k_cache);
  p.vc = static_cast<uint4*>(a->v_cache);
  p.kc_page = a->k_page_stride / per16;
  p.kc_head = a->k_cache_head_stride / per16;
  p.kc_token = a->k_token_stride / per16;
  p.vc_page = a->v_page_stride / per16;
  p.vc_head = a->v_cache_head_stride / per16;
  p.vc_token = a->v_token_stride / per16;
  p.status = a->status;
  const uint32_t total = (uint32_t)p.rows * p.per_row.d;
  auto run = [&](auto kernel, uint32_t unroll) {
    const dim3 grid((total + kCopyThreads * unroll - 1) / (kCopyThreads * unroll), 2);
    return launch(kernel, grid, dim3(kCopyThreads), 0, static_cast<cudaStream_t>(stream), p);
  };
  return total <= kOneEach ? run(append_kernel<1>, 1) : run(append_kernel<4>, 4);
}
