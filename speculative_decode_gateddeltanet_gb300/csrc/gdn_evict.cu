// Eviction from the paged cache: the choice of tokens that leave, and their moves.
#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>

#include "attn_common.cuh"
#include "gdnlong.h"

namespace gdnevict {

using gdnattn::Div;
using gdnattn::kFull;
using gdnattn::launch;
using gdnattn::make_div;
using gdnattn::pdl_trigger;
using gdnattn::pdl_wait;
using gdnattn::quotient;

// ---- the choice -----------------------------------------------------------------------------------------------------------
//
// One block of 1024 threads for a request, or a cluster of eight where its table row can hold more than kOneBlock tokens.
// A warp owns consecutive tokens.  Their weights are read once, as whole numbers in the same order (kStays for those that may
// not leave), into shared memory; the heaviest key that leaves is found digit by digit with histograms of 11, 11 and 10 bits;
// then three passes over the keys count the equal ones, count gaps and movers, and write the lists: each warp's place in
// them comes from the counts of the warps and blocks before it, so they are in index order whatever the timing.  Histograms
// and counts of the cluster's blocks are read from each other's shared memory, with one cluster barrier for each.
// Tokens beyond what shared memory holds (eight blocks: 393216) are read again in each pass.
// Bound by latency: 16 requests of 1000 to 8000 tokens take 15 us (lengths 0.6, keys 2.3, a digit 1.5 each, counts 1.2, lists
// 1.2, weights moved 0.6), 8 of 60000 to 130000 39 us, where a digit costs 4 us: a cluster barrier and eight blocks'
// histograms.  The host knows the table row's width alone, so a wide row costs short requests too: 19 clusters run at a time,
// and 128 requests of 1000 to 8000 tokens take 146 us in rows of 131072 tokens, 17 in rows of 16384 (with nothing over the
// budget, where the weights are read all the same, 38 and 6.6).

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32, kOneBlock = 16384;
constexpr int kHeld = 49152;  // keys that a block of a cluster holds
constexpr int kBins = 2048;
constexpr uint32_t kStays = 0xffffffffu;  // above every weight's key

// weights as whole numbers in the same order; NaN as -infinity, -0 as 0
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct SelectShared {
  alignas(8) int hist[3][kBins];  // read two bins at once
  int warps[2][kSelectWarps];  // counts of each warp, then those before it
  int counts[4][2];            // this block's, by exchange
  int found[3];                // a pass's digit, how many of that digit leave, and whether those are all
};

static_assert(alignof(SelectShared) >= alignof(int2) && kBins % 2 == 0);

template <int kC>
__global__ void __launch_bounds__(kSelectThreads, 1) select_kernel(const gdn_evict_args p, const Div by_page) {
  extern __shared__ uint32_t held[];
  __shared__ SelectShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = kC == 1 ? 0 : blockIdx.x % kC, b = blockIdx.x / kC;
  for (int i = tid; i < 3 * kBins; i += kSelectThreads) (&sh.hist[0][0])[i] = 0;
  pdl_wait();
  pdl_trigger();
  const int L = p.ctx_len[b], budget = max(p.budget[b], 0), pinned = p.pinned ? max(p.pinned[b], 0) : 0;
  const bool bound = p.keep_from && p.born;
  const int keep_from = bound ? p.keep_from[b] : 0;
  const int32_t* const pages = p.block_table + (size_t)b * p.table_stride;
  auto leave = [&](int status) {  // as it was
    if (rank == 0 && tid == 0) {
      p.ctx_out[b] = L;
      p.n_moves[b] = 0;
      if (status && p.status) atomicOr(p.status, status);
    }
  };
  // every block of the cluster reads the length before any writes the new one: they meet below, or none goes that far
  const bool bad_length = L < 0 || L > (int64_t)p.max_pages * p.page_size;
  auto meet = [&]() {
    if constexpr (kC > 1) cg::this_cluster().sync();
    else __syncthreads();
  };
  if (bad_length) {
    meet();
    return leave(GDN_STATUS_BAD_LENGTH);
  }
  // this warp's tokens
  const int each = (int)(((int64_t)L + kC * kSelectThreads - 1) / (kC * kSelectThreads)) * 32;
  const int64_t first64 = ((int64_t)rank * kSelectWarps + warp) * each;
  const int first = (int)min(first64, (int64_t)L), mine = (int)min((int64_t)each, (int64_t)L - first);
  const bool staged = (int64_t)each * kSelectWarps <= (kC == 1 ? kOneBlock : kHeld);
  uint32_t* const keys = held + (staged ? warp * each : 0);
  auto slot_of = [&](int j, bool* good) {
    const int i = (int)quotient(j, by_page), page = pages[i];
    *good = (unsigned)page < (unsigned)p.n_pages;
    return page * p.page_size + j - i * p.page_size;
  };
  auto read_key = [&](int j, int* bad) {
    bool good;
    const int slot = slot_of(j, &good);
    if (!good) {
      *bad = 1;
      return kStays;
    }
    const float w = p.weight[slot];
    const int age = bound ? p.born[slot] : -1;
    return j >= pinned && (!bound || age < keep_from) ? weight_key(w) : kStays;
  };
  auto key_at = [&](int i) {
    int bad;
    return staged ? keys[i] : read_key(first + i, &bad);
  };
  int may = 0, bad = 0;
#pragma unroll 8
  for (int i = lane; i < mine; i += 32) {
    const uint32_t k = read_key(first + i, &bad);
    if (staged) keys[i] = k;
    may += k != kStays;
  }
  // sums over the cluster of two numbers of each warp (in lane 0), and over the warps before this one
  int round = 0;
  auto exchange = [&](int x, int y, int* before_x, int* before_y, int* all_x, int* all_y) {
    if (lane == 0) {
      sh.warps[0][warp] = x;
      sh.warps[1][warp] = y;
    }
    __syncthreads();
    if (warp < 2) {
      const int v = sh.warps[warp][lane];
      int inc = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(kFull, inc, off);
        if (lane >= off) inc += u;
      }
      sh.warps[warp][lane] = inc - v;
      if (lane == 31) sh.counts[round][warp] = inc;
    }
    meet();
    int bx = sh.warps[0][warp], by = sh.warps[1][warp], ax = 0, ay = 0;
#pragma unroll
    for (int r = 0; r < kC; ++r) {
      const int* const c = kC == 1 ? sh.counts[round] : cg::this_cluster().map_shared_rank(&sh.counts[round][0], r);
      if (r < rank) {
        bx += c[0];
        by += c[1];
      }
      ax += c[0];
      ay += c[1];
    }
    ++round;
    *before_x = bx;
    *before_y = by;
    *all_x = ax;
    *all_y = ay;
  };
  int bx, by, n_may, n_bad;
  exchange(__reduce_add_sync(kFull, may), __any_sync(kFull, bad), &bx, &by, &n_may, &n_bad);
  const int go = min(max(L - budget, 0), n_may), K = L - go;
  if (n_bad > 0 || go == 0) {
    if (kC > 1) meet();  // no block ends while another reads its counts
    return leave(n_bad > 0 ? GDN_STATUS_BAD_PAGE : 0);
  }
  // the go-th lightest key
  uint32_t key = 0, mask = 0;
  int ties = go;
  bool found_all = false;  // all keys that equal it leave
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    for (int i0 = 0; i0 < mine; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < mine ? key_at(i) : kStays;
      const bool in = k != kStays && (k & mask) == key;
      const unsigned any = __ballot_sync(kFull, in);
      if (any == 0) continue;
      const int bin = (int)(k >> shift) & (bins - 1), of_first = __shfl_sync(kFull, bin, __ffs(any) - 1);
      // one addition where all of the warp's are alike, as in a cache of equal weights
      if (__ballot_sync(kFull, in && bin == of_first) == any) {
        if (lane == 0) atomicAdd(&sh.hist[pass][of_first], __popc(any));
      } else if (in) {
        atomicAdd(&sh.hist[pass][bin], 1);
      }
    }
    meet();
    int n[2] = {0, 0};  // bins 2 tid and 2 tid + 1, of the whole cluster
    if (2 * tid < bins) {
#pragma unroll
      for (int r = 0; r < kC; ++r) {
        const int* const h = kC == 1 ? sh.hist[pass] : cg::this_cluster().map_shared_rank(&sh.hist[pass][0], r);
        const int2 v = *reinterpret_cast<const int2*>(h + 2 * tid);
        n[0] += v.x;
        n[1] += v.y;
      }
    }
    int inc = n[0] + n[1];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(kFull, inc, off);
      if (lane >= off) inc += u;
    }
    if (lane == 31) sh.warps[0][warp] = inc;
    __syncthreads();
    if (warp == 0) {
      const int v = sh.warps[0][lane];
      int s = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int u = __shfl_up_sync(kFull, s, off);
        if (lane >= off) s += u;
      }
      sh.warps[1][lane] = s - v;
    }
    __syncthreads();
    const int below = sh.warps[1][warp] + inc - n[0] - n[1];
    if (ties > below && ties <= below + n[0] + n[1]) {  // one thread
      const bool second = ties > below + n[0];
      sh.found[0] = 2 * tid + second;
      sh.found[1] = ties - below - (second ? n[0] : 0);
      sh.found[2] = sh.found[1] == (second ? n[1] : n[0]);
    }
    __syncthreads();
    key |= (uint32_t)sh.found[0] << shift;
    mask |= (uint32_t)(bins - 1) << shift;
    ties = sh.found[1];
    found_all = sh.found[2];
  }
  // `ties` of the keys that equal it leave, the last ones: all of them in most calls, and then one count of gaps and movers
  // does; otherwise it is made again once the equal keys before each warp are known
  int equal_before = 0, n_equal = ties;
  // f(token, whether it is one, whether it leaves) for each of the warp's tokens
  auto walk = [&](auto f) {
    int seen = equal_before;
    for (int i0 = 0; i0 < mine; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < mine ? key_at(i) : kStays;
      const unsigned same = __ballot_sync(kFull, k == key);
      const bool leaves = k < key || (k == key && seen + __popc(same & ((1u << lane) - 1)) >= n_equal - ties);
      seen += __popc(same);
      f(first + i, i < mine, leaves);
    }
    return seen - equal_before;
  };
  int gaps_before, movers_before, n_gaps, n_movers;
  auto count = [&](int* equal) {
    int gaps = 0, movers = 0;
    *equal = walk([&](int j, bool is, bool leaves) {
      gaps += is && leaves && j < K;
      movers += is && !leaves && j >= K;
    });
    exchange(__reduce_add_sync(kFull, gaps), __reduce_add_sync(kFull, movers), &gaps_before, &movers_before, &n_gaps, &n_movers);
  };
  int equal, n_ties;
  if (found_all) {
    count(&equal);
  } else {
    equal = 0;
    for (int i = lane; i < mine; i += 32) equal += key_at(i) == key;
    exchange(__reduce_add_sync(kFull, equal), 0, &equal_before, &by, &n_equal, &n_ties);
    count(&equal);
  }
  if (n_gaps > p.max_moves) {
    if (kC > 1) meet();
    return leave(GDN_STATUS_MOVES_FULL);
  }
  const size_t list = (size_t)b * p.max_moves;
  {
    int gap = gaps_before, mover = movers_before;
    walk([&](int j, bool is, bool leaves) {
      const unsigned g = __ballot_sync(kFull, is && leaves && j < K), m = __ballot_sync(kFull, is && !leaves && j >= K);
      const unsigned below = (1u << lane) - 1;
      if ((g | m) >> lane & 1) {
        bool good;
        const int slot = slot_of(j, &good);
        if (g >> lane & 1) p.move_to[list + gap + __popc(g & below)] = slot;
        else p.move_from[list + mover + __popc(m & below)] = slot;
      }
      gap += __popc(g);
      mover += __popc(m);
    });
  }
  meet();  // the lists are whole
  for (int i = rank * kSelectThreads + tid; i < n_gaps; i += kC * kSelectThreads) {
    const int from = p.move_from[list + i], to = p.move_to[list + i];
    const float w = p.weight[from];
    const int age = p.born ? p.born[from] : 0;
    p.weight[to] = w;
    if (p.born) p.born[to] = age;
  }
  if (rank == 0 && tid == 0) {
    p.ctx_out[b] = K;
    p.n_moves[b] = n_gaps;
  }
}

int run_select(const gdn_evict_args& a, cudaStream_t st) {
  const Div by_page = make_div((uint32_t)a.page_size);
  const int64_t most = (int64_t)a.max_pages * a.page_size;
  if (most <= kOneBlock) {
    const int smem = (int)((most + kSelectThreads - 1) / kSelectThreads * kSelectThreads * sizeof(uint32_t));
    if (cudaFuncSetAttribute(select_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOneBlock * (int)sizeof(uint32_t)) != cudaSuccess)
      return GDN_ERR_LAUNCH;
    return launch(select_kernel<1>, dim3(a.B), dim3(kSelectThreads), smem, st, a, by_page);
  }
  constexpr int kC = 8;
  const int64_t each = (most + kC * kSelectThreads - 1) / (kC * kSelectThreads) * kSelectThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.B * kC);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = (size_t)(each < kHeld ? each : kHeld) * sizeof(uint32_t);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kC;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaFuncSetAttribute(select_kernel<kC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * (int)sizeof(uint32_t)) != cudaSuccess ||
      cudaLaunchKernelEx(&cfg, select_kernel<kC>, a, by_page) != cudaSuccess || cudaGetLastError() != cudaSuccess)
    return GDN_ERR_LAUNCH;
  return GDN_OK;
}

// ---- moves ------------------------------------------------------------------------------------------------------------------
//
// A copy, bound by HBM, or by a chain of three reads where it is small: count and slots at once, the data, the store.  A
// thread moves one or four 16-byte chunks, all loads in flight before the first store: sources and destinations are disjoint.

struct MoveParams {
  int max_moves, first, moves;  // this launch's moves of each request
  int n_slots, page_size;
  Div per_row, per_pool, per_head, page;  // chunks of K and V of a token, of one of them, of a head
  int row_chunks, pool_chunks, head_chunks;
  const int32_t *from, *to, *n;
  uint4 *k, *v;  // strides in 16-byte chunks
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;
  int32_t* status;
};

constexpr int kMoveThreads = 256;

template <int kUnroll>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y;
  const int n = p.n[b];
  const uint32_t total = (uint32_t)p.moves * p.row_chunks, base = blockIdx.x * (kMoveThreads * kUnroll) + threadIdx.x;
  if (n < 0 || n > p.max_moves) {
    if (base == 0 && p.first == 0 && p.status) atomicOr(p.status, GDN_STATUS_BAD_LENGTH);
    return;
  }
  uint4 val[kUnroll];
  uint4* to[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const uint32_t i = base + u * kMoveThreads;
    to[u] = nullptr;
    if (i >= total) continue;
    const uint32_t move = quotient(i, p.per_row), in_row = i - move * p.row_chunks;
    if (p.first + (int)move >= n) continue;
    const size_t at = (size_t)b * p.max_moves + p.first + move;
    const int from = p.from[at], dest = p.to[at];
    if ((unsigned)from >= (unsigned)p.n_slots || (unsigned)dest >= (unsigned)p.n_slots) {
      if (in_row == 0 && p.status) atomicOr(p.status, GDN_STATUS_BAD_PAGE);
      continue;
    }
    const uint32_t is_v = quotient(in_row, p.per_pool), in_pool = in_row - is_v * p.pool_chunks;
    const uint32_t head = quotient(in_pool, p.per_head), c = in_pool - head * p.head_chunks;
    uint4* const pool = (is_v ? p.v : p.k) + head * (is_v ? p.v_head : p.k_head) + c;
    const int64_t page = is_v ? p.v_page : p.k_page, token = is_v ? p.v_token : p.k_token;
    const int from_page = (int)quotient(from, p.page), to_page = (int)quotient(dest, p.page);
    val[u] = __ldcs(pool + from_page * page + (from - from_page * p.page_size) * token);  // read once
    to[u] = pool + to_page * page + (dest - to_page * p.page_size) * token;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (to[u]) *to[u] = val[u];
}

// One chunk a thread where they are few (16 x 64 moves of 8 heads of 128 in bf16: 2.7 us, with four 3.5; 64 x 64 6.4 and 6.7),
// four where HBM is the bound (16 x 512 10.9 and 10.3; 15 requests of 500 to 1999 moves in f32 79.7 and 54.1: 6.3 TB/s).
// The host knows the lists' length alone: with 10 moves in each of 16 the 8 heads of 128 in bf16 take 2.1 us in lists of 64, 4.7
// in 512, 17.5 in 4096 and 66.6 in 16384, the time of the blocks that find nothing.
constexpr int64_t kOneEach = 1 << 20;

int run_move(const gdn_kv_move_args& a, cudaStream_t st) {
  const int per16 = a.in_dtype == GDN_DTYPE_BF16 ? 8 : 4;
  MoveParams p = {};
  p.max_moves = a.max_moves;
  p.n_slots = a.n_pages * a.page_size;
  p.page_size = a.page_size;
  p.head_chunks = a.d / per16;
  p.pool_chunks = a.H_kv * p.head_chunks;
  p.row_chunks = 2 * p.pool_chunks;
  p.per_row = make_div((uint32_t)p.row_chunks);
  p.per_pool = make_div((uint32_t)p.pool_chunks);
  p.per_head = make_div((uint32_t)p.head_chunks);
  p.page = make_div((uint32_t)a.page_size);
  p.from = a.move_from;
  p.to = a.move_to;
  p.n = a.n_moves;
  p.k = static_cast<uint4*>(a.k_cache);
  p.v = static_cast<uint4*>(a.v_cache);
  p.k_page = a.k_page_stride / per16;
  p.k_head = a.k_head_stride / per16;
  p.k_token = a.k_token_stride / per16;
  p.v_page = a.v_page_stride / per16;
  p.v_head = a.v_head_stride / per16;
  p.v_token = a.v_token_stride / per16;
  p.status = a.status;
  const int most = (INT32_MAX - 4 * kMoveThreads) / p.row_chunks;  // of one launch: chunk numbers are 32-bit
  for (p.first = 0; p.first < a.max_moves; p.first += p.moves) {
    p.moves = std::min(most, a.max_moves - p.first);
    const int64_t chunks = (int64_t)p.moves * p.row_chunks;
    auto run = [&](auto kernel, int unroll) {
      const dim3 grid((unsigned)((chunks + kMoveThreads * unroll - 1) / (kMoveThreads * unroll)), a.B);
      return launch(kernel, grid, dim3(kMoveThreads), 0, st, p);
    };
    const int rc = chunks * a.B <= kOneEach ? run(move_kernel<1>, 1) : run(move_kernel<4>, 4);
    if (rc != GDN_OK) return rc;
  }
  return GDN_OK;
}

// ---- host --------------------------------------------------------------------------------------------------------------------

bool aligned(const void* ptr, uintptr_t n) { return reinterpret_cast<uintptr_t>(ptr) % n == 0; }

}  // namespace gdnevict

using namespace gdnevict;

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
  return run_select(*a, static_cast<cudaStream_t>(stream));
}

extern "C" GDN_API int gdn_kv_move(const gdn_kv_move_args* a, void* stream) {
  if (!a) return GDN_ERR_INVALID_ARG;
  if (a->B < 0 || a->max_moves < 0 || a->H_kv < 1 || a->d < 1 || a->page_size < 1 || a->n_pages < 1 || a->reserved != 0) return GDN_ERR_INVALID_ARG;
  if (a->in_dtype != GDN_DTYPE_BF16 && a->in_dtype != GDN_DTYPE_F32) return GDN_ERR_UNSUPPORTED;
  const int size = a->in_dtype == GDN_DTYPE_BF16 ? 2 : 4, per16 = 16 / size;
  if ((int64_t)a->d * size % 16 != 0 || (int64_t)a->H_kv * (a->d / per16) > INT32_MAX / 4 || (int64_t)a->n_pages * a->page_size > INT32_MAX ||
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
  return run_move(*a, static_cast<cudaStream_t>(stream));
}
