// What the paged-attention kernels share: the call's parameters, the division
// of its work over blocks, and the join of partial results.
//
// Rows.  For one request and kv head, the G = H_q / H_kv query heads of the n
//   new tokens are one matrix of n*G rows (row r: token r / G, head r % G), cut
//   into tiles of kRows rows; K and V are cut into blocks of kKeys positions.
//   A tile needs the blocks up to its last row's position:
//     c(m) = floor((ctx + floor((last row of m) / G)) / kKeys) + 1.
// Division.  All (request, kv head, tile, key block) units of a call form one
//   line, with some units more for each tile's own cost (its q rows in, its o
//   rows out); block i takes units [i*per, (i+1)*per).  Every block so has the
//   same work however ragged the lengths are: a long context is split over many
//   blocks, many short ones share a block.  The line's length needs only sums of
//   c(m), which a floor-sum gives without a loop over tiles, so each block finds
//   its own part in a scan over the requests, with no planning launch before it.
// Join.  A tile whose units lie in several blocks is split: its first block
//   writes a head partial (slot 1) and a note of how many blocks follow, each
//   of those writes a tail partial (slot 0): the running maximum, sum and
//   unnormalised output in 32 bits.  combine_kernel adds them up in block
//   order, so the result does not depend on timing.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdnhybrid.h"

namespace gdnattn {

constexpr unsigned kFull = 0xffffffffu;
// the kernels' positions and row numbers are 32-bit, and run up to a block past a request's last
constexpr int kMaxIndex = INT32_MAX - 1023;

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// x / d for 0 <= x < 2^31 as a multiplication and a shift
struct Div {
  uint32_t mul, shift;
};
__device__ __forceinline__ uint32_t quotient(uint32_t x, const Div& k) { return k.mul ? __umulhi(x, k.mul) >> k.shift : x; }
inline Div make_div(uint32_t d) {
  if (d == 1) return {0, 0};
  const uint32_t l = 31 - __builtin_clz(d) - ((d & (d - 1)) == 0);  // a power of two: the multiplier is 2^31
  return {(uint32_t)(((uint64_t(1) << (32 + l)) + d - 1) / d), l};
}

struct Params {
  int B, R, H_kv, G, d;
  int page_size, n_pages, table_stride, n_q_rows;
  int max_tokens, max_rows;  // of a request: max_pages * page_size and kMaxIndex / G, below 2^31 by a block of keys and more
  float scale_log2;    // scale * log2(e): scores are kept in the exponent of 2
  Div by_G, by_page;
  const void* q;
  int64_t q_row, q_head;
  const void *k, *v;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;
  const int32_t *table, *ctx_len, *n_rows, *row_start;
  void* o;
  int64_t o_row, o_head;
  int4* notes;      // [blocks] note_of a split tile's first block; zeros where the block begins none
  float* partials;  // [blocks][2 slots][kRows][d + 2]: outputs, then the rows' maxima and sums
  int32_t* status;
  int n_blocks;     // blocks of the attention launch
};

struct Request {
  int ctx, n, row0;
};

// request b's lengths; n = 0 where it takes no part
__device__ __forceinline__ Request request(const Params& p, int b, int* why = nullptr) {
  Request r;
  r.ctx = p.ctx_len[b];
  r.n = p.n_rows[b];
  r.row0 = p.row_start ? p.row_start[b] : b * p.R;
  int bad = 0;
  if (r.n < 0 || (p.R > 0 && r.n > p.R)) bad |= GDN_STATUS_BAD_NROWS;
  if (r.n > 0 && (r.ctx < 0 || (int64_t)r.ctx + r.n > p.max_tokens || r.n > p.max_rows || r.row0 < 0 ||
                  (int64_t)r.row0 + r.n > p.n_q_rows))
    bad |= GDN_STATUS_BAD_LENGTH;
  if (bad) r.n = 0;
  if (why) *why |= bad;
  return r;
}

// sum over i in [0, n) of floor((a*i + b) / m), the lattice points under a line: whole multiples of m are taken out of a
// and b, the points under what is left are counted along the other axis.  That is Euclid's algorithm on (m, a); the
// exchange of axes is the reciprocity law of floor sums (Graham, Knuth, Patashnik: Concrete Mathematics, section 3.5).
__device__ inline long long floor_sum(long long n, long long m, long long a, long long b) {
  long long s = 0;
  while (n > 0) {
    if (a >= m) {
      s += n * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      s += n * (b / m);
      b %= m;
    }
    const long long y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y % m;
    const long long t = m;
    m = a;
    a = t;
  }
  return s;
}

template <int kRows, int kKeys>
struct Tiles {
  __device__ static int count(const Params& p, const Request& r) { return (int)(((unsigned long long)r.n * p.G + kRows - 1) / kRows); }
  __device__ static int blocks(const Params& p, const Request& r, int m) {
    const long long last = min((long long)(m + 1) * kRows, (long long)r.n * p.G) - 1;
    const int token = last >> 31 ? (int)(last / p.G) : (int)quotient((uint32_t)last, p.by_G);
    return (int)((unsigned)(r.ctx + token) / kKeys) + 1;
  }
  // Units that a tile costs beside its key blocks, in the time of one: about 3 us from a tile's last product to the next
  // one's first on the tensor cores.  Measured (64-key blocks, 128-key blocks): 16 x 4 rows at d = 256 take 35.7 us with
  // 5, 39.2 with 3 or 4, 36.1 with 10; prompt chunks of up to 4096 485 with 3, 493 with 2, 516 with 1, 504 with 6; 256
  // ragged requests 172 with 3, 177 with 6.
  static constexpr int kExtra = kRows < 128 ? 0 : kKeys == 64 ? 5 : 3;
  // units of the tiles before m
  __device__ static long long before(const Params& p, const Request& r, int m) {
    if (m == 0) return 0;
    return (long long)m * (1 + kExtra) + floor_sum(m, (long long)p.G * kKeys, kRows, (long long)p.G * r.ctx + kRows - 1);
  }
  // units of one kv head of the request
  __device__ static long long sum(const Params& p, const Request& r) {
    if (r.n <= 0) return 0;
    const int M = count(p, r);
    return before(p, r, M - 1) + kExtra + blocks(p, r, M - 1);
  }
};

// one block's walk over its units, tile by tile
template <int kRows, int kKeys>
struct Walk {
  using T = Tiles<kRows, kKeys>;
  Request req;
  int b, h, m, tiles, left;  // left: units still to do
  int at;                    // the segment's first unit within its tile: the tile's own units come first
  int kb0, kb1, blocks;      // its key blocks, and how many the whole tile has

  __device__ void segment() {
    blocks = T::blocks(*p, req, m);
    const int end = min(T::kExtra + blocks, at + left);
    kb0 = max(0, at - T::kExtra);
    kb1 = end - T::kExtra;
    if (kb1 <= kb0) left = 0;  // the block's part ends before the tile's first key block
  }
  __device__ bool done() const { return left <= 0; }
  __device__ void next() {
    left -= kb1 + T::kExtra - at;
    if (left <= 0) return;
    at = 0;
    if (++m == tiles) {
      m = 0;
      if (++h == p->H_kv) {
        h = 0;
        do {
          req = request(*p, ++b);
        } while (req.n <= 0);
        tiles = T::count(*p, req);
      }
    }
    segment();
  }
  const Params* p;
};

struct Start {
  long long total;  // units of the call
  long long off;    // units from the first request's first to the block's first
  long long head;   // units of one kv head of that request
  Request req;      // the request the block begins in
  int b, per;
};

// Every thread of the block calls this; all get the block's first unit.  scan:
// kThreads/32 words of shared memory.  The thread that meets the block's first
// unit passes its request on, so nothing is read twice before the first tile.
template <int kRows, int kKeys, int kThreads>
__device__ __forceinline__ void find_start(const Params& p, int min_units, long long* scan, Start* out) {
  using T = Tiles<kRows, kKeys>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int each = (p.B + kThreads - 1) / kThreads;
  const int b0 = threadIdx.x * each, b1 = min(p.B, b0 + each);
  long long mine = 0, head = 0;
  Request req = {0, 0, 0};
  int why = 0;
  for (int b = b0; b < b1; ++b) {
    req = request(p, b, &why);
    head = T::sum(p, req);
    mine += p.H_kv * head;
  }
  if (why && blockIdx.x == 0 && p.status) atomicOr(p.status, why);
  long long inc = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long v = __shfl_up_sync(kFull, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  const long long at = before + inc - mine;
  // 32-bit division where the sum allows it
  const long long want = total >> 31 ? (total + p.n_blocks - 1) / p.n_blocks
                                     : (long long)(((uint32_t)total + (uint32_t)p.n_blocks - 1) / (uint32_t)p.n_blocks);
  const long long per = max(want, (long long)min_units);
  const long long first = per * blockIdx.x;
  if (threadIdx.x == 0) {
    out->total = total;
    out->per = (int)min(per, (long long)INT32_MAX);
  }
  if (first >= at && first < at + mine) {  // one thread at most
    long long off = first - at;
    int b = b0;
    if (each > 1) {
      for (;; ++b) {
        req = request(p, b);
        head = T::sum(p, req);
        if (off < p.H_kv * head) break;
        off -= p.H_kv * head;
      }
    }
    out->b = b;
    out->off = off;
    out->head = head;
    out->req = req;
  }
  __syncthreads();
}

template <int kRows, int kKeys>
__device__ __forceinline__ bool begin(Walk<kRows, kKeys>& w, const Params& p, const Start& s) {
  using T = Tiles<kRows, kKeys>;
  w.p = &p;
  const long long first = (long long)s.per * blockIdx.x;
  w.left = (int)max(0ll, min((long long)s.per, s.total - first));
  if (w.left <= 0) return false;
  w.b = s.b;
  w.req = s.req;
  w.tiles = T::count(p, w.req);
  long long off = s.off;
  w.h = (off | s.head) >> 31 ? (int)(off / s.head) : (int)((uint32_t)off / (uint32_t)s.head);
  off -= w.h * s.head;
  int lo = 0, hi = w.tiles;  // before(lo) <= off < before(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (T::before(p, w.req, mid) <= off) lo = mid;
    else hi = mid;
  }
  w.m = lo;
  w.at = (int)(off - T::before(p, w.req, lo));
  w.segment();
  return !w.done();
}

// The note of a split tile at its first block: the blocks that follow this one
// in it, its request's first row, kv head and rows, and its first row's number.
template <int kRows, int kKeys>
__device__ __forceinline__ int4 note_of(const Walk<kRows, kKeys>& w, const Start& s) {
  const int followers = (w.blocks - w.kb1 + s.per - 1) / s.per;
  const int rows = (int)min((long long)kRows, (long long)w.req.n * w.p->G - (long long)w.m * kRows);
  return {followers, w.req.row0, w.h << 8 | rows, w.m * kRows};
}

__device__ __forceinline__ float* partial(const Params& p, int block, int slot, int rows) {
  return p.partials + (size_t)(block * 2 + slot) * rows * (p.d + 2);
}

// And blocks a tile: eight for bf16 (4 lose 1 to 3 us where partials are many, 16 and 32 where few), four for the smaller
// tiles of 32 bits.
constexpr int kCombineWarps = 4;

// Joins the partials of the split tile that block blockIdx.x of the attention
// begins; gridDim.y blocks share its rows.  Up to eight partials: a warp per row,
// or per two rows at once where there are two partials, as in a prompt's tiles (3
// prompts of 608 tokens over 9000: 250 -> 244 us, 8 of 300 over 700 at d = 256: 72 ->
// 66).  More (few tiles, long contexts): a block per row, warp w taking partials w,
// w + 4, ..., and the warps' sums added in warp order (one token over 65537: 54.3 us,
// with a warp per row 55.8; the other way round 16 requests of 4 tokens take 44.1
// instead of 40.0).  The order is fixed by the lengths alone.  Bound by the latency
// of three dependent reads and by instruction misses: a third variant of the few
// partials' loop made every call 0.5 to 1 us slower.
template <typename T, int kD, int kRows>
__global__ void __launch_bounds__(32 * kCombineWarps) combine_kernel(const Params p) {
  constexpr int kPer = kD / 32;
  __shared__ float sums[kCombineWarps][kD];
  pdl_wait();
  pdl_trigger();
  const int4 note = p.notes[blockIdx.x];
  const int parts = note.x + 1;
  if (parts <= 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = note.z & 255, kv_head = note.z >> 8;
  auto part = [&](int i) { return partial(p, blockIdx.x + i, i == 0, kRows); };
  auto stats = [&](int i, int row) { return reinterpret_cast<const float2*>(part(i) + (size_t)kRows * kD)[row]; };
  // this lane's columns of partial i's row
  auto load = [&](float (&x)[kPer], int i, int row) {
    const float* src = part(i) + (size_t)row * kD + lane * 2;
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c) {
      const float2 v = *reinterpret_cast<const float2*>(src + c * 64);
      x[2 * c] = v.x;
      x[2 * c + 1] = v.y;
    }
  };
  auto write = [&](int row, const float (&acc)[kPer], float sum) {
    const float inv = 1.f / sum;
    const int at = note.w + row, token = (int)quotient(at, p.by_G), head = kv_head * p.G + at - token * p.G;
    T* dst = static_cast<T*>(p.o) + (int64_t)(note.y + token) * p.o_row + (int64_t)head * p.o_head + lane * 2;
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c) {
      const float a = acc[2 * c] * inv, b = acc[2 * c + 1] * inv;
      if constexpr (sizeof(T) == 2) *reinterpret_cast<__nv_bfloat162*>(dst + c * 64) = __floats2bfloat162_rn(a, b);
      else *reinterpret_cast<float2*>(dst + c * 64) = make_float2(a, b);
    }
  };
  // up to kMost partials, kAtOnce rows of this warp at a time
  auto few = [&](auto most, auto at_once) {
    constexpr int kMost = decltype(most)::value, kAtOnce = decltype(at_once)::value;
    const int step = (int)gridDim.y * kCombineWarps;
    for (int row0 = (int)blockIdx.y * kCombineWarps + warp; row0 < rows; row0 += step * kAtOnce) {
      float x[kAtOnce][kMost][kPer];
      float2 st[kAtOnce][kMost];
#pragma unroll
      for (int r = 0; r < kAtOnce; ++r)
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          const int row = min(row0 + r * step, rows - 1), from = min(i, parts - 1);
          st[r][i] = stats(from, row);
          load(x[r][i], from, row);
        }
#pragma unroll
      for (int r = 0; r < kAtOnce; ++r) {
        if (row0 + r * step >= rows) break;
        float top = st[r][0].x, sum = 0.f, acc[kPer] = {};
#pragma unroll
        for (int i = 1; i < kMost; ++i) top = fmaxf(top, st[r][i].x);
        if (top == -INFINITY) top = 0.f;
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          const float weight = i < parts ? exp2f(st[r][i].x - top) : 0.f;
          sum += st[r][i].y * weight;
#pragma unroll
          for (int c = 0; c < kPer; ++c) acc[c] = fmaf(weight, x[r][i][c], acc[c]);
        }
        write(row0 + r * step, acc, sum);
      }
    }
  };
  if (parts <= 2) return few(std::integral_constant<int, 2>(), std::integral_constant<int, 2>());
  if (parts <= 8) return few(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  constexpr int kBatch = 8;  // partials whose loads are under way at once
  for (int row = (int)blockIdx.y; row < rows; row += (int)gridDim.y) {
    float x[kBatch][kPer], tops[kBatch], acc[kPer] = {};
    auto batch = [&](int i0) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = min(i0 + j * kCombineWarps, parts - 1);
        tops[j] = stats(i, row).x;
        load(x[j], i, row);
      }
    };
    batch(warp);  // on their way while the maximum and the sum are formed
    float top = -INFINITY, sum = 0.f;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, stats(i, row).x);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    if (top == -INFINITY) top = 0.f;
    for (int i = lane; i < parts; i += 32) {
      const float2 s = stats(i, row);
      sum += s.y * exp2f(s.x - top);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
    for (int i0 = warp; i0 < parts; i0 += kCombineWarps * kBatch) {
      if (i0 != warp) batch(i0);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (i0 + j * kCombineWarps >= parts) break;
        const float weight = exp2f(tops[j] - top);
#pragma unroll
        for (int c = 0; c < kPer; ++c) acc[c] = fmaf(weight, x[j][c], acc[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < kPer / 2; ++c)
      *reinterpret_cast<float2*>(&sums[warp][c * 64 + lane * 2]) = make_float2(acc[2 * c], acc[2 * c + 1]);
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int c = 0; c < kPer; ++c) {
        acc[c] = 0.f;
        for (int w = 0; w < kCombineWarps; ++w) acc[c] += sums[w][(c / 2) * 64 + lane * 2 + (c & 1)];
      }
      write(row, acc, sum);
    }
    __syncthreads();
  }
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

}  // namespace gdnattn
